// The 8-bit layer's element passes: token quantization with the layer's input transforms, and the
// output transforms.
//
//   quant_*_kernel        x' = V S_X^-1 x, a = max |x'| per token, s = a / 127,
//                         q = rint(x' / s) (of the exact quotient, ties to even), sum = sum q
//   out_*_kernel          y = S_G^-1 U^T y' (signs after the Hadamard blocks, which are symmetric)
//
// Hadamard stages commute, so each of them runs where its elements share a thread. A row takes three
// phases, with the row in shared memory between them:
//   groups   of 4 neighbours, and for long blocks 2, 4 or 8 of them that differ in the top bits of
//            their place in the block (2 bits, and up to 3 from the top)
//   columns  2 .. 32 elements that are 32 apart (index bits 5 .. 9)
//   strips   of 32 neighbours (bits 2 .. 4, or 0 .. 4)
// Groups touch device memory in whole lines, with the channel scales and signs they need, columns do
// for fp32. The token pass ends with the strips, which stay in registers until the token's scale is
// known; the output pass takes columns, strips, groups (short blocks have a kernel of their own).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int TQ_MAX_THREADS = 384;
constexpr int TQ_CTAS = 2;        // of that size per SM (85 registers a thread)
constexpr int UNIT_THREADS = 512; // out_units_kernel
constexpr int TQ_THREADS = 256;   // unrotated tokens
constexpr int TQ_HOLD = 6;        // units a thread keeps there

__device__ __forceinline__ void tq_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void tq_prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void tq_launch_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Eight elements from j0 on, zero past d. VEC: every pointer and row is 16-byte aligned and d is a
// multiple of 8.
template <bool VEC>
__device__ __forceinline__ void tq_load8(const float* p, int j0, int d, float (&v)[8]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = reinterpret_cast<const float4*>(p + j0)[i];
      v[4 * i] = f.x;
      v[4 * i + 1] = f.y;
      v[4 * i + 2] = f.z;
      v[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j0 + e < d ? p[j0 + e] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void tq_load8(const __nv_bfloat16* p, int j0, int d, float (&v)[8]) {
  if (VEC) {
    const uint4 r = *reinterpret_cast<const uint4*>(p + j0);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j0 + e < d ? __bfloat162float(p[j0 + e]) : 0.f;
  }
}
// Eight elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 r;
  template <bool VEC>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int j0, int d) {
    if (VEC) {
      r = *reinterpret_cast<const uint4*>(p + j0);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = j0 + 2 * k < d ? h[j0 + 2 * k] : 0u;
        const uint32_t hi = j0 + 2 * k + 1 < d ? h[j0 + 2 * k + 1] : 0u;
        w[k] = lo | (hi << 16);
      }
      r = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // the largest magnitude's bit pattern as fp32 (infinities and NaN come out largest)
  __device__ __forceinline__ uint32_t most() const {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = max2(max2(r.x & k, r.y & k), max2(r.z & k, r.w & k));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float r[8];
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p, int j0, int d) {
    tq_load8<VEC>(p, j0, d, r);
  }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(r[e]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r[e];
  }
};
template <bool VEC>
__device__ __forceinline__ void tq_signs8(const int8_t* p, int j0, int d, float (&v)[8]) {
  uint32_t w[2] = {0u, 0u};
  if (VEC) {
    const uint2 r = *reinterpret_cast<const uint2*>(p + j0);
    w[0] = r.x;
    w[1] = r.y;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j0 + e < d) w[e >> 2] |= (static_cast<uint32_t>(p[j0 + e]) & 0xffu) << (8 * (e & 3));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = __uint_as_float(__float_as_uint(v[e]) ^ ((w[e >> 2] << (24 - 8 * (e & 3))) & 0x80000000u));
}
template <bool VEC>
__device__ __forceinline__ void tq_store8(float* p, int j0, int d, const float (&v)[8]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<float4*>(p + j0)[i] =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j0 + e < d) p[j0 + e] = v[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void tq_store8(__nv_bfloat16* p, int j0, int d, const float (&v)[8]) {
  if (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p + j0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j0 + e < d) p[j0 + e] = __float2bfloat16_rn(v[e]);
  }
}

// ---- pairs of fp32 in one 64-bit register pair (packed arithmetic)
__device__ __forceinline__ uint64_t tq_pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 tq_unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t tq_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t tq_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t tq_sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// a / b to 2 ulp (b normal, below 2^126), subnormal a and quotients included: with them flushed to zero a
// rotated token of subnormal entries lost its codes. 2 ulp are small beside the roundings of a rotation's
// log2(b) stages. Rotated 2048 x 8192: 27.2 us flushed, 28.0 like this, 35.5 with the quotient rounded to
// nearest; one token through a layer of 8192 x 8192: 22.7, 22.9, 28.8.
__device__ __forceinline__ float tq_quotient(float a, float b) {
  float r;
  asm("div.approx.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Stages of the index bits inside a register array of N elements, for blocks of b: the first between
// neighbours, the others on pairs.
template <int N>
__device__ __forceinline__ void butterflies(float (&v)[N], int b) {
  if (b == 1) return;
  if constexpr (N == 2) {
    const float u = v[0], t = v[1];
    v[0] = u + t;
    v[1] = u - t;
  } else {
    uint64_t p[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) p[j] = tq_pack2(v[2 * j] + v[2 * j + 1], v[2 * j] - v[2 * j + 1]);
#pragma unroll
    for (int h = 1; h < N / 2; h <<= 1) {
      if (2 * h >= b) break;
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        if (!(j & h)) {
          const uint64_t u = p[j], t = p[j + h];
          p[j] = tq_add2(u, t);
          p[j + h] = tq_sub2(u, t);
        }
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float2 f = tq_unpack2(p[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}

// Stages of the pair-index bits h = LO, 2 LO .. below HI of a pair array (element bits one higher).
template <int N>
__device__ __forceinline__ void pair_stages(uint64_t (&p)[N], int lo, int hi) {
#pragma unroll
  for (int h = 1; h < N; h <<= 1) {
    if (h < lo || h >= hi) continue;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!(j & h)) {
        const uint64_t u = p[j], t = p[j + h];
        p[j] = tq_add2(u, t);
        p[j + h] = tq_sub2(u, t);
      }
  }
}

// The row in shared memory: strips of 32 elements, whose 8 groups of 4 are permuted by the strip's
// number, so that neighbouring groups, the same group of neighbouring strips and the columns of a
// strip all lie in different banks. Word offset of element e:
__device__ __forceinline__ int tq_at(int e) {
  return (e & ~31) | ((e ^ (((e >> 5) & 7) << 2)) & 31);
}
__device__ __forceinline__ ulonglong2* tq_group(float* xs, int g) {
  return reinterpret_cast<ulonglong2*>(xs + tq_at(4 * g));
}
__device__ __forceinline__ void strip_get(float* xs, int c, uint64_t (&p)[16]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const ulonglong2 w = *tq_group(xs, 8 * c + g);
    p[2 * g] = w.x;
    p[2 * g + 1] = w.y;
  }
}
__device__ __forceinline__ void strip_put(float* xs, int c, const uint64_t (&p)[16]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) *tq_group(xs, 8 * c + g) = make_ulonglong2(p[2 * g], p[2 * g + 1]);
}

// Stages of the index bits [SH, SH + R) of len elements (a multiple of 2^(SH + R), SH >= 5), in
// shared memory or, with GLOBAL, taken from device memory.
template <int R, int SH, bool GLOBAL>
__device__ __forceinline__ void column_pass(float* xs, const float* from, int len) {
  constexpr int N = 1 << R;
#pragma unroll(N < 16 ? 16 / N : 1)
  for (int w = threadIdx.x; w < (len >> R); w += blockDim.x) {
    const int e = (w & ((1 << SH) - 1)) | ((w >> SH) << (SH + R));
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = GLOBAL ? from[e + (j << SH)] : xs[tq_at(e | (j << SH))];
    butterflies<N>(v, N);
#pragma unroll
    for (int j = 0; j < N; ++j) xs[tq_at(e | (j << SH))] = v[j];
  }
  __syncthreads();
}
// Bits 5 .. 9 of blocks of 2^L, in shared memory.
__device__ __forceinline__ void columns(float* xs, int len, int L) {
  switch (L) {
    case 4:
    case 5: break;
    case 6: column_pass<1, 5, false>(xs, xs, len); break;
    case 7: column_pass<2, 5, false>(xs, xs, len); break;
    case 8: column_pass<3, 5, false>(xs, xs, len); break;
    case 9: column_pass<4, 5, false>(xs, xs, len); break;
    default: column_pass<5, 5, false>(xs, xs, len);
  }
}
// What columns, strips and three top bits leave of blocks above 8192.
__device__ __forceinline__ void middle_bits(float* xs, int len, int L) {
  if (L == 14) column_pass<1, 10, false>(xs, xs, len);
  if (L == 15) column_pass<2, 10, false>(xs, xs, len);
}
// The top bits that the groups take.
int top_bits(int log_b) { return std::min(3, std::max(0, log_b - 10)); }

// Largest magnitude; a NaN stays.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

struct QuantArgs {
  const void* x;
  int64_t ld_x;
  int d, b, log_b;
  const float* s_x;        // NULL: no scaling
  const int8_t* sign_in;   // NULL: no rotation
  float inv_sqrt_b;
  int8_t* q;
  int64_t ld_q;
  float* tok_scale;
  int32_t* tok_sum;
  int chained;             // the kernel behind it is the layer's product: let it start early
};

// Eight codes rint(x / s) (of the exact quotient, ties to even) as two words, for |x| <= 127 s
// (1 + 2^-23) and a normal s. Adding 1.5 2^23 to x inv_s rounds it to an integer q, whose low byte is
// the float's low byte. q is off by at most one, and only next to a half: there the remainder x - q s is
// exact in fp32 (a multiple of the smaller ulp and below 2^24 of them), so that 2 |x - q s| against s
// tells. (A test of the quotient's estimate instead sent most warps of bf16 tokens into the slow branch:
// their values repeat, and so do those next to a half; 4096 x 11008 took 60 us.)
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float s, float inv_s, int& sum) {
  const uint64_t magic = tq_pack2(12582912.f, 12582912.f), unmagic = tq_pack2(-12582912.f, -12582912.f);
  const uint64_t inv2 = tq_pack2(inv_s, inv_s), neg2 = tq_pack2(-s, -s);
  uint32_t t[8];
  float r[8];
  float off = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t v = tq_pack2(x[2 * k], x[2 * k + 1]);
    const uint64_t f = tq_fma2(v, inv2, magic);
    const float2 d = tq_unpack2(tq_fma2(tq_add2(f, unmagic), neg2, v));     // x - q s
    r[2 * k] = d.x;
    r[2 * k + 1] = d.y;
    off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
    const float2 b = tq_unpack2(f);
    t[2 * k] = __float_as_uint(b.x);
    t[2 * k + 1] = __float_as_uint(b.y);
  }
  if (off + off >= s) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fabsf(r[k]) + fabsf(r[k]);
      if (a > s || (a == s && (t[k] & 1u))) t[k] += r[k] > 0.f ? 1u : 0xffffffffu;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040),
                       __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040), 0x5410);
    sum = __dp4a(static_cast<int>(w[i]), 0x01010101, sum);
  }
  return make_uint2(w[0], w[1]);
}

// What both quantization kernels do around a token's transformed values.
struct TokenScale {
  float s, inv_s;
  bool zero;               // no codes: nothing to scale, or not finite
};
// From the largest magnitude (as a bit pattern: infinities and NaN come out largest) of each thread.
__device__ __forceinline__ TokenScale token_scale(uint32_t m, uint32_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, lane < (blockDim.x >> 5) ? red[lane] : 0u);
  const bool finite = m < 0x7f800000u;
  TokenScale r;
  r.s = __uint_as_float(m) / 127.f;
  r.zero = !finite || r.s < 1.17549435e-38f;
  if (!finite) r.s = __int_as_float(0x7fc00000);
  else if (r.zero) r.s = 1.f;
  r.inv_s = 1.f / r.s;
  return r;
}
template <bool VEC>
__device__ __forceinline__ void put_codes(int8_t* q, int c, int d, const float (&v)[8],
                                          const TokenScale& ts, int& sum) {
  uint2 w = make_uint2(0u, 0u);
  if (!ts.zero) w = quant8(v, ts.s, ts.inv_s, sum);
  if (VEC || 8 * c + 8 <= d) {
    *reinterpret_cast<uint2*>(q + 8 * c) = w;
  } else {
    const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * c + e < d) q[8 * c + e] = static_cast<int8_t>((ws[e >> 2] >> (8 * (e & 3))) & 0xffu);
  }
}
__device__ __forceinline__ void token_out(const QuantArgs& a, int64_t t, float s, int sum, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = __reduce_add_sync(0xffffffffu, lane < (blockDim.x >> 5) ? red[lane] : 0);
    if (lane == 0) {
      a.tok_scale[t] = s;
      a.tok_sum[t] = sum;
    }
  }
}

// Four elements from j0 on. VEC: in one load.
template <bool VEC>
__device__ __forceinline__ float4 tq_load4(const float* p, int j0) {
  if (VEC) return *reinterpret_cast<const float4*>(p + j0);
  return make_float4(p[j0], p[j0 + 1], p[j0 + 2], p[j0 + 3]);
}
template <bool VEC>
__device__ __forceinline__ uint32_t tq_signs4(const int8_t* p, int j0) {
  if (VEC) return *reinterpret_cast<const uint32_t*>(p + j0);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) w |= (static_cast<uint32_t>(p[j0 + e]) & 0xffu) << (8 * e);
  return w;
}
__device__ __forceinline__ float tq_signed(float v, uint32_t signs, int e) {
  return __uint_as_float(__float_as_uint(v) ^ ((signs << (24 - 8 * e)) & 0x80000000u));
}
// Four signed elements.
template <bool VEC>
__device__ __forceinline__ float4 tq_load4(const float* p, int j0, uint32_t signs) {
  const float4 v = tq_load4<VEC>(p, j0);
  return make_float4(tq_signed(v.x, signs, 0), tq_signed(v.y, signs, 1), tq_signed(v.z, signs, 2),
                     tq_signed(v.w, signs, 3));
}
template <bool VEC>
__device__ __forceinline__ float4 tq_load4(const __nv_bfloat16* p, int j0, uint32_t signs) {
  uint2 r;
  if (VEC) {
    r = *reinterpret_cast<const uint2*>(p + j0);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p) + j0;
    r = make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                   h[2] | (static_cast<uint32_t>(h[3]) << 16));
  }
  r.x ^= __byte_perm(signs, 0u, 0x1404) & 0x80008000u;   // two sign bits at once
  r.y ^= __byte_perm(signs, 0u, 0x3424) & 0x80008000u;
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}

// Tokens whose Hadamard blocks are above 8: one CTA per token, which holds the row in shared memory.
// Bound by the latency of a row's steps, one behind the other, and by instructions (about 37 a warp for 32
// elements, 64 % of the issue slots of active cycles): 2048 x 8192 bf16 in 30 us, 1.7 TB/s. With 8
// neighbours a thread and four passes it took 38.5 us.
template <typename T, bool VEC, int TOP>
__global__ void __launch_bounds__(TQ_MAX_THREADS, TQ_CTAS) quant_rotated_kernel(QuantArgs a) {
  extern __shared__ __align__(16) float xs[];
  __shared__ uint32_t red_max[TQ_MAX_THREADS / 32];
  __shared__ int red_sum[TQ_MAX_THREADS / 32];
  constexpr int G = 1 << TOP;      // groups that meet in a thread
  constexpr int U = 8 / G;         // sets of them under way together
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
  const int tid = threadIdx.x, nthr = blockDim.x;
  tq_wait();                       // x may come from the kernel before
  if (a.chained) tq_launch_next();
  const int log_step = a.log_b - TOP - 2, sets = a.d >> (TOP + 2);
  for (int w0 = tid; w0 < sets; w0 += U * nthr) {
    float4 v[U][G];
    int g0[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = min(w0 + u * nthr, sets - 1);
      g0[u] = (w & ((1 << log_step) - 1)) | ((w >> log_step) << (log_step + TOP));
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int j0 = 4 * (g0[u] + (j << log_step));
        v[u][j] = tq_load4<VEC>(x, j0, tq_signs4<VEC>(a.sign_in, j0));
      }
    }
    if (a.s_x) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float4 s = tq_load4<VEC>(a.s_x, 4 * (g0[u] + (j << log_step)));
          v[u][j] = make_float4(tq_quotient(v[u][j].x, s.x), tq_quotient(v[u][j].y, s.y),
                                tq_quotient(v[u][j].z, s.z), tq_quotient(v[u][j].w, s.w));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float e[4 * G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        e[4 * j] = v[u][j].x;
        e[4 * j + 1] = v[u][j].y;
        e[4 * j + 2] = v[u][j].z;
        e[4 * j + 3] = v[u][j].w;
      }
      butterflies<4 * G>(e, 4 * G);
      if (w0 + u * nthr < sets) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          *tq_group(xs, g0[u] + (j << log_step)) =
              make_ulonglong2(tq_pack2(e[4 * j], e[4 * j + 1]), tq_pack2(e[4 * j + 2], e[4 * j + 3]));
      }
    }
  }
  const int strips = (a.d + 31) >> 5;
  if ((a.d & 31) && tid < 4)       // blocks of 16: the last strip's other half
    *tq_group(xs, (a.d >> 2) + tid) = make_ulonglong2(0, 0);
  __syncthreads();
  columns(xs, a.d, a.log_b);
  middle_bits(xs, a.d, a.log_b);
  float amax = 0.f;
  int sum = 0;
  int8_t* q = a.q + t * a.ld_q;
  auto last_stages = [&](uint64_t (&p)[16]) {
    pair_stages(p, 2, 8);          // bits 2, 3
    if (a.log_b > 4) pair_stages(p, 8, 16);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = tq_unpack2(p[i]);
      amax = max_abs(max_abs(amax, f.x), f.y);
    }
  };
  auto codes = [&](int c, const uint64_t (&p)[16], const TokenScale& ts) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (32 * c + 16 * h >= a.d) break;
      uint2 w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = tq_unpack2(p[8 * h + 4 * i + k]);
          v[2 * k] = f.x * a.inv_sqrt_b;
          v[2 * k + 1] = f.y * a.inv_sqrt_b;
        }
        w[i] = make_uint2(0u, 0u);
        if (!ts.zero) w[i] = quant8(v, ts.s, ts.inv_s, sum);
      }
      *reinterpret_cast<uint4*>(q + 32 * c + 16 * h) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    }
  };
  auto scale = [&]() {
    return token_scale(__float_as_uint(amax * a.inv_sqrt_b) & 0x7fffffffu, red_max);
  };
  float s;
  if (strips <= nthr) {
    uint64_t p[16];
    if (tid < strips) {
      strip_get(xs, tid, p);
      last_stages(p);
    }
    const TokenScale ts = scale();
    if (tid < strips) codes(tid, p, ts);
    s = ts.s;
  } else {
    for (int c = tid; c < strips; c += nthr) {
      uint64_t p[16];
      strip_get(xs, c, p);
      last_stages(p);
      strip_put(xs, c, p);
    }
    const TokenScale ts = scale();
    for (int c = tid; c < strips; c += nthr) {
      uint64_t p[16];
      strip_get(xs, c, p);
      codes(c, p, ts);
    }
    s = ts.s;
  }
  token_out(a, t, s, sum, red_sum);
}

// Tokens without a rotation, or with blocks of at most 8: one CTA per token. A thread keeps its first
// TQ_HOLD units as they came (all of them up to a width of 12288) and reads others again.
// 4096 x 11008 bf16: 33 us, 4.1 TB/s, 57 % of the issue slots (fp32 43 us, 5.2 TB/s); the floor is 21
// us. Each row waits for its maximum between its loads and its stores, and four rows per SM do not hide
// all of that.
template <typename T, bool VEC>
__global__ void __launch_bounds__(TQ_THREADS, 4) quant_plain_kernel(QuantArgs a) {
  __shared__ uint32_t red_max[TQ_THREADS / 32];
  __shared__ int red_sum[TQ_THREADS / 32];
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int units = (a.d + 7) >> 3;
  // S_X^-1 x, the signs and the stages
  auto take = [&](int c, const Raw8<T>& raw, float (&v)[8]) {
    raw.get(v);
    if (a.s_x) {
      float s[8];
      tq_load8<VEC>(a.s_x, 8 * c, a.d, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = VEC || 8 * c + e < a.d ? v[e] / s[e] : 0.f;
    }
    if (a.sign_in) {
      tq_signs8<VEC>(a.sign_in, 8 * c, a.d, v);
      butterflies<8>(v, a.b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.inv_sqrt_b;
    }
  };
  tq_wait();                       // x may come from the kernel before
  if (a.chained) tq_launch_next();
  Raw8<T> raw[TQ_HOLD];
#pragma unroll
  for (int h = 0; h < TQ_HOLD; ++h)
    if (tid + h * nthr < units) raw[h].template load<VEC>(x, 8 * (tid + h * nthr), a.d);
  uint32_t m = 0;
  const bool plain = !a.s_x && !a.sign_in;
  auto most = [&](int c, const Raw8<T>& r) {
    if (plain) {
      m = max(m, r.most());
      return;
    }
    float v[8];
    take(c, r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  };
#pragma unroll
  for (int h = 0; h < TQ_HOLD; ++h)
    if (tid + h * nthr < units) most(tid + h * nthr, raw[h]);
  for (int c = tid + TQ_HOLD * nthr; c < units; c += nthr) {
    Raw8<T> r;
    r.template load<VEC>(x, 8 * c, a.d);
    most(c, r);
  }
  const TokenScale ts = token_scale(m, red_max);
  int sum = 0;
  int8_t* q = a.q + t * a.ld_q;
#pragma unroll
  for (int h = 0; h < TQ_HOLD; ++h)
    if (tid + h * nthr < units) {
      float v[8];
      take(tid + h * nthr, raw[h], v);
      put_codes<VEC>(q, tid + h * nthr, a.d, v, ts, sum);
    }
  for (int c = tid + TQ_HOLD * nthr; c < units; c += nthr) {
    Raw8<T> r;
    r.template load<VEC>(x, 8 * c, a.d);
    float v[8];
    take(c, r, v);
    put_codes<VEC>(q, c, a.d, v, ts, sum);
  }
  token_out(a, t, ts.s, sum, red_sum);
}

struct OutArgs {
  const float* yp;
  int64_t ld_yp;
  int d, b, log_b, span;
  const float* s_g;        // NULL: no scaling
  const int8_t* sign_out;
  float inv_sqrt_b;
  void* y;
  int64_t ld_y;
};

// The output kernels start while the product still runs: what they read last comes to L2 meanwhile.
__device__ __forceinline__ void prefetch_channels(const OutArgs& a, int j0, int len) {
  for (int c = 32 * threadIdx.x; c < len; c += 32 * blockDim.x) {
    if (a.s_g) tq_prefetch(a.s_g + j0 + c);
    if ((c & 127) == 0) tq_prefetch(a.sign_out + j0 + c);
  }
}

// Element i of a row in shared memory sits at i + i / 32: the 8 consecutive elements of 32 threads,
// and 32 consecutive elements, lie in different banks.
__device__ __forceinline__ int units_at(int i) { return i + (i >> 5); }

// Stages of the index bits [SH, SH + R) of len elements (a multiple of 2^(SH + R)).
template <int R, int SH>
__device__ __forceinline__ void unit_pass(float* xs, int len) {
  constexpr int N = 1 << R;
  // In the first pass (SH = 3) eight threads share the low bits; four groups of them would meet in
  // the same banks 2^(3 + R) apart, and do not 256 apart: the bits of w above 3 that a warp counts
  // through become index bits 8 and 9.
  constexpr int B8 = SH == 3 ? 5 - R : 0;            // bits between 3 + R and 8
  const bool spread = SH == 3 && (len & 1023) == 0;
  for (int w = threadIdx.x; w < (len >> R); w += blockDim.x) {
    int hi = w >> SH;
    if (spread)
      hi = (hi & ~((4 << B8) - 1)) | ((hi & 3) << B8) | ((hi >> 2) & ((1 << B8) - 1));
    float* const p = xs + units_at((w & ((1 << SH) - 1)) | (hi << (SH + R)));
    // units_at of 2^SH j past it (for SH = 3 its low five bits are below 8)
    auto off = [](int j) { return (j << SH) + ((j << SH) >> 5); };
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = p[off(j)];
    butterflies<N>(v, N);
#pragma unroll
    for (int j = 0; j < N; ++j) p[off(j)] = v[j];
  }
  __syncthreads();
}

// The stages above the first three of every block of 2^L (3 < L <= 10). Written out per L, so that
// every offset is a constant of its instruction.
__device__ __forceinline__ void unit_passes(float* xs, int len, int L) {
  switch (L) {
    case 4: unit_pass<1, 3>(xs, len); break;
    case 5: unit_pass<2, 3>(xs, len); break;
    case 6: unit_pass<3, 3>(xs, len); break;
    case 7: unit_pass<4, 3>(xs, len); break;
    case 10:
      unit_pass<4, 3>(xs, len);
      unit_pass<3, 7>(xs, len);
      break;
    default:
      unit_pass<3, 3>(xs, len);
      if (L == 8) unit_pass<2, 6>(xs, len);
      else unit_pass<3, 6>(xs, len);
  }
}

// Blocks up to 1024. One CTA per (token, span of whole blocks). A thread takes units of 8 neighbours
// (their three stages in registers), the other stages go through shared memory in one or two passes of
// up to 16 elements a thread.
template <typename Y, bool VEC>
__global__ void __launch_bounds__(UNIT_THREADS, 3) out_units_kernel(OutArgs a) {
  extern __shared__ float xs[];
  const int64_t t = blockIdx.y;
  const int j0 = blockIdx.x * a.span;
  const int len = min(a.span, a.d - j0);
  const int units = (len + 7) >> 3;
  const float* yp = a.yp + t * a.ld_yp + j0;
  Y* y = static_cast<Y*>(a.y) + t * a.ld_y + j0;
  auto finish = [&](int c, float (&v)[8]) {
    tq_signs8<VEC>(a.sign_out + j0, 8 * c, len, v);
    if (a.s_g) {
      float s[8];
      tq_load8<VEC>(a.s_g + j0, 8 * c, len, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tq_quotient(v[e] * a.inv_sqrt_b, s[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.inv_sqrt_b;
    }
    tq_store8<VEC>(y, 8 * c, len, v);
  };
  prefetch_channels(a, j0, len);
  tq_wait();
  if (a.b <= 8) {
    for (int c = threadIdx.x; c < units; c += blockDim.x) {
      float v[8];
      tq_load8<VEC>(yp, 8 * c, len, v);
      butterflies<8>(v, a.b);
      finish(c, v);
    }
    return;
  }
#pragma unroll 2
  for (int c = threadIdx.x; c < units; c += blockDim.x) {
    float v[8];
    tq_load8<VEC>(yp, 8 * c, len, v);
    butterflies<8>(v, 8);
    float* p = xs + units_at(8 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = v[e];
  }
  __syncthreads();
  unit_passes(xs, len, a.log_b);
  for (int c = threadIdx.x; c < units; c += blockDim.x) {
    const float* p = xs + units_at(8 * c);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e];
    finish(c, v);
  }
}

template <bool VEC>
__device__ __forceinline__ void tq_store4(float* p, int j0, const float (&v)[4]) {
  if (VEC) {
    *reinterpret_cast<float4*>(p + j0) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[j0 + e] = v[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void tq_store4(__nv_bfloat16* p, int j0, const float (&v)[4]) {
  if (VEC) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p + j0) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                   *reinterpret_cast<const uint32_t*>(&hi));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[j0 + e] = __float2bfloat16_rn(v[e]);
  }
}

// Blocks of 2048 and more. One CTA per (token, span of whole blocks): columns, strips, groups.
template <typename Y, bool VEC, int TOP>
__global__ void __launch_bounds__(TQ_MAX_THREADS, TQ_CTAS)
    out_transform_kernel(OutArgs a) {
  extern __shared__ __align__(16) float xs[];
  constexpr int G = 1 << TOP, U = 8 / G;
  const int64_t t = blockIdx.y;
  const int j0 = blockIdx.x * a.span;
  const int len = min(a.span, a.d - j0);
  const int tid = threadIdx.x, nthr = blockDim.x;
  Y* y = static_cast<Y*>(a.y) + t * a.ld_y + j0;
  prefetch_channels(a, j0, len);
  tq_wait();
  column_pass<5, 5, true>(xs, a.yp + t * a.ld_yp + j0, len);
  for (int c = tid; c < len >> 5; c += nthr) {
    uint64_t p[16];
    strip_get(xs, c, p);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = tq_unpack2(p[i]);
      p[i] = tq_pack2(f.x + f.y, f.x - f.y);
    }
    pair_stages(p, 1, 16);
    strip_put(xs, c, p);
  }
  __syncthreads();
  middle_bits(xs, len, a.log_b);
  const int log_step = a.log_b - TOP - 2, sets = len >> (TOP + 2);
  const float* s_g = a.s_g ? a.s_g + j0 : nullptr;
  for (int w0 = tid; w0 < sets; w0 += U * nthr) {
    uint64_t p[U][2 * G];
    uint32_t sg[U][G];
    int g0[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = min(w0 + u * nthr, sets - 1);
      g0[u] = (w & ((1 << log_step) - 1)) | ((w >> log_step) << (log_step + TOP));
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int g = g0[u] + (j << log_step);
        sg[u][j] = tq_signs4<VEC>(a.sign_out + j0, 4 * g);
        const ulonglong2 r = *tq_group(xs, g);
        p[u][2 * j] = r.x;
        p[u][2 * j + 1] = r.y;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (w0 + u * nthr >= sets) break;
      pair_stages(p[u], 2, 2 * G);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float2 lo = tq_unpack2(p[u][2 * j]), hi = tq_unpack2(p[u][2 * j + 1]);
        float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = tq_signed(v[e] * a.inv_sqrt_b, sg[u][j], e);
        const int c0 = 4 * (g0[u] + (j << log_step));
        if (s_g) {
          const float4 s = tq_load4<VEC>(s_g, c0);
          v[0] = tq_quotient(v[0], s.x);
          v[1] = tq_quotient(v[1], s.y);
          v[2] = tq_quotient(v[2], s.z);
          v[3] = tq_quotient(v[3], s.w);
        }
        tq_store4<VEC>(y, c0, v);
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// threads for `units` units of 8: two a thread, evenly
int unit_threads(int units) {
  const int per = std::max(2, (units + UNIT_THREADS - 1) / UNIT_THREADS);
  return std::max(32, ((units + per - 1) / per + 31) / 32 * 32);
}
size_t unit_smem(int len) { return static_cast<size_t>(33) * ((len + 31) / 32) * sizeof(float); }
// threads for a row of len elements: a strip each, or several, evenly
int row_threads(int len) {
  const int strips = (len + 31) / 32;
  const int per = (strips + TQ_MAX_THREADS - 1) / TQ_MAX_THREADS;
  return ((strips + per - 1) / per + 31) / 32 * 32;
}
int pow2_part(int d) { return d & (-d); }
int log2_of(int b) {
  int l = 0;
  while ((1 << l) < b) ++l;
  return l;
}
size_t row_smem(int len) { return static_cast<size_t>((len + 31) / 32) * 32 * sizeof(float); }

// A kernel as a type, so that what is kept for a kernel has a place of its own.
template <auto K>
struct Kern {
  static constexpr auto value = K;
};
// Lets a kernel hold the longest row that it is ever launched with: the limit belongs to the kernel, not
// to the call, and calls of other threads launch it with rows of other lengths.
template <auto K>
kronq_status allow_row(int longest) {
  static std::atomic<uint64_t> allowed{0};
  return allow_smem(reinterpret_cast<const void*>(K), row_smem(longest), allowed);
}

}  // namespace

kronq_status run_quant_tokens(const QuantTokensArgs& q, cudaStream_t stream) {
  QuantArgs a{};
  a.x = q.x;
  a.ld_x = q.ld_x;
  a.d = q.d;
  a.b = pow2_part(q.d);
  a.log_b = log2_of(a.b);
  a.s_x = q.s_x;
  a.sign_in = q.sign_in;
  a.inv_sqrt_b = static_cast<float>(1.0 / std::sqrt(static_cast<double>(a.b)));
  a.q = q.q;
  a.ld_q = q.ld_q;
  a.tok_scale = q.tok_scale;
  a.tok_sum = q.tok_sum;
  a.chained = q.chained;
  const bool smem_row = q.sign_in && a.b > 8;
  const size_t smem = smem_row ? row_smem(q.d) : 0;
  const bool vec = q.d % 8 == 0 && aligned16(q.x) && (q.n == 1 || q.ld_x % 8 == 0) &&
                   aligned16(q.s_x) && aligned16(q.sign_in);
  const int units = (q.d + 7) / 8;
  // unrotated: two units a thread as far as TQ_THREADS go
  const int threads = smem_row ? row_threads(q.d)
                               : std::min(TQ_THREADS, std::max(32, ((units + 1) / 2 + 31) / 32 * 32));
  auto run = [&](auto kern) -> kronq_status {
    if (smem_row) KQ_TRY(allow_row<decltype(kern)::value>(kMaxRotatedWidth));
    return launch_chained(decltype(kern)::value, dim3(q.n), dim3(threads), smem, stream, 1,
                          "quantize_tokens kernel", a);
  };
  auto launch = [&](auto aligned, auto other) { return vec ? run(aligned) : run(other); };
  auto typed = [&](auto x) -> kronq_status {
    using T = decltype(x);
    if (smem_row)
      switch (top_bits(a.log_b)) {
        case 0: return launch(Kern<quant_rotated_kernel<T, true, 0>>(), Kern<quant_rotated_kernel<T, false, 0>>());
        case 1: return launch(Kern<quant_rotated_kernel<T, true, 1>>(), Kern<quant_rotated_kernel<T, false, 1>>());
        case 2: return launch(Kern<quant_rotated_kernel<T, true, 2>>(), Kern<quant_rotated_kernel<T, false, 2>>());
        default: return launch(Kern<quant_rotated_kernel<T, true, 3>>(), Kern<quant_rotated_kernel<T, false, 3>>());
      }
    return launch(Kern<quant_plain_kernel<T, true>>(), Kern<quant_plain_kernel<T, false>>());
  };
  return q.x_dtype == KRONQ_DTYPE_BF16 ? typed(__nv_bfloat16()) : typed(0.f);
}

kronq_status run_out_transform(const float* yp, int64_t ld_yp, int n, int d, const float* s_g,
                               const int8_t* sign_out, void* y, int y_dtype, int64_t ld_y,
                               cudaStream_t stream) {
  OutArgs a{};
  a.yp = yp;
  a.ld_yp = ld_yp;
  a.d = d;
  a.b = pow2_part(d);
  a.log_b = log2_of(a.b);
  a.span = std::max(a.b, 16);
  while (a.span < 1024 && a.span < d) a.span *= 2;
  a.s_g = s_g;
  a.sign_out = sign_out;
  a.inv_sqrt_b = static_cast<float>(1.0 / std::sqrt(static_cast<double>(a.b)));
  a.y = y;
  a.ld_y = ld_y;
  const bool vec = d % 8 == 0 && aligned16(yp) && ld_yp % 4 == 0 && aligned16(y) &&
                   (n == 1 || ld_y % 8 == 0) && aligned16(s_g) && aligned16(sign_out);
  const dim3 grid((d + a.span - 1) / a.span, n);
  // The kernel goes by the block alone, so that a token's bits do not depend on the batch. Either side,
  // us a layer (d_out x d_in, tokens; units / strips): 11008 x 4096, 1: 17.9 / 19.5, 2048: 122 / 121;
  // 8192 x 8192, 1: 22.8 / 21.7, 2048: 173 / 161; 28672 x 8192, 8: 53.7 / 55.8, 2048: 460 / 435.
  const bool units = a.b <= 1024;
  const int threads = units ? unit_threads(a.span / 8) : row_threads(a.span);
  const size_t smem = a.b <= 8 ? 0 : units ? unit_smem(a.span) : row_smem(a.span);
  auto run = [&](auto kern) -> kronq_status {
    if (!units) KQ_TRY(allow_row<decltype(kern)::value>(kMaxOutBlock));
    return launch_chained(decltype(kern)::value, grid, dim3(threads), smem, stream, 1,
                          "output transform kernel", a);
  };
  auto launch = [&](auto aligned, auto other) { return vec ? run(aligned) : run(other); };
  auto typed = [&](auto out) -> kronq_status {
    using Y = decltype(out);
    if (units) return launch(Kern<out_units_kernel<Y, true>>(), Kern<out_units_kernel<Y, false>>());
    switch (top_bits(a.log_b)) {
      case 1: return launch(Kern<out_transform_kernel<Y, true, 1>>(), Kern<out_transform_kernel<Y, false, 1>>());
      case 2: return launch(Kern<out_transform_kernel<Y, true, 2>>(), Kern<out_transform_kernel<Y, false, 2>>());
      default: return launch(Kern<out_transform_kernel<Y, true, 3>>(), Kern<out_transform_kernel<Y, false, 3>>());
    }
  };
  return y_dtype == KRONQ_DTYPE_BF16 ? typed(__nv_bfloat16()) : typed(0.f);
}

}  // namespace kq
