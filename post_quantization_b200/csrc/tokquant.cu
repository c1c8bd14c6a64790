// The 8-bit layer's element passes: token quantization with the layer's input transforms, and the
// output transforms.
//
//   quant_tokens_kernel   x' = V S_X^-1 x, a = max |x'| per token, s = a / 127,
//                         q = rint(x' / s) (of the exact quotient, ties to even), sum = sum q
//   out_transform_kernel  y = S_G^-1 U^T y' (signs after the Hadamard blocks, which are symmetric)
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int TQ_THREADS = 512;

__device__ __forceinline__ float tq_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float tq_load(const float* p) { return *p; }
__device__ __forceinline__ void tq_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void tq_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// element i of a transformed row sits at i + i / 16: the radix-16 passes below are then free of
// bank conflicts
__device__ __forceinline__ int tq_at(int i) { return i + (i >> 4); }

// Unnormalised Hadamard transform of every aligned block of b (a power of two) elements of the
// len (a multiple of b) elements in xs. In the pass over index bits [sh, sh + 4) a thread gathers
// the 16 elements that differ only in those bits and applies four stages in registers.
__device__ __forceinline__ void hadamard_smem(float* xs, int len, int b) {
  const int L = 31 - __clz(b);
  int sh = 0;
  for (; sh + 4 <= L; sh += 4) {
    for (int w = threadIdx.x; w < (len >> 4); w += blockDim.x) {
      const int base = (w & ((1 << sh) - 1)) | ((w >> sh) << (sh + 4));
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = xs[tq_at(base + (j << sh))];
#pragma unroll
      for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!(j & h)) {
            const float u = v[j], t = v[j + h];
            v[j] = u + t;
            v[j + h] = u - t;
          }
#pragma unroll
      for (int j = 0; j < 16; ++j) xs[tq_at(base + (j << sh))] = v[j];
    }
    __syncthreads();
  }
  for (; sh < L; ++sh) {
    const int h = 1 << sh;
    for (int w = threadIdx.x; w < (len >> 1); w += blockDim.x) {
      const int i = ((w >> sh) << (sh + 1)) | (w & (h - 1));
      const float u = xs[tq_at(i)], t = xs[tq_at(i + h)];
      xs[tq_at(i)] = u + t;
      xs[tq_at(i + h)] = u - t;
    }
    __syncthreads();
  }
}

struct QuantArgs {
  const void* x;
  int64_t ld_x;
  int d, b;
  const float* s_x;        // NULL: no scaling
  const int8_t* sign_in;   // NULL: no rotation
  float inv_sqrt_b;
  int8_t* q;
  int64_t ld_q;
  float* tok_scale;
  int32_t* tok_sum;
};

// rint(x / s) for |x| <= 127 s (1 + 2^-23) and a normal s, exactly as the real quotient rounds
// (ties to even): the fp32 estimate is off by at most one, next to a border, and the remainder
// x - q s is exact in fp32 there (it is a multiple of the smaller ulp and below 2^24 of them).
__device__ __forceinline__ int quant_code(float x, float s, float inv_s) {
  const float q0 = rintf(x * inv_s);
  const float r = 2.f * fmaf(-q0, s, x);
  float q = q0;
  if (r > s || (r == s && (static_cast<int>(q0) & 1))) q += 1.f;
  if (r < -s || (r == -s && (static_cast<int>(q0) & 1))) q -= 1.f;
  return static_cast<int>(q);
}

// One CTA per token.
template <typename T>
__global__ void __launch_bounds__(TQ_THREADS) quant_tokens_kernel(QuantArgs a) {
  extern __shared__ float xs[];
  __shared__ uint32_t red_max[TQ_THREADS / 32];
  __shared__ int red_sum[TQ_THREADS / 32];
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool rot = a.sign_in != nullptr;
  auto scaled = [&](int j) {
    const float v = tq_load(x + j);
    return a.s_x ? v / a.s_x[j] : v;
  };
  if (rot) {
    for (int j = tid; j < a.d; j += TQ_THREADS) {
      const float v = scaled(j);
      xs[tq_at(j)] = a.sign_in[j] < 0 ? -v : v;
    }
    __syncthreads();
    hadamard_smem(xs, a.d, a.b);
  }
  auto value = [&](int j) { return rot ? xs[tq_at(j)] * a.inv_sqrt_b : scaled(j); };
  // magnitudes compare as their bit patterns, and infinities and NaN come out largest
  uint32_t m = 0;
  for (int j = tid; j < a.d; j += TQ_THREADS)
    m = max(m, __float_as_uint(value(j)) & 0x7fffffffu);
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) red_max[warp] = m;
  __syncthreads();
  m = 0;
  for (int w = 0; w < TQ_THREADS / 32; ++w) m = max(m, red_max[w]);
  const bool finite = m < 0x7f800000u;
  float s = __uint_as_float(m) / 127.f;
  const bool zero = !finite || s < 1.17549435e-38f;
  if (!finite) s = __int_as_float(0x7fc00000);
  else if (zero) s = 1.f;
  const float inv_s = 1.f / s;
  int sum = 0;
  int8_t* q = a.q + t * a.ld_q;
  for (int j0 = tid * 16; j0 < a.d; j0 += TQ_THREADS * 16) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      int c = 0;
      if (j0 + e < a.d && !zero) c = quant_code(value(j0 + e), s, inv_s);
      sum += c;
      w[e >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (e & 3));
    }
    if (j0 + 16 <= a.d) {
      *reinterpret_cast<uint4*>(q + j0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int e = 0; j0 + e < a.d; ++e)
        q[j0 + e] = static_cast<int8_t>((w[e >> 2] >> (8 * (e & 3))) & 0xffu);
    }
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) red_sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    int tot = 0;
    for (int w = 0; w < TQ_THREADS / 32; ++w) tot += red_sum[w];
    a.tok_scale[t] = s;
    a.tok_sum[t] = tot;
  }
}

struct OutArgs {
  const float* yp;
  int64_t ld_yp;
  int d, b, span;
  const float* s_g;        // NULL: no scaling
  const int8_t* sign_out;
  float inv_sqrt_b;
  void* y;
  int64_t ld_y;
};

// One CTA per (token, span of whole Hadamard blocks).
template <typename Y>
__global__ void __launch_bounds__(256) out_transform_kernel(OutArgs a) {
  extern __shared__ float xs[];
  const int64_t t = blockIdx.y;
  const int j0 = blockIdx.x * a.span;
  const int len = min(a.span, a.d - j0);
  const float* yp = a.yp + t * a.ld_yp + j0;
  for (int j = threadIdx.x; j < len; j += blockDim.x) xs[tq_at(j)] = yp[j];
  __syncthreads();
  hadamard_smem(xs, len, a.b);
  Y* y = static_cast<Y*>(a.y) + t * a.ld_y + j0;
  for (int j = threadIdx.x; j < len; j += blockDim.x) {
    float v = xs[tq_at(j)] * (a.sign_out[j0 + j] < 0 ? -a.inv_sqrt_b : a.inv_sqrt_b);
    if (a.s_g) v = v / a.s_g[j0 + j];
    tq_store(y + j, v);
  }
}

size_t padded_floats(int len) { return static_cast<size_t>(len) + len / 16 + 1; }
int pow2_part(int d) { return d & (-d); }

}  // namespace

kronq_status run_quant_tokens(const QuantTokensArgs& q, cudaStream_t stream) {
  QuantArgs a{};
  a.x = q.x;
  a.ld_x = q.ld_x;
  a.d = q.d;
  a.b = pow2_part(q.d);
  a.s_x = q.s_x;
  a.sign_in = q.sign_in;
  a.inv_sqrt_b = static_cast<float>(1.0 / std::sqrt(static_cast<double>(a.b)));
  a.q = q.q;
  a.ld_q = q.ld_q;
  a.tok_scale = q.tok_scale;
  a.tok_sum = q.tok_sum;
  const size_t smem = q.sign_in ? padded_floats(q.d) * sizeof(float) : 0;
  auto launch = [&](auto kern) -> kronq_status {
    if (smem > 48 * 1024)
      KQ_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem)));
    kern<<<q.n, TQ_THREADS, smem, stream>>>(a);
    return check_launch("quant_tokens_kernel");
  };
  return q.x_dtype == KRONQ_DTYPE_BF16 ? launch(quant_tokens_kernel<__nv_bfloat16>)
                                       : launch(quant_tokens_kernel<float>);
}

kronq_status run_out_transform(const float* yp, int64_t ld_yp, int n, int d, const float* s_g,
                               const int8_t* sign_out, void* y, int y_dtype, int64_t ld_y,
                               cudaStream_t stream) {
  OutArgs a{};
  a.yp = yp;
  a.ld_yp = ld_yp;
  a.d = d;
  a.b = pow2_part(d);
  a.span = a.b;
  while (a.span < 1024 && a.span < d) a.span *= 2;
  a.s_g = s_g;
  a.sign_out = sign_out;
  a.inv_sqrt_b = static_cast<float>(1.0 / std::sqrt(static_cast<double>(a.b)));
  a.y = y;
  a.ld_y = ld_y;
  const size_t smem = padded_floats(a.span) * sizeof(float);
  const dim3 grid((d + a.span - 1) / a.span, n);
  auto launch = [&](auto kern) -> kronq_status {
    if (smem > 48 * 1024)
      KQ_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem)));
    kern<<<grid, 256, smem, stream>>>(a);
    return check_launch("out_transform_kernel");
  };
  return y_dtype == KRONQ_DTYPE_BF16 ? launch(out_transform_kernel<__nv_bfloat16>)
                                     : launch(out_transform_kernel<float>);
}

}  // namespace kq
