// Matrix product in 8-bit integers with scales per token and per channel:
//     y[t][o] = s_t s_o (sum_i q[t][i] c[o][i] - z_o sum_i q[t][i])
// with token codes q (int8, token-major), weight codes c (uint8 or int8, one row per channel) and
// the per-row grid (scale s_o, zero z_o) of the column solve. The integer sums are exact.
//
// The weight codes are the MMA's A operand (M = 128 channels), the tokens its B operand (N = BN):
// an accumulator row (TMEM lane) is then a channel and a column a token, so an epilogue thread
// keeps its channel's grid in registers and 32 lanes store 32 consecutive outputs of one token.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int MM_BM = 128;        // channels per tile (MMA M)
constexpr int MM_BK = 128;        // K bytes per pipeline stage (one 128-byte swizzled row)
constexpr int MM_THREADS = 192;   // TMA producer, MMA issuer, 4 epilogue warps
constexpr int MM_GROUP = 16;      // channel tiles visited together (operand reuse in L2)

struct MmParams {
  const float* tok_scale;
  const int32_t* tok_sum;
  const float* scale;
  const float* zero;              // may be NULL (no zero point)
  const float* out_div;           // may be NULL: s_o is divided by it
  void* y;
  int64_t ld_y;
  int n, d_out, d_in;
  int is_signed;
  int tiles_m, tiles_n, kblocks;
  int* err;
};

// kind::i8: D int32, A unsigned or signed 8-bit, B signed 8-bit, both K-major.
__host__ __device__ constexpr uint32_t mm_idesc(int m, int n, bool a_signed) {
  return (2u << 4) | ((a_signed ? 1u : 0u) << 7) | (1u << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D(tmem) (+)= A(smem desc) * B(smem desc), 8-bit integers, int32 sums.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void mm_tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// A channel's part of the epilogue. The zero-point correction acc - z sum is done in int32 when
// z is a whole number and every value it can reach fits (|q| <= 128 and codes in [lo, lo + 255]:
// 128 d_in max|c - z| < 2^31; intermediate wrap-around is harmless); any other z (a grid whose
// range lies far from zero) takes fp64.
struct Channel {
  float s;         // s_o (over out_div)
  float z;
  int zi;
  bool wide;
};

__device__ __forceinline__ Channel load_channel(const MmParams& p, int ch) {
  Channel c{0.f, 0.f, 0, false};
  if (ch < p.d_out) {
    c.s = p.scale[ch];
    if (p.out_div) c.s = c.s / p.out_div[ch];
    if (p.zero) {
      c.z = p.zero[ch];
      const float lo = p.is_signed ? -128.f : 0.f;
      const float far = fmaxf(fabsf(c.z - lo), fabsf(c.z - (lo + 255.f)));
      // far <= 2^24 keeps the comparison itself exact enough; NaN fails it
      const bool fits = 128.0 * p.d_in * static_cast<double>(far) < 2147483648.0 &&
                        c.z == rintf(c.z);
      c.wide = !fits;
      c.zi = fits ? static_cast<int>(c.z) : 0;
    }
  }
  return c;
}

template <typename Y>
__device__ __forceinline__ Y mm_out(float v);
template <>
__device__ __forceinline__ float mm_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 mm_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// One output from its exact sum; sum_t and s_t are the token's. One fp32 product of the scales
// and one with the (exactly formed, once rounded) sum.
__device__ __forceinline__ float mm_value(const Channel& c, int acc, float s_t, int sum_t) {
  float f;
  if (c.wide)
    f = static_cast<float>(static_cast<double>(acc) -
                           static_cast<double>(c.z) * static_cast<double>(sum_t));
  else
    f = static_cast<float>(static_cast<int>(static_cast<uint32_t>(acc) -
                                            static_cast<uint32_t>(c.zi) *
                                                static_cast<uint32_t>(sum_t)));
  return f * (c.s * s_t);
}

template <int BN>
struct MmCfg {
  static constexpr int A_BYTES = MM_BM * MM_BK;
  static constexpr int B_BYTES = BN * MM_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN >= 256 ? 4 : 6;
  static constexpr int TOK_BYTES = 4 * BN * 8;              // (s_t, sum_t) pairs per epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + TOK_BYTES + 1024 + 256;
  static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
};

__device__ __forceinline__ void mm_tile(const MmParams& p, int t, int& tm, int& tn) {
  const int per_group = MM_GROUP * p.tiles_n;
  const int g = t / per_group, r = t % per_group;
  const int rows = min(MM_GROUP, p.tiles_m - g * MM_GROUP);
  tm = g * MM_GROUP + r % rows;
  tn = r / rows;
}

template <int BN, typename Y>
__global__ void __launch_bounds__(MM_THREADS, 1)
    i8matmul_kernel(const __grid_constant__ CUtensorMap tma_w,
                    const __grid_constant__ CUtensorMap tma_q, const MmParams p) {
  using C = MmCfg<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float2* tok_all = reinterpret_cast<float2*>(smem + STAGES * C::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES + C::TOK_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tma_w);
    prefetch_tensormap(&tma_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        int tm, tn;
        mm_tile(p, t, tm, tn);
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.err, DEV_ERR_TMA_WAIT)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE_BYTES;
          mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
          tma_load_2d(st, &tma_w, &full[s], kb * MM_BK, tm * MM_BM);
          tma_load_2d(st + C::A_BYTES, &tma_q, &full[s], kb * MM_BK, tn * BN);
        }
      }
      if (!ok) {
        for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          mbar_drain(&full[j % STAGES], (j / STAGES) & 1u, 1000000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = mm_idesc(MM_BM, BN, p.is_signed != 0);
      uint32_t it = 0, ui = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x, ++ui) {
        const uint32_t a = ui & 1u, aph = (ui >> 1) & 1u;
        if (!mbar_wait(&tempty[a], aph ^ 1u, abort_flag, p.err, DEV_ERR_MMA_WAIT)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + a * BN;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(&full[s], ph, abort_flag, p.err, DEV_ERR_MMA_WAIT)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t base = smem_u32(smem + s * C::STAGE_BYTES);
#pragma unroll
          for (int kk = 0; kk < MM_BK / 32; ++kk)
            umma_i8(d_tmem, smem_desc_sw128(base + kk * 32, 16, 1024),
                    smem_desc_sw128(base + C::A_BYTES + kk * 32, 16, 1024), idesc,
                    (kb == 0 && kk == 0) ? 0u : 1u);
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&tfull[a]);
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;
    float2* tok = tok_all + q * BN;
    uint32_t ui = 0;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++ui) {
      int tm, tn;
      mm_tile(p, t, tm, tn);
      const uint32_t a = ui & 1u, aph = (ui >> 1) & 1u;
      const int ch = tm * MM_BM + q * 32 + lane;
      const int t0 = tn * BN, cols = min(BN, p.n - t0);
      const Channel c = load_channel(p, ch);
      for (int j = lane; j < cols; j += 32)
        tok[j] = make_float2(p.tok_scale[t0 + j], __int_as_float(p.tok_sum ? p.tok_sum[t0 + j] : 0));
      __syncwarp();
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&tfull[a], aph, abort_flag, p.err, DEV_ERR_EPI_WAIT) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((q * 32u) << 16) + a * BN;
      Y* yp = static_cast<Y*>(p.y) + static_cast<int64_t>(t0) * p.ld_y + ch;
      for (int cb = 0; cb < cols; cb += 16) {
        uint32_t v[16];
        mm_tmem_ld_x16(taddr + cb, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (cb + j < cols && ch < p.d_out) {
            const float2 ts = tok[cb + j];
            yp[static_cast<int64_t>(cb + j) * p.ld_y] =
                mm_out<Y>(mm_value(c, static_cast<int>(v[j]), ts.x, __float_as_int(ts.y)));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[a]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int BN, typename Y>
kronq_status launch_mm(const I8MatmulArgs& a, MmParams p, cudaStream_t stream) {
  using C = MmCfg<BN>;
  p.tiles_m = (a.d_out + MM_BM - 1) / MM_BM;
  p.tiles_n = (a.n + BN - 1) / BN;
  CUtensorMap mw, mq;
  const uint64_t wd[2] = {static_cast<uint64_t>(a.d_in), static_cast<uint64_t>(a.d_out)};
  const uint64_t ws[1] = {static_cast<uint64_t>(a.ld_codes)};
  const uint32_t wb[2] = {MM_BK, MM_BM};
  KQ_TRY(encode_tiled_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, wd, ws, wb,
                          CU_TENSOR_MAP_SWIZZLE_128B));
  const uint64_t qd[2] = {static_cast<uint64_t>(a.d_in), static_cast<uint64_t>(a.n)};
  const uint64_t qs[1] = {static_cast<uint64_t>(a.ld_q)};
  const uint32_t qb[2] = {MM_BK, BN};
  KQ_TRY(encode_tiled_map(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.q, qd, qs, qb,
                          CU_TENSOR_MAP_SWIZZLE_128B));
  auto kern = i8matmul_kernel<BN, Y>;
  KQ_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   C::SMEM_BYTES));
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const int grid = static_cast<int>(std::min<int64_t>(tiles, sm_budget()));
  kern<<<grid, MM_THREADS, C::SMEM_BYTES, stream>>>(mw, mq, p);
  return check_launch("i8matmul_kernel");
}

template <typename Y>
kronq_status dispatch_mm(const I8MatmulArgs& a, const MmParams& p, cudaStream_t stream) {
  if (a.n <= 16) return launch_mm<16, Y>(a, p, stream);
  if (a.n <= 32) return launch_mm<32, Y>(a, p, stream);
  if (a.n <= 64) return launch_mm<64, Y>(a, p, stream);
  if (a.n <= 128) return launch_mm<128, Y>(a, p, stream);
  return launch_mm<256, Y>(a, p, stream);
}

}  // namespace

kronq_status run_i8matmul(const I8MatmulArgs& a, cudaStream_t stream) {
  MmParams p{};
  p.tok_scale = a.tok_scale;
  p.tok_sum = a.tok_sum;
  p.scale = a.scale;
  p.zero = a.zero;
  p.out_div = a.out_div;
  p.y = a.y;
  p.ld_y = a.ld_y;
  p.n = a.n;
  p.d_out = a.d_out;
  p.d_in = a.d_in;
  p.is_signed = a.is_signed;
  p.kblocks = (a.d_in + MM_BK - 1) / MM_BK;
  p.err = device_error_word();
  if (!p.err) return fail(KRONQ_ERR_CUDA, "device error word unavailable");
  return a.y_dtype == KRONQ_DTYPE_BF16 ? dispatch_mm<__nv_bfloat16>(a, p, stream)
                                       : dispatch_mm<float>(a, p, stream);
}

}  // namespace kq
