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
constexpr int MM_THREADS = 192;   // pair kernel: TMA producer, MMA issuer, 4 epilogue warps
constexpr int SP_THREADS = 256;   // split kernel: warps 0 and 1 produce and issue, all 8 finish
constexpr int MM_GROUP = 8;       // channel tiles visited together (operand reuse in L2)

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
  int after_quant;         // the kernel before is the layer's token quantization (see below)
  int before_transform;    // the kernel behind is the layer's output transform
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

// One output from its exact sum.
__device__ __forceinline__ float mm_value(const Channel& c, int acc, float s_t, int sum_t) {
  const float f =
      c.wide ? static_cast<float>(static_cast<double>(acc) -
                                  static_cast<double>(c.z) * static_cast<double>(sum_t))
             : static_cast<float>(static_cast<int>(static_cast<uint32_t>(acc) -
                                                   static_cast<uint32_t>(c.zi) *
                                                       static_cast<uint32_t>(sum_t)));
  return f * (c.s * s_t);
}

// 16 outputs of a channel from their exact sums and the tokens' (s_t, sum_t): one fp32 product of
// the scales and one with the (exactly formed, once rounded) sum.
__device__ __forceinline__ void mm_values(const Channel& c, bool any_wide, const uint32_t (&acc)[16],
                                          const float2 (&tok)[16], float (&out)[16]) {
  if (any_wide && c.wide) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      out[j] = static_cast<float>(static_cast<double>(static_cast<int>(acc[j])) -
                                  static_cast<double>(c.z) *
                                      static_cast<double>(__float_as_int(tok[j].y))) *
               (c.s * tok[j].x);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      out[j] = static_cast<float>(static_cast<int>(
                   acc[j] - static_cast<uint32_t>(c.zi) *
                                static_cast<uint32_t>(__float_as_int(tok[j].y)))) *
               (c.s * tok[j].x);
  }
}

__device__ __forceinline__ void mm_tile(const MmParams& p, int t, int& tm, int& tn) {
  const int per_group = MM_GROUP * p.tiles_n;
  const int g = t / per_group, r = t % per_group;
  const int rows = min(MM_GROUP, p.tiles_m - g * MM_GROUP);
  tm = g * MM_GROUP + r % rows;
  tn = r / rows;
}

// One epilogue warp's part of a tile: 32 channels (lane = channel) by `cols` tokens from t0. All 16
// outputs of a step are formed before any is stored: a store would hold back the loads behind it.
template <typename Y>
__device__ __forceinline__ void store_tile(const MmParams& p, const Channel& c, const float2* tok,
                                           uint32_t taddr, int t0, int cols, int ch) {
  Y* yp = static_cast<Y*>(p.y) + static_cast<int64_t>(t0) * p.ld_y + ch;
  const bool any_wide = __any_sync(0xffffffffu, c.wide);
  const bool in = ch < p.d_out;
  for (int cb = 0; cb < cols; cb += 16, yp += 16 * p.ld_y) {
    uint32_t v[16];
    float2 ts[16];
    float out[16];
    mm_tmem_ld_x16(taddr + cb, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 two = reinterpret_cast<const float4*>(tok + cb)[j];
      ts[2 * j] = make_float2(two.x, two.y);
      ts[2 * j + 1] = make_float2(two.z, two.w);
    }
    tmem_ld_wait();
    mm_values(c, any_wide, v, ts, out);
    if (in) {
      if (cb + 16 <= cols) {
#pragma unroll
        for (int j = 0; j < 16; ++j) yp[j * p.ld_y] = mm_out<Y>(out[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (cb + j < cols) yp[j * p.ld_y] = mm_out<Y>(out[j]);
      }
    }
  }
}

kronq_status byte_map(CUtensorMap* map, const void* base, int64_t ld, int cols, int64_t rows,
                      uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(ld)};
  const uint32_t box[2] = {MM_BK, box_rows};
  return encode_tiled_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

// ---------------------------------------------------------------------------------------------
// Few tokens, or few tiles: K split over a cluster
// ---------------------------------------------------------------------------------------------
// A tile is 128 channels by BN (16 .. 128) tokens; the cl CTAs of a cluster take consecutive parts
// of K, so that a matrix with few channel tiles still has enough CTAs to stream it (two per SM,
// about 90 KB in flight each). Their int32 sums meet in distributed shared memory: the CTAs share
// the tile's outputs out among their threads, each of which adds the cl sums of an output. Integer
// sums: the split changes no bit. A tcgen05 MMA of up to 128 columns takes 63 cycles for 4 KB of
// codes (measured), three times the rate at which HBM delivers them. A thread keeps one channel,
// whose grid it loads before the codes arrive.
// One token, 8192 x 8192 codes: 14.9 us a call, 4.5 TB/s (floor 10.4 us); the stream itself runs near
// HBM's rate, and launch, the first copies' latency and the join of the sums are the rest.
template <int BN>
struct MmCfg {
  static constexpr int A_BYTES = MM_BM * MM_BK;
  static constexpr int B_BYTES = BN * MM_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BN * 8 + 1024 + 128;
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  static_assert(STAGES * STAGE_BYTES >= BN * MM_BM * 4, "the sums reuse the ring");
};

__device__ __forceinline__ void mm_wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void mm_launch_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ uint32_t mm_map(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void mm_cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// grid: x = K part (the cluster), y = channel tile, z = token tile
template <int BN, typename Y>
__global__ void __launch_bounds__(SP_THREADS, 2)
    i8matmul_split_kernel(const __grid_constant__ CUtensorMap tma_w,
                          const __grid_constant__ CUtensorMap tma_q, const MmParams p) {
  using C = MmCfg<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* sums = reinterpret_cast<int*>(smem);          // [token][channel], once the ring is done
  float2* tok = reinterpret_cast<float2*>(smem + STAGES * C::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES + BN * 8);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cl = gridDim.x, rank = blockIdx.x;
  const int tm = blockIdx.y, tn = blockIdx.z;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / cl);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / cl);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
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
  const int cols = min(BN, p.n - tn * BN);
  const int ch = tm * MM_BM + (threadIdx.x & (MM_BM - 1));    // this thread's channel
  Channel c{};

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      // behind the layer's own token quantization, which started after everything before it had
      // ended, the first stages' weight codes need not wait for the kernel before; the tokens do
      const int pre = p.after_quant ? min(STAGES, kb1 - kb0) : 0;
      for (int i = 0; i < pre; ++i) {
        mbar_arrive_expect_tx(&full[i], C::STAGE_BYTES);
        tma_load_2d(smem + i * C::STAGE_BYTES, &tma_w, &full[i], (kb0 + i) * MM_BK, tm * MM_BM);
      }
      mm_wait_previous();
      int it = 0;
      for (; it < kb1 - kb0; ++it) {
        const int s = it % STAGES;
        const uint32_t ph = (it / STAGES) & 1u;
        uint8_t* st = smem + s * C::STAGE_BYTES;
        if (it >= pre) {
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.err, DEV_ERR_TMA_WAIT)) break;
          mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
          tma_load_2d(st, &tma_w, &full[s], (kb0 + it) * MM_BK, tm * MM_BM);
        }
        tma_load_2d(st + C::A_BYTES, &tma_q, &full[s], (kb0 + it) * MM_BK, tn * BN);
      }
      if (it < kb1 - kb0)
        for (int j = max(0, it - STAGES); j < it; ++j)
          mbar_drain(&full[j % STAGES], (j / STAGES) & 1u, 1000000000ull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = mm_idesc(MM_BM, BN, p.is_signed != 0);
      for (int it = 0; it < kb1 - kb0; ++it) {
        const int s = it % STAGES;
        if (!mbar_wait(&full[s], (it / STAGES) & 1u, abort_flag, p.err, DEV_ERR_MMA_WAIT)) break;
        tc_fence_after();
        const uint32_t base = smem_u32(smem + s * C::STAGE_BYTES);
#pragma unroll
        for (int kk = 0; kk < MM_BK / 32; ++kk)
          umma_i8(tmem_base, smem_desc_sw128(base + kk * 32, 16, 1024),
                  smem_desc_sw128(base + C::A_BYTES + kk * 32, 16, 1024), idesc,
                  (it == 0 && kk == 0) ? 0u : 1u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);
    }
  }
  if (p.after_quant) c = load_channel(p, ch);
  mm_wait_previous();
  if (!p.after_quant) c = load_channel(p, ch);
  if (p.before_transform) mm_launch_next();
  if (warp >= 2)
    for (int j = threadIdx.x - 64; j < cols; j += SP_THREADS - 64)
      tok[j] = make_float2(p.tok_scale[tn * BN + j],
                           __int_as_float(p.tok_sum ? p.tok_sum[tn * BN + j] : 0));
  __syncwarp();
  // every role has left its loop; the MMAs and the copies they used are done, or all threads skip the
  // accumulator (its loads are for whole warps)
  const bool ok = __syncthreads_and(mbar_wait(done, 0, abort_flag, p.err, DEV_ERR_EPI_WAIT)) != 0;
  tc_fence_after();
  const int q = warp & 3, half = warp >> 2;
  const uint32_t taddr = tmem_base + ((q * 32u) << 16);
  if (cl == 1) {
    // columns 32 k + 16 half .. + 15: two warps per 32 channels
    if (ok)
      for (int cb = 16 * half; cb < cols; cb += 32)
        store_tile<Y>(p, c, tok + cb, taddr + cb, tn * BN + cb, min(16, cols - cb), ch);
  } else {
    if (ok)
      for (int cb = 16 * half; cb < cols; cb += 32) {
        uint32_t v[16];
        mm_tmem_ld_x16(taddr + cb, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[(cb + j) * MM_BM + q * 32 + lane] = static_cast<int>(v[j]);
      }
    mm_cluster_sync();
    Y* y = static_cast<Y*>(p.y) + static_cast<int64_t>(tn) * BN * p.ld_y + ch;
    // token t of the tile belongs to CTA (t / 2) mod cl, its half t mod 2 of the threads; the
    // remote reads of four tokens are under way together
    uint32_t peer[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      peer[r] = mm_map(sums + q * 32 + lane, r < cl ? r : 0);
    constexpr int U = 4;
    for (int t0 = 2 * rank + half; t0 < cols; t0 += U * 2 * cl) {
      int part[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          part[u][r] = 0;
          const int t = t0 + u * 2 * cl;
          if (r < cl && t < cols)
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(part[u][r])
                         : "r"(peer[r] + t * (MM_BM * 4))
                         : "memory");
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * 2 * cl;
        if (t < cols && ch < p.d_out) {
          int acc = 0;
#pragma unroll
          for (int r = 0; r < 8; ++r) acc += part[u][r];
          y[t * p.ld_y] = mm_out<Y>(mm_value(c, acc, tok[t].x, __float_as_int(tok[t].y)));
        }
      }
    }
  }
  tc_fence_before();
  if (cl > 1)
    mm_cluster_sync();                               // no CTA ends while a peer reads its sums
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------------
// Prompts: two SMs on one tile
// ---------------------------------------------------------------------------------------------
// A pair of CTAs multiplies 256 channels by 256 tokens (tcgen05 cta_group::2, M = 256): each CTA
// holds its 128 channels and half of the tokens, so an operand byte from L2 feeds 1.5 times the
// tensor work of a 128 x 256 tile of one CTA (32 KB per CTA and 128 columns of K instead of 48).
// The even CTA of the pair issues the MMAs; each CTA's producer fills its own shared memory and
// counts the bytes on the even CTA's barrier; accumulators are double-buffered in tensor memory
// (2 x 256 columns), each CTA drains its own 128 channels.
// 4096 tokens, 28672 x 8192: 647 us alone, 2970 TOP/s (732 us, 2630, when the power limit holds the SMs
// at 1.6 GHz); the floor is 560 us. A K block of 128 columns takes about 770 cycles; the tensor cores
// need 512 of them, the shared memory's copies in and operand reads by estimate 704.
// Tiles of 8 channel rows visited together (MM_GROUP); 16, 32 and 64 took 701, 736 and 805 us
// where 8 took 699. One CTA a tile (128 x 256) took 970 us.
namespace pr {
constexpr int BN = 256;
constexpr int A_BYTES = 128 * MM_BK, B_BYTES = 128 * MM_BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 6;
constexpr int TOK_BYTES = 4 * BN * 8;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + TOK_BYTES + 1024 + 256;
constexpr int TMEM_COLS = 512;
}  // namespace pr

// 2-D tiled TMA load into this CTA's shared memory, completion counted on a barrier of the pair.
__device__ __forceinline__ void pr_load(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                        int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pr_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on `bar` of both CTAs when this thread's MMAs so far have completed.
__device__ __forceinline__ void pr_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void pr_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <typename Y>
__global__ void __launch_bounds__(MM_THREADS, 1)
    i8matmul_pair_kernel(const __grid_constant__ CUtensorMap tma_w,
                         const __grid_constant__ CUtensorMap tma_q, const MmParams p) {
  using namespace pr;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float2* tok_all = reinterpret_cast<float2*>(smem + STAGES * STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + TOK_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;                   // the cluster is (2, 1, 1)
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int num_tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);                      // four epilogue warps of each CTA
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tma_w);
    prefetch_tensormap(&tma_q);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  mm_cluster_sync();                                 // the peer's barriers exist
  tc_fence_after();
  mm_wait_previous();
  if (p.before_transform) mm_launch_next();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; t < num_tiles && ok; t += pairs) {
        int tm, tn;
        mm_tile(p, t, tm, tn);
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.err, DEV_ERR_TMA_WAIT)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * STAGE_BYTES;
          // the even CTA's barrier counts both CTAs' bytes (a peer's copy may come before this)
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * STAGE_BYTES);
          const uint32_t bar = mm_map(&full[s], 0);
          pr_load(st, &tma_w, bar, kb * MM_BK, tm * 256 + rank * 128);
          pr_load(st + A_BYTES, &tma_q, bar, kb * MM_BK, tn * BN + rank * 128);
        }
      }
      // after a wait that gave up, the copies in flight land before the CTA ends (both CTAs count on
      // the even one's barriers, which the odd one cannot wait for: it waits out the time)
      if (!ok) {
        for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          mbar_drain(&full[j % STAGES], (j / STAGES) & 1u, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = mm_idesc(256, BN, p.is_signed != 0);
      uint32_t it = 0, ui = 0;
      bool ok = true;
      for (int t = pair; t < num_tiles && ok; t += pairs, ++ui) {
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
          const uint32_t base = smem_u32(smem + s * STAGE_BYTES);
#pragma unroll
          for (int kk = 0; kk < MM_BK / 32; ++kk)
            pr_mma(d_tmem, smem_desc_sw128(base + kk * 32, 16, 1024),
                   smem_desc_sw128(base + A_BYTES + kk * 32, 16, 1024), idesc,
                   (kb == 0 && kk == 0) ? 0u : 1u);
          pr_commit(&empty[s]);
        }
        if (!ok) break;
        pr_commit(&tfull[a]);
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;
    float2* tok = tok_all + q * BN;
    uint32_t ui = 0;
    for (int t = pair; t < num_tiles; t += pairs, ++ui) {
      int tm, tn;
      mm_tile(p, t, tm, tn);
      const uint32_t a = ui & 1u, aph = (ui >> 1) & 1u;
      const int ch = tm * 256 + rank * 128 + q * 32 + lane;
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
      store_tile<Y>(p, c, tok, tmem_base + ((q * 32u) << 16) + a * BN, t0, cols, ch);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) pr_arrive_remote(mm_map(&tempty[a], 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  mm_cluster_sync();       // no MMA, copy or arrival of the pair is under way any more
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

template <typename Y>
kronq_status launch_pair(const I8MatmulArgs& a, MmParams p, cudaStream_t stream) {
  p.tiles_m = (a.d_out + 255) / 256;
  p.tiles_n = (a.n + pr::BN - 1) / pr::BN;
  CUtensorMap mw, mq;
  KQ_TRY(byte_map(&mw, a.codes, a.ld_codes, a.d_in, a.d_out, 128));
  KQ_TRY(byte_map(&mq, a.q, a.ld_q, a.d_in, a.n, 128));
  auto kern = i8matmul_pair_kernel<Y>;
  static std::atomic<uint64_t> allowed{0};
  KQ_TRY(allow_smem(reinterpret_cast<const void*>(kern), pr::SMEM_BYTES, allowed));
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const unsigned ctas =
      2 * static_cast<unsigned>(std::min<int64_t>(tiles, std::max(1, sm_budget() / 2)));
  return launch_chained(kern, dim3(ctas), dim3(MM_THREADS), pr::SMEM_BYTES, stream, 2,
                        "i8matmul_pair_kernel", mw, mq, p);
}

template <int BN, typename Y>
kronq_status launch_split(const I8MatmulArgs& a, const MmParams& p, int cl, cudaStream_t stream) {
  using C = MmCfg<BN>;
  CUtensorMap mw, mq;
  KQ_TRY(byte_map(&mw, a.codes, a.ld_codes, a.d_in, a.d_out, MM_BM));
  KQ_TRY(byte_map(&mq, a.q, a.ld_q, a.d_in, a.n, BN));
  auto kern = i8matmul_split_kernel<BN, Y>;
  static std::atomic<uint64_t> allowed{0};
  KQ_TRY(allow_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, allowed));
  const dim3 grid(cl, (a.d_out + MM_BM - 1) / MM_BM, (a.n + BN - 1) / BN);
  return launch_chained(kern, grid, dim3(SP_THREADS), C::SMEM_BYTES, stream, cl,
                        "i8matmul_split_kernel", mw, mq, p);
}

// Which kernel, and into how many parts K is cut: by estimated nanoseconds, from measurements on one
// B200 (K blocks of 128 columns; a launch's own 4 us left out). A split CTA takes 260 a K block for
// up to 64 tokens, 300 when two share an SM, 360 and 440 for 128 tokens; joining the sums takes
// about 90 a token and CTA of the cluster, a further wave of CTAs 2500; a pair tile 370 a K block.
// Measured on either side of the choices (d_out x d_in, tokens: us):
//   8192 x 8192, 1:    K in 2 / 4 / 8 parts 15.8 / 15.3 / 19.2, pair 23.6
//   1024 x 8192, 1:    K in 1 / 4 / 8 parts 22.0 / 9.5 / 7.4
//   28672 x 8192, 128: K whole / 2 parts 46.8 / 62.3, pair 53.5
//   4096 x 4096, 512:  K whole / 2 parts 15.6 / 20.6, pair 18.5
//   8192 x 8192, 512:  K whole / 2 parts 34.2 / 52.3, pair 29.1
template <typename Y>
kronq_status dispatch_mm(const I8MatmulArgs& a, const MmParams& p, cudaStream_t stream) {
  const int sms = device_sms();
  const int bn = a.n <= 16 ? 16 : a.n <= 32 ? 32 : a.n <= 64 ? 64 : 128;
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int64_t tiles = up(a.d_out, MM_BM) * up(a.n, bn);
  int cl = 1;
  int64_t best = -1;
  for (int c = 1; c <= 8 && c <= p.kblocks; c *= 2) {
    const int64_t waves = up(tiles * c, 2 * sms);
    const int block = tiles * c > sms ? (bn == 128 ? 440 : 300) : (bn == 128 ? 360 : 260);
    const int64_t cost = waves * (up(p.kblocks, c) * block + 2500) + (c > 1 ? 90 * bn / c : 0);
    if (best < 0 || cost < best) {
      best = cost;
      cl = c;
    }
  }
  const int64_t pair_cost =
      up(up(a.d_out, 256) * up(a.n, 256), sms / 2) * (static_cast<int64_t>(p.kblocks) * 370 + 2500);
  // under an SM budget only the pair kernel runs: it alone keeps to a number of SMs
  if (pair_cost < best || sm_budget() < sms || up(a.d_out, MM_BM) > 65535 || up(a.n, bn) > 65535)
    return launch_pair<Y>(a, p, stream);
  switch (bn) {
    case 16: return launch_split<16, Y>(a, p, cl, stream);
    case 32: return launch_split<32, Y>(a, p, cl, stream);
    case 64: return launch_split<64, Y>(a, p, cl, stream);
    default: return launch_split<128, Y>(a, p, cl, stream);
  }
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
  p.after_quant = a.after_quant;
  p.before_transform = a.before_transform;
  p.kblocks = (a.d_in + MM_BK - 1) / MM_BK;
  p.err = device_error_word();
  if (!p.err) return fail(KRONQ_ERR_CUDA, "device error word unavailable");
  return a.y_dtype == KRONQ_DTYPE_BF16 ? dispatch_mm<__nv_bfloat16>(a, p, stream)
                                       : dispatch_mm<float>(a, p, stream);
}

}  // namespace kq
