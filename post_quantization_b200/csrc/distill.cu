// Distillation from a teacher's top logits: loss per token and the gradient of the logits.
//
// For a token with student logits z (V entries), temperature tau, and the teacher's k listed
// entries (id_j, t_j):
//     p_j  = exp(t_j / tau - L_t),   L_t = logsumexp_j(t_j / tau)  or the caller's top_lse
//     loss = w tau^2 sum_j p_j (log p_j - z[id_j] / tau + lse),  lse = logsumexp_v(z_v / tau)
//     dz_v = w tau (P q_v - sum_{j: id_j = v} p_j),  P = sum_j p_j,  q_v = exp(z_v / tau - lse)
// z is streamed with a running maximum and sum per thread: sum of 2^((z - m) c), c = log2(e) / tau.
// The difference is taken before the scaling: it is exact or rounds relative to itself, nothing
// overflows (a mask of the type's lowest value included), and the rounding of c moves an exponent
// by 2^-24 of the difference only.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int DS_THREADS = 512;
constexpr int DS_MAX_K = 1024;
constexpr int DS_HASH = 2048;
constexpr float kNegInf = -INFINITY;

struct DsArgs {
  const void* z;
  int64_t ld_z;
  const int32_t* ids;
  int64_t ld_ids;
  const void* top;
  int64_t ld_top;
  int top_bf16;
  const float* top_lse;    // NULL: the listed entries are normalised among themselves
  const float* weight;     // NULL: 1
  const float* lse_in;     // backward
  float* loss;
  float* lse;              // NULL: not written
  void* dz;
  int64_t ld_dz;
  int v, k;
  float tau;
  double inv_tau;
  float c;                 // log2(e) / tau
};

__device__ __forceinline__ float ds_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ds_ld(const float* p) { return *p; }
__device__ __forceinline__ void ds_st(float* p, float v) { *p = v; }
__device__ __forceinline__ void ds_st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Running maximum and sum of 2^((z - m) c). m = -inf, s = 0: nothing but -inf seen.
struct RunSum {
  float m, s;
};
__device__ __forceinline__ RunSum ds_join(RunSum a, RunSum b, float c) {
  if (b.m == kNegInf && b.s == 0.f) return a;
  if (a.m == kNegInf && a.s == 0.f) return b;
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * ex2((a.m - m) * c) + b.s * ex2((b.m - m) * c)};
}

// The teacher's side of one row, in shared memory.
struct Teacher {
  int id[DS_MAX_K];        // entry, or -1 where absent
  float p[DS_MAX_K];
  float logp[DS_MAX_K];
  int key[DS_HASH];        // backward: id -> first j that lists it
  int first[DS_HASH];
  float mass;
  int repeated;            // some id is listed twice
};

// p, log p and P of the row by warp 0. Entries whose id is outside 0 .. v - 1 are absent; their
// logits are not looked at.
__device__ __forceinline__ void ds_teacher(const DsArgs& a, int64_t row, Teacher& te) {
  const int lane = threadIdx.x;
  auto logit = [&](int j) {
    const int64_t o = row * a.ld_top + j;
    return a.top_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.top)[o])
                      : static_cast<const float*>(a.top)[o];
  };
  const float it = static_cast<float>(a.inv_tau);
  float m = kNegInf;
  for (int j = lane; j < a.k; j += 32) {
    const int id = a.ids[row * a.ld_ids + j];
    const bool there = id >= 0 && id < a.v;
    te.id[j] = there ? id : -1;
    if (there) m = fmaxf(m, logit(j));
  }
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == kNegInf) m = 0.f;                   // only -inf logits: every p below is 0
  float s = 0.f;
  for (int j = lane; j < a.k; j += 32)
    if (te.id[j] >= 0) s += expf((logit(j) - m) * it);
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  // log p_j = t_j / tau - norm, in fp64: the difference of two numbers of the logits' size
  const double norm = a.top_lse ? static_cast<double>(a.top_lse[row])
                                : m * a.inv_tau + (s == 0.f ? 0.f : logf(s));
  float mass = 0.f;
  for (int j = lane; j < a.k; j += 32) {
    const float lp =
        te.id[j] >= 0 ? static_cast<float>(logit(j) * a.inv_tau - norm) : kNegInf;
    te.logp[j] = lp;
    te.p[j] = expf(lp);
    mass += te.p[j];
  }
  for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  if (lane == 0) te.mass = mass;
}

// Which j is the first to list its id (open addressing; called by the whole CTA).
__device__ __forceinline__ void ds_hash(const DsArgs& a, Teacher& te) {
  for (int i = threadIdx.x; i < DS_HASH; i += blockDim.x) {
    te.key[i] = -1;
    te.first[i] = DS_MAX_K;
  }
  if (threadIdx.x == 0) te.repeated = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
    const int id = te.id[j];
    if (id < 0) continue;
    uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 21;     // 11 bits
    while (true) {
      const int old = atomicCAS(&te.key[h], -1, id);
      if (old == -1 || old == id) break;
      h = (h + 1) & (DS_HASH - 1);
    }
    atomicMin(&te.first[h], j);
  }
  __syncthreads();
}
__device__ __forceinline__ int ds_first(const Teacher& te, int id) {
  uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 21;
  while (te.key[h] != id) h = (h + 1) & (DS_HASH - 1);
  return te.first[h];
}

// One CTA per row. LSE: the row's log-sum-exp is computed (else lse_in); GRAD: dz is written.
template <typename T, typename D, bool LSE, bool GRAD>
__global__ void __launch_bounds__(DS_THREADS) distill_kernel(DsArgs a) {
  __shared__ Teacher te;
  __shared__ RunSum red[DS_THREADS / 32];
  __shared__ double red_loss[DS_THREADS / 32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  const float w = a.weight ? a.weight[row] : 1.f;
  if (warp == 0) ds_teacher(a, row, te);
  RunSum rs{kNegInf, 0.f};
  if (LSE) {
    for (int v = tid; v < a.v; v += DS_THREADS) {
      const float x = ds_ld(z + v);
      if (x > rs.m) {
        rs.s *= ex2((rs.m - x) * a.c);
        rs.m = x;
      }
      if (x != kNegInf) rs.s += ex2((x - rs.m) * a.c);
    }
    for (int o = 16; o; o >>= 1)
      rs = ds_join(rs, {__shfl_xor_sync(0xffffffffu, rs.m, o),
                        __shfl_xor_sync(0xffffffffu, rs.s, o)}, a.c);
    if (lane == 0) red[warp] = rs;
  }
  __syncthreads();
  if (LSE) {
    rs = red[0];
    for (int i = 1; i < DS_THREADS / 32; ++i) rs = ds_join(rs, red[i], a.c);
    const double lse = rs.m * a.inv_tau + logf(rs.s);      // -inf where nothing was seen
    double part = 0.0;
    for (int j = tid; j < a.k; j += DS_THREADS) {
      const float p = te.p[j];
      if (p != 0.f) {
        const float x = ds_ld(z + te.id[j]);
        // a listed entry that the student masks has an infinite loss
        part += x == kNegInf ? static_cast<double>(INFINITY)
                             : p * (te.logp[j] - x * a.inv_tau + lse);
      }
    }
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) red_loss[warp] = part;
    __syncthreads();
    if (tid == 0) {
      double tot = 0.0;
      for (int i = 0; i < DS_THREADS / 32; ++i) tot += red_loss[i];
      a.loss[row] = w == 0.f ? 0.f
                             : static_cast<float>(static_cast<double>(w) * a.tau * a.tau * tot);
      if (a.lse) a.lse[row] = static_cast<float>(lse);
    }
  } else {
    // q = 2^((z - m) c) / s with m = lse tau rounded to fp32, s = what the rounding left
    const float l = a.lse_in[row];
    rs.m = l * a.tau;
    rs.s = l == kNegInf ? 0.f : expf(static_cast<float>(l - rs.m * a.inv_tau));
  }
  if (!GRAD) return;
  D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
  const float wt = w * a.tau;
  const float mass = te.mass;
  // no gradient where the weight or the teacher's list is empty, none by q where z is all -inf
  const float coef = (wt == 0.f || mass == 0.f || rs.s == 0.f) ? 0.f : wt * mass / rs.s;
  ds_hash(a, te);
  // the listed entries' gradients, read before the row is written (dz may be z)
  float patch[DS_MAX_K / DS_THREADS];
  int patch_id[DS_MAX_K / DS_THREADS];
#pragma unroll
  for (int i = 0; i < DS_MAX_K / DS_THREADS; ++i) {
    const int j = tid + i * DS_THREADS;
    patch_id[i] = -1;
    if (j < a.k && te.id[j] >= 0 && ds_first(te, te.id[j]) == j) {
      const int id = te.id[j];
      float p = 0.f;
      for (int l = j; l < a.k; ++l)
        if (te.id[l] == id) p += te.p[l];
      patch_id[i] = id;
      patch[i] = coef == 0.f ? -wt * p
                             : fmaf(coef, ex2((ds_ld(z + id) - rs.m) * a.c), -wt * p);
      if (wt == 0.f) patch[i] = 0.f;
    }
  }
  __syncthreads();
  for (int v = tid; v < a.v; v += DS_THREADS)
    ds_st(dz + v, coef == 0.f ? 0.f : coef * ex2((ds_ld(z + v) - rs.m) * a.c));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < DS_MAX_K / DS_THREADS; ++i)
    if (patch_id[i] >= 0) ds_st(dz + patch_id[i], patch[i]);
}

template <typename T, typename D>
kronq_status launch_distill(const DsArgs& a, int n, bool lse, bool grad, cudaStream_t stream) {
  auto kern = lse ? (grad ? distill_kernel<T, D, true, true> : distill_kernel<T, D, true, false>)
                  : distill_kernel<T, D, false, true>;
  kern<<<n, DS_THREADS, 0, stream>>>(a);
  return check_launch("distill_kernel");
}

}  // namespace

kronq_status run_distill(const DistillArgs& q, cudaStream_t stream) {
  DsArgs a{};
  a.z = q.logits;
  a.ld_z = q.ld_logits;
  a.ids = q.ids;
  a.ld_ids = q.ld_ids;
  a.top = q.top;
  a.ld_top = q.ld_top;
  a.top_bf16 = q.top_dtype == KRONQ_DTYPE_BF16;
  a.top_lse = q.top_lse;
  a.weight = q.row_weight;
  a.lse_in = q.lse_in;
  a.loss = q.loss;
  a.lse = q.lse;
  a.dz = q.dlogits;
  a.ld_dz = q.ld_dlogits;
  a.v = q.v;
  a.k = q.k;
  a.tau = q.temperature;
  a.inv_tau = 1.0 / static_cast<double>(q.temperature);
  a.c = static_cast<float>(1.4426950408889634 * a.inv_tau);
  const bool lse = q.lse_in == nullptr, grad = q.dlogits != nullptr;
  const bool zb = q.logits_dtype == KRONQ_DTYPE_BF16, db = q.dlogits_dtype == KRONQ_DTYPE_BF16;
  if (zb) return db || !grad ? launch_distill<__nv_bfloat16, __nv_bfloat16>(a, q.n, lse, grad, stream)
                             : launch_distill<__nv_bfloat16, float>(a, q.n, lse, grad, stream);
  return db ? launch_distill<float, __nv_bfloat16>(a, q.n, lse, grad, stream)
            : launch_distill<float, float>(a, q.n, lse, grad, stream);
}

}  // namespace kq
