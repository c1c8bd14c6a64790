// Distillation from a teacher's top logits: loss per token and the gradient of the logits.
//
// For a token with student logits z (V entries), temperature tau, and the teacher's k listed
// entries (id_j, t_j):
//     p_j  = exp(t_j / tau - L_t),   L_t = logsumexp_j(t_j / tau)  or the caller's top_lse
//     loss = w tau^2 sum_j p_j (log p_j - z[id_j] / tau + lse),  lse = logsumexp_v(z_v / tau)
//     dz_v = w tau (P q_v - sum_{j: id_j = v} p_j),  P = sum_j p_j,  q_v = exp(z_v / tau - lse)
// z is streamed with a running maximum m and sum per thread: sum of 2^(z c - fl(m c)), with
// c = log2(e) / tau. The exponent is one FMA, rounded relative to the small difference; the
// rounding of m c is the same in a row's sum and in its q, where it cancels, and lse undoes it.
// Where m c overflows (a row that holds nothing but the type's lowest value) the exponent is
// (z - m) c instead.
// Per element and use of z: an unpack, half a packed fp32 FMA, one ex2, half a packed fp32 add or
// multiply. The two ex2 of loss + gradient (16 a cycle and SM) stay below the time of the bytes.
//
// A row is cut into cl slices of 16-byte vectors, one CTA each. Where the row's statistics are
// needed the CTAs of a row form a cluster and exchange (m, s) through distributed shared memory.
//   distill_hold_kernel     loss and gradient in one read: a thread keeps its vectors of z in
//                           registers between the statistics and the gradient
//   distill_stream_kernel   the loss alone, the gradient from a given lse, and loss + gradient of
//                           rows too long to hold (which are then read twice)
// Listed entries are few: their p, their part of the loss and their gradients are computed by
// one thread each, which fetches its id, logit and z[id] while the row streams; the gradient of
// a listed entry is stored over the streamed one after a barrier.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kq {
namespace {

constexpr int DS_THREADS = 256;
constexpr int DS_WARPS = DS_THREADS / 32;
constexpr int DS_KPT_MAX = kMaxDistillTop / DS_THREADS;   // listed entries per thread
constexpr int DS_MAX_CL = 8;                          // CTAs per row (portable cluster size)
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
  int64_t row0;            // the launch's first row
  int cl;                  // CTAs per row (the grid's x extent; y counts rows)
  int per;                 // vectors per CTA
  int hash_mask;           // entries of the id table in use - 1 (a power of two, >= 2 k)
  float tau;
  double inv_tau;
  float c;                 // log2(e) / tau
  double nat;              // inv_tau / c: from the exponents' unit to z / tau
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

// streaming accesses: each byte is used once by this kernel
__device__ __forceinline__ uint4 ds_ldg(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// ---- pairs of fp32 in one 64-bit register pair (packed arithmetic)
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- 16-byte vectors of z: VE elements as VE / 2 pairs
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int VE = 4;
  static constexpr uint32_t NONE = 0xff800000u;                 // -inf
  static __device__ __forceinline__ void get(const uint4& r, uint64_t (&x)[2]) {
    x[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
    x[1] = pack2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
  static __device__ __forceinline__ float max(const uint4& r) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                 fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int VE = 8;
  static constexpr uint32_t NONE = 0xff80ff80u;
  static __device__ __forceinline__ void get(const uint4& r, uint64_t (&x)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ float max(const uint4& r) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <typename T>
__device__ __forceinline__ uint4 none_vec() {                   // a vector of -inf: adds nothing
  return make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
}

// The part of a row that a CTA streams: vectors [i0, i1) of the row's aligned 16-byte vectors. The
// elements before the first and after the last vector (fewer than VE each) are part 0's, one
// per thread.
template <typename T>
struct Slice {
  const T* row;
  int v, head, nvec;
  int i0, i1;
  int edge;                // this thread's edge element, or -1
  __device__ __forceinline__ Slice(const T* r, int v_, int part, int per) : row(r), v(v_) {
    constexpr int VE = Vec<T>::VE;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    head = min(v, off ? VE - off : 0);
    nvec = (v - head) / VE;
    i0 = min(nvec, part * per);
    i1 = min(nvec, i0 + per);
    const int t = threadIdx.x, tail0 = head + nvec * VE;
    edge = -1;
    if (part == 0) {
      if (t < VE && t < head) edge = t;
      if (t >= VE && t < 2 * VE && tail0 + t - VE < v) edge = tail0 + t - VE;
    }
  }
  // entry e is streamed by this CTA
  __device__ __forceinline__ bool owns(int e, int part) const {
    if (e < head || e >= head + nvec * Vec<T>::VE) return part == 0;
    const int i = (e - head) / Vec<T>::VE;
    return i >= i0 && i < i1;
  }
  __device__ __forceinline__ uint4 load(int i) const {
    return ds_ldg(row + head + static_cast<int64_t>(i) * Vec<T>::VE);
  }
};

// Stores a vector's gradients at d: as 8- or 16-byte words where aligned, else one by one.
template <typename D, int VE>
__device__ __forceinline__ void store_vec(D* d, bool aligned, const uint64_t (&g)[VE / 2]) {
  if constexpr (sizeof(D) == 4) {
    if (aligned) {
#pragma unroll
      for (int e = 0; e < VE / 4; ++e) {
        const float2 a = unpack2(g[2 * e]), b = unpack2(g[2 * e + 1]);
        __stcs(reinterpret_cast<float4*>(d) + e, make_float4(a.x, a.y, b.x, b.y));
      }
      return;
    }
  } else if (aligned) {
    uint32_t w[VE / 2];
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
      const __nv_bfloat162 h = __float22bfloat162_rn(unpack2(g[e]));
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (VE == 8)
      __stcs(reinterpret_cast<uint4*>(d), make_uint4(w[0], w[1], w[2], w[3]));
    else
      __stcs(reinterpret_cast<uint2*>(d), make_uint2(w[0], w[1]));
    return;
  }
#pragma unroll
  for (int e = 0; e < VE / 2; ++e) {
    const float2 a = unpack2(g[e]);
    ds_st(d + 2 * e, a.x);
    ds_st(d + 2 * e + 1, a.y);
  }
}
template <typename T, typename D>
__device__ __forceinline__ bool store_aligned(const Slice<T>& s, const D* dz) {
  constexpr int bytes = Vec<T>::VE * sizeof(D) < 16 ? Vec<T>::VE * sizeof(D) : 16;
  return reinterpret_cast<uintptr_t>(dz + s.head) % bytes == 0;
}

// Running maximum and sum of 2^(z c - fl(m c)). m = -inf, s = 0: nothing but -inf seen.
struct RunSum {
  float m, s;
};
__device__ __forceinline__ bool ds_wide(float m, float c) { return !(fabsf(m * c) < INFINITY); }
// the exponent of one element
__device__ __forceinline__ float ds_exponent(float z, float m, float c) {
  return ds_wide(m, c) ? (z - m) * c : fmaf(z, c, -(m * c));
}
__device__ __forceinline__ float ds_rescale(float from, float to, float c) {
  return ex2(ds_wide(to, c) ? (from - to) * c : from * c - to * c);
}
// Joins groups of W consecutive lanes that hold the same W values in every group (W = 32: the
// warp): the common maximum first, so that each lane rescales its sum once.
template <int W>
__device__ __forceinline__ RunSum ds_join_lanes(RunSum r, float c) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(r.m));
  float s = r.m == m ? r.s : r.s * ds_rescale(r.m, m, c);
#pragma unroll
  for (int o = W / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return {m, s};
}
// acc += the terms of one vector against a maximum that covers it
template <typename T>
__device__ __forceinline__ uint64_t ds_terms(uint64_t acc, const uint4& raw, bool wide, float m,
                                             float c) {
  constexpr int NP = Vec<T>::VE / 2;
  uint64_t x[NP];
  Vec<T>::get(raw, x);
  if (wide) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 z = unpack2(x[e]);
      acc = add2(acc, pack2(ex2((z.x - m) * c), ex2((z.y - m) * c)));
    }
  } else {
    const uint64_t cc = pack2(c, c), ref = pack2(-(m * c), -(m * c));
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 d = unpack2(fma2(x[e], cc, ref));
      acc = add2(acc, pack2(ex2(d.x), ex2(d.y)));
    }
  }
  return acc;
}

__device__ __forceinline__ void ds_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void ds_cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ds_remote(const void* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

struct DsShared {
  RunSum row[DS_WARPS];          // statistics per warp
  RunSum list[DS_WARPS];         // and of the listed logits
  RunSum mine;                   // this CTA's statistics, read by the cluster
  double loss[DS_WARPS];
  float mass[DS_WARPS];
};

// With a gradient, in dynamic shared memory: the list, for repeated ids, and a table from an id to
// the first j that lists it and how many do.
struct IdTable {
  float* p;                      // k
  int* id;                       // k
  int* key;                      // hash_mask + 1 each
  int* first;
  int* count;
  __device__ __forceinline__ explicit IdTable(const DsArgs& a) {
    extern __shared__ int ds_table[];
    key = ds_table;
    first = key + a.hash_mask + 1;
    count = first + a.hash_mask + 1;
    id = count + a.hash_mask + 1;
    p = reinterpret_cast<float*>(id + a.k);
  }
};
size_t id_table_bytes(const DsArgs& a) {
  return (3 * (static_cast<size_t>(a.hash_mask) + 1) + 2 * static_cast<size_t>(a.k)) * 4;
}

// The listed entries of a row: thread t has entries t, t + 256, ... (KPT of them)
template <int KPT>
struct Entries {
  int id[KPT];                   // -1: absent
  float t[KPT], z[KPT], p[KPT];
};

__device__ __forceinline__ uint32_t ds_slot(const DsArgs& a, int id) {
  return (static_cast<uint32_t>(id) * 2654435761u >> 16) & a.hash_mask;
}

// z[id] is read where it is used: for the loss (all entries), and for the gradients of the entries
// in the CTA's own slice (other slices may already be overwritten when dz is z).
template <typename T, int KPT>
__device__ __forceinline__ void load_entries(const DsArgs& a, int64_t row, const Slice<T>& s,
                                             int part, bool all, Entries<KPT>& e) {
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int j = threadIdx.x + i * DS_THREADS;
    e.id[i] = -1;
    e.t[i] = kNegInf;
    e.z[i] = 0.f;
    if (j < a.k) {
      const int id = a.ids[row * a.ld_ids + j];
      if (id >= 0 && id < a.v) {
        const int64_t o = row * a.ld_top + j;
        e.id[i] = id;
        e.t[i] = a.top_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.top)[o])
                            : static_cast<const float*>(a.top)[o];
        if (all || s.owns(id, part)) e.z[i] = ds_ld(s.row + id);
      }
    }
  }
}

// -inf where nothing was seen
__device__ __forceinline__ double ds_lse(const DsArgs& a, RunSum r) {
  return (ds_wide(r.m, a.c) ? r.m * a.inv_tau : r.m * a.c * a.nat) + logf(r.s);
}

// Joins the CTA's (and, with a cluster, the row's) statistics and the listed entries'; gives p and,
// in the CTA that reports the row, the loss. GRAD: fills the id table.
template <bool LSE, bool GRAD, int KPT>
__device__ __forceinline__ void row_statistics(const DsArgs& a, int64_t row, int part, float w,
                                               DsShared& sh, RunSum& rs, Entries<KPT>& e,
                                               float& mass) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lists = warp * 32 < a.k;            // some thread of the warp has an entry
  if (LSE) {
    rs = ds_join_lanes<32>(rs, a.c);
    if (lane == 0) sh.row[warp] = rs;
  }
  RunSum ls{kNegInf, 0.f};
  if (lists) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) ls.m = fmaxf(ls.m, e.t[i]);
#pragma unroll
    for (int i = 0; i < KPT; ++i)                // a NaN logit makes s NaN
      if (e.t[i] != kNegInf) ls.s += ex2(ds_exponent(e.t[i], ls.m == kNegInf ? 0.f : ls.m, a.c));
    ls = ds_join_lanes<32>(ls, a.c);
  }
  if (lane == 0) sh.list[warp] = ls;
  __syncthreads();
  if (LSE) {
    rs = ds_join_lanes<DS_WARPS>(sh.row[lane % DS_WARPS], a.c);
    if (a.cl > 1) {
      if (tid == 0) sh.mine = rs;
      ds_cluster_arrive();
      ds_cluster_wait();
      const int r = lane % DS_MAX_CL;
      rs = {kNegInf, 0.f};
      if (r < a.cl) rs = {ds_remote(&sh.mine.m, r), ds_remote(&sh.mine.s, r)};
      rs = ds_join_lanes<DS_MAX_CL>(rs, a.c);
      ds_cluster_arrive();                         // waited for before the CTA ends
    }
  }
  double part_loss = 0.0;
  const bool report = LSE && part == 0;
  const double lse = report ? ds_lse(a, rs) : 0.0;
  mass = 0.f;
#pragma unroll
  for (int i = 0; i < KPT; ++i) e.p[i] = 0.f;
  if (lists) {
    // log p_j = t_j / tau - L_t in fp64: the difference of two numbers of the logits' size
    ls = ds_join_lanes<DS_WARPS>(sh.list[lane % DS_WARPS], a.c);
    const double norm = a.top_lse ? static_cast<double>(a.top_lse[row]) : ds_lse(a, ls);
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = tid + i * DS_THREADS;
      if (j >= a.k) break;
      if (e.t[i] != kNegInf) {
        const double lp = e.t[i] * a.inv_tau - norm;
        const float p = expf(static_cast<float>(lp));
        e.p[i] = p;
        mass += p;
        // a listed entry that the student masks has an infinite loss
        if (report && p != 0.f)
          part_loss += e.z[i] == kNegInf ? static_cast<double>(INFINITY)
                                         : p * (lp - e.z[i] * a.inv_tau + lse);
      }
      if (GRAD) {
        const IdTable table(a);
        table.p[j] = e.p[i];
        table.id[j] = e.id[i];
        if (e.id[i] >= 0) {
          uint32_t h = ds_slot(a, e.id[i]);
          while (true) {                           // at most k of >= 2 k slots are taken
            const int old = atomicCAS(&table.key[h], -1, e.id[i]);
            if (old == -1 || old == e.id[i]) break;
            h = (h + 1) & a.hash_mask;
          }
          atomicMin(&table.first[h], j);
          atomicAdd(&table.count[h], 1);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    if (report) {
#pragma unroll
      for (int o = 16; o; o >>= 1) part_loss += __shfl_xor_sync(0xffffffffu, part_loss, o);
    }
  }
  if (lane == 0) {
    sh.mass[warp] = mass;
    if (report) sh.loss[warp] = part_loss;
  }
  __syncthreads();
  mass = 0.f;
#pragma unroll
  for (int i = 0; i < DS_WARPS; ++i) mass += sh.mass[i];
  if (report && tid == 0) {
    double tot = 0.0;
    for (int i = 0; i < DS_WARPS; ++i) tot += sh.loss[i];
    a.loss[row] = w == 0.f ? 0.f : static_cast<float>(static_cast<double>(w) * a.tau * a.tau * tot);
    if (a.lse) a.lse[row] = static_cast<float>(lse);
  }
}

__device__ __forceinline__ void clear_table(const DsArgs& a) {
  const IdTable table(a);
  for (int i = threadIdx.x; i <= a.hash_mask; i += DS_THREADS) {
    table.key[i] = -1;
    table.first[i] = kMaxDistillTop;
    table.count[i] = 0;
  }
}

// Gradients of the listed entries in this CTA's slice: the first thread that lists an id adds up
// all its p, in the order of the list. patch_id = -1: not this thread's to store.
template <typename T, int KPT>
__device__ __forceinline__ void list_gradients(const DsArgs& a, const Slice<T>& s,
                                               const Entries<KPT>& e, RunSum rs, float coef,
                                               float wt, int part, float (&patch)[KPT],
                                               int (&patch_id)[KPT]) {
  const IdTable table(a);
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int j = threadIdx.x + i * DS_THREADS;
    patch_id[i] = -1;
    patch[i] = 0.f;
    if (j < a.k && e.id[i] >= 0 && s.owns(e.id[i], part)) {
      uint32_t h = ds_slot(a, e.id[i]);
      while (table.key[h] != e.id[i]) h = (h + 1) & a.hash_mask;
      if (table.first[h] == j) {
        float p = e.p[i];
        if (table.count[h] > 1)
          for (int l = j + 1; l < a.k; ++l)
            if (table.id[l] == e.id[i]) p += table.p[l];
        patch_id[i] = e.id[i];
        if (wt != 0.f)
          patch[i] = coef == 0.f ? -wt * p : fmaf(coef, ex2(ds_exponent(e.z[i], rs.m, a.c)), -wt * p);
      }
    }
  }
}

template <typename T, typename D>
__device__ __forceinline__ void put_gradients(D* d, bool aligned, const uint4& raw, bool wide,
                                              float m, float c, float coef) {
  constexpr int NP = Vec<T>::VE / 2;
  uint64_t x[NP], g[NP];
  Vec<T>::get(raw, x);
  if (coef == 0.f) {                                   // whatever z holds
#pragma unroll
    for (int e = 0; e < NP; ++e) g[e] = 0;
  } else if (wide) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 z = unpack2(x[e]);
      g[e] = pack2(coef * ex2((z.x - m) * c), coef * ex2((z.y - m) * c));
    }
  } else {
    const uint64_t cc = pack2(c, c), ref = pack2(-(m * c), -(m * c)), k = pack2(coef, coef);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 t = unpack2(fma2(x[e], cc, ref));
      g[e] = mul2(k, pack2(ex2(t.x), ex2(t.y)));
    }
  }
  store_vec<D, Vec<T>::VE>(d, aligned, g);
}
template <typename T, typename D>
__device__ __forceinline__ void put_edge(const Slice<T>& s, D* dz, float z, float m, float c,
                                         float coef) {
  if (s.edge >= 0) ds_st(dz + s.edge, coef == 0.f ? 0.f : coef * ex2(ds_exponent(z, m, c)));
}

// w tau P / s: no gradient where the weight or the teacher's list is empty, none by q where z
// holds nothing but -inf
__device__ __forceinline__ float ds_coef(float wt, float mass, float s) {
  return (wt == 0.f || mass == 0.f || s == 0.f) ? 0.f : wt * mass / s;
}

// Loss and gradient; NV vectors of z per thread stay in registers.
template <typename T, typename D, int NV, int KPT>
__global__ void __launch_bounds__(DS_THREADS, NV > 8 ? 2 : (KPT == 1 ? 4 : 3)) distill_hold_kernel(DsArgs a) {
  __shared__ DsShared sh;
  const int64_t row = a.row0 + blockIdx.y;
  const int part = blockIdx.x;
  const int tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  const Slice<T> s(z, a.v, part, a.per);
  uint4 raw[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int i = s.i0 + tid + n * DS_THREADS;
    raw[n] = i < s.i1 ? s.load(i) : none_vec<T>();
  }
  const float ze = s.edge >= 0 ? ds_ld(z + s.edge) : kNegInf;
  Entries<KPT> e;
  load_entries(a, row, s, part, part == 0, e);
  clear_table(a);
  const float w = a.weight ? a.weight[row] : 1.f;
  RunSum rs{ze, 0.f};
#pragma unroll
  for (int n = 0; n < NV; ++n) rs.m = fmaxf(rs.m, Vec<T>::max(raw[n]));
  // a thread whose entries are all -inf adds nothing, to any reference (NaN it adds)
  const float m = rs.m == kNegInf ? 0.f : rs.m;
  const bool mwide = ds_wide(m, a.c);
  uint64_t acc = pack2(ex2(ds_exponent(ze, m, a.c)), 0.f);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    acc = ds_terms<T>(acc, raw[n], mwide, m, a.c);
    asm volatile("" : "+l"(acc));                      // one vector unpacked at a time
  }
  rs.s = unpack2(acc).x + unpack2(acc).y;
  // the gradient unpacks the vectors again: nothing unpacked lives across the statistics
#pragma unroll
  for (int n = 0; n < NV; ++n)
    asm volatile("" : "+r"(raw[n].x), "+r"(raw[n].y), "+r"(raw[n].z), "+r"(raw[n].w));
  float mass;
  row_statistics<true, true, KPT>(a, row, part, w, sh, rs, e, mass);
  const float wt = w * a.tau;
  const float coef = ds_coef(wt, mass, rs.s);
  float patch[KPT];
  int patch_id[KPT];
  list_gradients(a, s, e, rs, coef, wt, part, patch, patch_id);
  D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
  const bool al = store_aligned(s, dz), wide = ds_wide(rs.m, a.c);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int i = s.i0 + tid + n * DS_THREADS;
    if (i < s.i1)
      put_gradients<T, D>(dz + s.head + static_cast<int64_t>(i) * Vec<T>::VE, al, raw[n], wide,
                          rs.m, a.c, coef);
  }
  put_edge(s, dz, ze, rs.m, a.c, coef);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < KPT; ++i)
    if (patch_id[i] >= 0) ds_st(dz + patch_id[i], patch[i]);
  if (a.cl > 1) ds_cluster_wait();
}

// LSE: the row's statistics are taken from z (else lse_in). GRAD: dz is written.
template <typename T, typename D, bool LSE, bool GRAD, int KPT>
__global__ void __launch_bounds__(DS_THREADS) distill_stream_kernel(DsArgs a) {
  __shared__ DsShared sh;
  const int64_t row = a.row0 + blockIdx.y;
  const int part = blockIdx.x;
  const int tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  const Slice<T> s(z, a.v, part, a.per);
  Entries<KPT> e;
  load_entries(a, row, s, part, LSE && part == 0, e);
  if (GRAD) clear_table(a);
  const float w = a.weight ? a.weight[row] : 1.f;
  constexpr int U = 4;                               // vectors in flight per thread
  const float ze = s.edge >= 0 ? ds_ld(z + s.edge) : kNegInf;
  RunSum rs{kNegInf, 0.f};
  if (LSE) {
    rs = {ze, ze == kNegInf ? 0.f : ex2(ds_exponent(ze, ze, a.c))};       // 1, or NaN
    for (int i = s.i0 + tid; i < s.i1; i += U * DS_THREADS) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = i + u * DS_THREADS < s.i1 ? s.load(i + u * DS_THREADS) : none_vec<T>();
      float m = rs.m;
#pragma unroll
      for (int u = 0; u < U; ++u) m = fmaxf(m, Vec<T>::max(raw[u]));
      if (m > rs.m) {
        rs.s *= ds_rescale(rs.m, m, a.c);
        rs.m = m;
      }
      if (!(m > kNegInf)) m = 0.f;                   // nothing but -inf (or NaN) so far
      const bool mwide = ds_wide(m, a.c);
      uint64_t acc = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) acc = ds_terms<T>(acc, raw[u], mwide, m, a.c);
      rs.s += unpack2(acc).x + unpack2(acc).y;
    }
  } else {
    // q = 2^(z c - fl(m c)) / s with m = lse tau rounded to fp32, s = what the roundings left
    // (z tau^-1 - lse at z = lse tau, where q is not small)
    const float l = a.lse_in[row];
    rs.m = l * a.tau;
    const double left = ds_wide(rs.m, a.c) ? l - rs.m * a.inv_tau
                                           : (static_cast<double>(l) * a.tau * a.c -
                                              static_cast<double>(rs.m * a.c)) * 0.69314718055994531;
    rs.s = l == kNegInf ? 0.f : expf(static_cast<float>(left));
  }
  float mass;
  row_statistics<LSE, GRAD, KPT>(a, row, part, w, sh, rs, e, mass);
  if (GRAD) {
    const float wt = w * a.tau;
    const float coef = ds_coef(wt, mass, rs.s);
    float patch[KPT];
    int patch_id[KPT];
    list_gradients(a, s, e, rs, coef, wt, part, patch, patch_id);
    D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
    const bool al = store_aligned(s, dz), wide = ds_wide(rs.m, a.c);
    // dz may be z: every entry's z[id] was read before the first barrier above
    for (int i = s.i0 + tid; i < s.i1; i += U * DS_THREADS) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * DS_THREADS < s.i1) raw[u] = s.load(i + u * DS_THREADS);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * DS_THREADS < s.i1)
          put_gradients<T, D>(dz + s.head + static_cast<int64_t>(i + u * DS_THREADS) * Vec<T>::VE,
                              al, raw[u], wide, rs.m, a.c, coef);
    }
    put_edge(s, dz, ze, rs.m, a.c, coef);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (patch_id[i] >= 0) ds_st(dz + patch_id[i], patch[i]);
  }
  if (LSE && a.cl > 1) ds_cluster_wait();
}

kronq_status launch_rows(void (*kern)(DsArgs), DsArgs a, int n, bool cluster, bool table,
                         const char* what, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(DS_THREADS);
  cfg.dynamicSmemBytes = table ? id_table_bytes(a) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.cl);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster && a.cl > 1 ? 1 : 0;
  constexpr int most = 65535;                      // rows per launch: the grid's y extent
  for (a.row0 = 0; a.row0 < n; a.row0 += most) {
    cfg.gridDim = dim3(a.cl, static_cast<unsigned>(std::min<int64_t>(most, n - a.row0)));
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return fail(KRONQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
    KQ_TRY(check_launch(what));
  }
  return KRONQ_OK;
}

template <typename T, typename D, int KPT>
kronq_status launch_distill(DsArgs a, int n, bool lse, bool grad, cudaStream_t stream) {
  constexpr int NV = 8;
  const int64_t vecs = static_cast<int64_t>(a.v) / Vec<T>::VE + 1;    // at most, and at least one
  if (!lse) {
    // the gradient alone has no statistics to exchange: any number of slices, here of four
    // vectors per thread
    a.per = 4 * DS_THREADS;
    a.cl = static_cast<int>((vecs + a.per - 1) / a.per);
    return launch_rows(distill_stream_kernel<T, D, false, true, KPT>, a, n, false, true,
                       "distill_stream_kernel", stream);
  }
  // Slices: enough to give every SM two CTAs when rows are few, none shorter than one vector per
  // thread.
  a.cl = 1;
  while (a.cl < DS_MAX_CL && static_cast<int64_t>(n) * a.cl < 2 * device_sms() &&
         vecs > static_cast<int64_t>(a.cl) * DS_THREADS)
    a.cl *= 2;
  auto cut = [&] { return static_cast<int>((vecs + a.cl - 1) / a.cl); };
  a.per = cut();
  if (!grad)
    return launch_rows(distill_stream_kernel<T, D, true, false, KPT>, a, n, true, false,
                       "distill_stream_kernel", stream);
  while (a.cl < DS_MAX_CL && vecs > static_cast<int64_t>(a.cl) * DS_THREADS * NV) a.cl *= 2;
  a.per = cut();
  auto kern = a.per <= DS_THREADS * NV       ? distill_hold_kernel<T, D, NV, KPT>
              : a.per <= DS_THREADS * 2 * NV ? distill_hold_kernel<T, D, 2 * NV, KPT>
                                           : distill_stream_kernel<T, D, true, true, KPT>;
  return launch_rows(kern, a, n, true, true, "distill kernel", stream);
}

template <typename T, typename D>
kronq_status launch_distill(const DsArgs& a, int n, bool lse, bool grad, cudaStream_t stream) {
  return a.k <= DS_THREADS ? launch_distill<T, D, 1>(a, n, lse, grad, stream)
                           : launch_distill<T, D, DS_KPT_MAX>(a, n, lse, grad, stream);
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
  a.hash_mask = 31;
  while (a.hash_mask + 1 < 2 * a.k) a.hash_mask = 2 * a.hash_mask + 1;
  a.tau = q.temperature;
  a.inv_tau = 1.0 / static_cast<double>(q.temperature);
  a.c = static_cast<float>(1.4426950408889634 * a.inv_tau);
  a.nat = a.inv_tau / a.c;
  const bool lse = q.lse_in == nullptr, grad = q.dlogits != nullptr;
  const bool zb = q.logits_dtype == KRONQ_DTYPE_BF16, db = q.dlogits_dtype == KRONQ_DTYPE_BF16;
  if (zb) return db || !grad ? launch_distill<__nv_bfloat16, __nv_bfloat16>(a, q.n, lse, grad, stream)
                             : launch_distill<__nv_bfloat16, float>(a, q.n, lse, grad, stream);
  return db ? launch_distill<float, __nv_bfloat16>(a, q.n, lse, grad, stream)
            : launch_distill<float, float>(a, q.n, lse, grad, stream);
}

}  // namespace kq
