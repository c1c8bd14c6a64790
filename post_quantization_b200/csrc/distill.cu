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
// Where |m c| is 2^20 or more (a row that holds nothing but a mask's large value, say) the exponent
// is (z - m) c instead: there the rounding of m c could leave the range of 2^x.
// Per element: an unpack, half a packed fp32 FMA, one ex2 (16 a cycle and SM), half a packed add.
//
// A row is cut into cl slices of 16-byte vectors, one CTA each. Where the row's statistics are
// needed the CTAs of a row form a cluster and exchange (m, s) through distributed shared memory.
//   distill_ring_kernel     loss and gradient of long rows in one read. Persistent clusters, two
//                           CTAs per SM so that one's barriers hide behind the other's work. A
//                           producer warp fetches chunks of the CTA's slices, row after row, into
//                           a ring in shared memory (bulk copies); eight warps take the statistics
//                           as chunks arrive, keep the row there, and free each chunk as its
//                           gradient is written, so that the next row's reads go on; two list warps
//                           do all that concerns the teacher's entries, for rows in turn
//   distill_hold_kernel     loss and gradient of short rows, or of few: a thread keeps its vectors
//                           of z in registers between the statistics and the gradient
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
constexpr int DS_RING_THREADS = DS_THREADS + 96;      // ring kernel: a producer and two list warps
constexpr int DS_MAX_CL = 8;                          // CTAs per row (portable cluster size)
constexpr int DS_CHUNK_VECS = 4 * DS_THREADS;         // vectors per ring chunk (16 KB)
constexpr int DS_MAX_CHUNKS = 13;                     // chunks in the ring
constexpr int DS_RING_MIN_VECS = 2048;                // rows below 32 KB do not use the ring
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
  __device__ __forceinline__ const T* at(int i) const {
    return row + head + static_cast<int64_t>(i) * Vec<T>::VE;
  }
  __device__ __forceinline__ uint4 load(int i) const { return ds_ldg(at(i)); }
};

// Bulk copy global -> shared, completion on `bar` (no multicast); 16-byte addresses and size.
__device__ __forceinline__ void ds_bulk_load(void* dst, const void* src, uint32_t bytes,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

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
struct __align__(8) RunSum {      // sent as one 8-byte word
  float m, s;
};
__device__ __forceinline__ bool ds_wide(float m, float c) { return !(fabsf(m * c) < 1048576.f); }
// the exponent of one element
__device__ __forceinline__ float ds_exponent(float z, float m, float c) {
  return ds_wide(m, c) ? (z - m) * c : fmaf(z, c, -(m * c));
}
// From a sum's reference to another. Narrow references are rounded products, as in ds_exponent: a
// contraction into one FMA would leave that of `from` exact, and the sums off by its rounding (at
// tau = 2^-8 by 1e-3). Of a narrow and a wide one the wide one's product is exact.
__device__ __forceinline__ float ds_rescale(float from, float to, float c) {
  const bool wide_from = ds_wide(from, c), wide_to = ds_wide(to, c);
  const float f = __fmul_rn(from, c), t = __fmul_rn(to, c);
  if (wide_from != wide_to) return ex2(wide_to ? -fmaf(to, c, -f) : fmaf(from, c, -t));
  return ex2(wide_to ? (from - to) * c : __fsub_rn(f, t));
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
// The sum of the terms of U vectors against a reference m. One branch for all of them: the
// exponentials of different vectors overlap only within one straight run of code.
template <typename T, int U>
__device__ __forceinline__ float ds_terms(const uint4 (&raw)[U], bool wide, float m, float c) {
  constexpr int NP = Vec<T>::VE / 2;
  uint64_t acc[2] = {0, 0};                          // two chains of packed sums
  if (wide) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t x[NP];
      Vec<T>::get(raw[u], x);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float2 z = unpack2(x[e]);
        acc[0] = add2(acc[0], pack2(ex2((z.x - m) * c), ex2((z.y - m) * c)));
      }
    }
  } else {
    const uint64_t cc = pack2(c, c), ref = pack2(-(m * c), -(m * c));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t x[NP];
      Vec<T>::get(raw[u], x);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float2 d = unpack2(fma2(x[e], cc, ref));
        acc[e & 1] = add2(acc[e & 1], pack2(ex2(d.x), ex2(d.y)));
      }
    }
  }
  const float2 s = unpack2(add2(acc[0], acc[1]));
  return s.x + s.y;
}

__device__ __forceinline__ void ds_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void ds_cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Eight bytes into a peer's shared memory, counted on a barrier there.
__device__ __forceinline__ void ds_send(const RunSum* dst, const uint64_t* bar, uint32_t rank,
                                        RunSum v) {
  uint32_t a, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(dst)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(a),
      "l"(pack2(v.m, v.s)), "r"(b)
      : "memory");
}
__device__ __forceinline__ float ds_remote(const void* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

struct DsShared {
  RunSum row[DS_WARPS];      // statistics per warp
  RunSum list[DS_WARPS];     // and of the listed logits
  RunSum mine;                   // this CTA's statistics, read by the cluster
  double loss[DS_WARPS];
  float mass[DS_WARPS];
  float z[kMaxDistillTop];       // the listed entries' z
  int repeated;                  // an id is listed twice
};

// With a gradient, in dynamic shared memory: the list, and a table of its ids. Of the entries with one
// id the first stands for all; only where a row has such entries are lists searched, by a warp for each
// repeated id, and their p added up in an order that the list alone fixes.
struct IdTable {
  static constexpr int SINGLE = 1 << 30;
  float* p;                      // k
  int* id;                       // k; -1: absent
  int* slot;                     // hash_mask + 1: first entry with the slot's id, + SINGLE while it is
                                 // the only one; -1: free
  __device__ __forceinline__ IdTable(const DsArgs& a, int* mem) {
    slot = mem;
    id = slot + a.hash_mask + 1;
    p = reinterpret_cast<float*>(id + a.k);
  }
  // Two products by 2^32 / golden ratio with a shift between them: one alone maps some arithmetic
  // progressions of ids to a few slots (4096 x 128256, rows of random steps: 547 us, with both 475).
  // The upper half gives the first slot, the lower half the (odd) step to the next, so that runs of
  // taken slots do not grow together (k = 512: 234 us with steps of one).
  __device__ __forceinline__ uint32_t hash(int j) const {
    const uint32_t h = static_cast<uint32_t>(id[j]) * 2654435769u;
    return (h ^ (h >> 15)) * 2654435769u;
  }
  // What the first slot of entry j (of hash h) held when j asked for it; -1: j has it
  __device__ __forceinline__ int ask(const DsArgs& a, int j, uint32_t h) const {
    return atomicCAS(&slot[(h >> 16) & a.hash_mask], -1, j + SINGLE);
  }
  // Enters entry j, given what ask returned; true where its id was there already. Every id[] is
  // written before.
  __device__ __forceinline__ bool settle(const DsArgs& a, int j, uint32_t h, int old) const {
    uint32_t at = (h >> 16) & a.hash_mask;
    while (old != -1) {          // at most k of >= 2 k slots are taken
      const int first = old & (SINGLE - 1);
      if (id[first] == id[j]) {  // a slot's entries may change, its id does not
        atomicMin(&slot[at], min(first, j));
        return true;
      }
      at = (at + (h | 1)) & a.hash_mask;
      old = atomicCAS(&slot[at], -1, j + SINGLE);
    }
    return false;
  }
  // The slot of entry j, when all are entered
  __device__ __forceinline__ int find(const DsArgs& a, int j) const {
    const uint32_t h = hash(j);
    uint32_t at = (h >> 16) & a.hash_mask;
    while (id[slot[at] & (SINGLE - 1)] != id[j]) at = (at + (h | 1)) & a.hash_mask;
    return slot[at];
  }
  // For a whole warp, one entry j a lane (mine: it asks). mine stays where j is its id's first entry;
  // p becomes the sum over the id's entries.
  __device__ __forceinline__ void join(const DsArgs& a, int j, bool& mine, float& pj) const {
    const int at = mine ? find(a, j) : 0;
    mine = mine && (at & (SINGLE - 1)) == j;
    const int lane = threadIdx.x & 31;
    unsigned todo = __ballot_sync(0xffffffffu, mine && !(at & SINGLE));
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      const int want = id[__shfl_sync(0xffffffffu, j, from)];
      float sum = 0.f;
      for (int l = lane; l < a.k; l += 32)
        if (id[l] == want) sum += p[l];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == from) pj = sum;
    }
  }
};
__host__ __device__ inline int id_table_words(const DsArgs& a) {
  return a.hash_mask + 1 + 2 * a.k;
}

// The listed entries of a row: thread t has entries t, t + NT, ... (KPT of them)
template <int KPT>
struct Entries {
  int id[KPT];                   // -1: absent
  float t[KPT], z[KPT], p[KPT];
};

template <int NT, int KPT>
__device__ __forceinline__ void load_entries(const DsArgs& a, int64_t row, Entries<KPT>& e) {
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int j = threadIdx.x + i * NT;
    e.id[i] = -1;
    e.t[i] = kNegInf;
    if (j < a.k) {
      const int id = a.ids[row * a.ld_ids + j];
      const int64_t o = row * a.ld_top + j;
      const float t = a.top_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.top)[o])
                                 : static_cast<const float*>(a.top)[o];
      if (id >= 0 && id < a.v && t != kNegInf) {       // -inf counts nothing
        e.id[i] = id;
        e.t[i] = t;
      }
    }
  }
}
// z[id] is read where it is used: for the loss (all entries), and for the gradients of the entries
// in the CTA's own slice (other slices may already be overwritten when dz is z).
template <typename T, int KPT>
__device__ __forceinline__ void gather_logits(const Slice<T>& s, int part, bool all,
                                              Entries<KPT>& e) {
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    e.z[i] = 0.f;
    if (e.id[i] >= 0 && (all || s.owns(e.id[i], part))) e.z[i] = ds_ld(s.row + e.id[i]);
  }
}

// A log-sum in two parts, the reference's and the sum's: a logit's distance from it keeps the second
// where the first is large. -inf where nothing was seen.
struct LogSum {
  double ref;
  float log;
  __device__ __forceinline__ double total() const { return ref + log; }
};
__device__ __forceinline__ LogSum ds_lse(const DsArgs& a, RunSum r) {
  return {ds_wide(r.m, a.c) ? __dmul_rn(r.m, a.inv_tau) : r.m * a.c * a.nat, logf(r.s)};
}
// log of an entry's share. The product is rounded as that of the reference: equal ones cancel.
__device__ __forceinline__ double ds_log_share(const DsArgs& a, float x, LogSum l) {
  return __dsub_rn(__dmul_rn(x, a.inv_tau), l.ref) - l.log;
}

// Joins the CTA's statistics, the row's (exchange: what other CTAs have) and the listed entries';
// gives p and, in the CTA that reports the row, the loss. GRAD: fills the id table. sync(): a
// barrier of the NT threads.
template <int NT, bool LSE, bool GRAD, int KPT, typename Sync, typename Exchange>
__device__ __forceinline__ void row_statistics(const DsArgs& a, int64_t row, int part, float w,
                                               float top_lse, DsShared& sh, int* table_mem,
                                               RunSum& rs, Entries<KPT>& e, float& mass, Sync sync,
                                               Exchange exchange) {
  constexpr int NW = NT / 32;
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
  const bool report = LSE && part == 0;
  if (lane == 0) sh.list[warp] = ls;
  // z[id] has arrived before any other CTA learns of this one's statistics and stores its part
  // of the row (dz may be z)
  if (report && lists) {
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (tid + i * NT < a.k) *const_cast<volatile float*>(&sh.z[tid + i * NT]) = e.z[i];
  }
  if (GRAD) {
    const IdTable table(a, table_mem);
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (tid + i * NT < a.k) table.id[tid + i * NT] = e.id[i];
    if (tid == 0) sh.repeated = 0;
  }
  sync();
  if (LSE) {
    rs = ds_join_lanes<NW>(sh.row[lane % NW], a.c);
    if (a.cl > 1) rs = exchange(rs);
  }
  double part_loss = 0.0;
  const LogSum lse = report ? ds_lse(a, rs) : LogSum{0.0, 0.f};
  mass = 0.f;
#pragma unroll
  for (int i = 0; i < KPT; ++i) e.p[i] = 0.f;
  if (lists) {
    // log p_j = t_j / tau - L_t in fp64: the difference of two numbers of the logits' size
    ls = ds_join_lanes<NW>(sh.list[lane % NW], a.c);
    const LogSum norm = a.top_lse ? LogSum{static_cast<double>(top_lse), 0.f} : ds_lse(a, ls);
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = tid + i * NT;
      if (j >= a.k) break;
      if (e.t[i] != kNegInf) {
        const double lp = ds_log_share(a, e.t[i], norm);
        const float p = expf(static_cast<float>(lp));
        e.p[i] = p;
        mass += p;
        // a listed entry that the student masks has an infinite loss
        if (report && p != 0.f)
          part_loss += e.z[i] == kNegInf ? static_cast<double>(INFINITY)
                                         : p * (lp - ds_log_share(a, e.z[i], lse));
      }
      if (GRAD) {
        const IdTable table(a, table_mem);
        table.p[j] = e.p[i];
        if (e.id[i] >= 0) {
          const uint32_t h = table.hash(j);
          if (table.settle(a, j, h, table.ask(a, j, h))) sh.repeated = 1;
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
  sync();
  mass = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) mass += sh.mass[i];
  if (report && tid == 0) {
    double tot = 0.0;
    for (int i = 0; i < NW; ++i) tot += sh.loss[i];
    a.loss[row] = w == 0.f ? 0.f : static_cast<float>(static_cast<double>(w) * a.tau * a.tau * tot);
    if (a.lse) a.lse[row] = static_cast<float>(lse.total());
  }
}

// The row's statistics from those of the cluster's CTAs. The second arrival is waited for before
// the CTA ends.
__device__ __forceinline__ RunSum exchange_cluster(const DsArgs& a, DsShared& sh, RunSum mine) {
  if (threadIdx.x == 0) sh.mine = mine;
  ds_cluster_arrive();
  ds_cluster_wait();
  const int r = (threadIdx.x & 31) % DS_MAX_CL;
  RunSum all{kNegInf, 0.f};
  if (r < a.cl) all = {ds_remote(&sh.mine.m, r), ds_remote(&sh.mine.s, r)};
  all = ds_join_lanes<DS_MAX_CL>(all, a.c);
  ds_cluster_arrive();
  return all;
}

template <int NT>
__device__ __forceinline__ void clear_table(const DsArgs& a, int* table_mem) {
  const IdTable table(a, table_mem);
  for (int i = threadIdx.x; i <= a.hash_mask; i += NT) table.slot[i] = -1;
}

// Gradients of the listed entries in this CTA's slice. patch_id = -1: not this thread's to store.
template <int NT, typename T, int KPT>
__device__ __forceinline__ void list_gradients(const DsArgs& a, const DsShared& sh,
                                               const Slice<T>& s, const Entries<KPT>& e, RunSum rs,
                                               float coef, float wt, int part, int* table_mem,
                                               float (&patch)[KPT], int (&patch_id)[KPT]) {
  const IdTable table(a, table_mem);
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int j = threadIdx.x + i * NT;
    patch_id[i] = -1;
    patch[i] = 0.f;
    bool mine = j < a.k && e.id[i] >= 0 && s.owns(e.id[i], part);
    float p = e.p[i];
    if (sh.repeated) table.join(a, j, mine, p);
    if (mine) {
      patch_id[i] = e.id[i];
      if (wt != 0.f)
        patch[i] = coef == 0.f ? -wt * p
                               : fmaf(coef, ex2(ds_exponent(e.z[i], rs.m, a.c)), -wt * p);
    }
  }
}

// Gradients of U vectors, `stride` elements apart from d on; vector u is stored where u < have.
template <typename T, typename D, int U>
__device__ __forceinline__ void put_gradients(D* d, int64_t stride, int have, bool aligned,
                                              const uint4 (&raw)[U], bool wide, float m, float c,
                                              float coef) {
  constexpr int NP = Vec<T>::VE / 2;
  uint64_t g[U][NP];
  if (coef == 0.f) {                                   // whatever z holds
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NP; ++e) g[u][e] = 0;
  } else {
    const uint64_t cc = pack2(c, c), k = pack2(coef, coef);
    const float r = wide ? -m : -(m * c);
    const uint64_t ref = pack2(r, r);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t x[NP];
      Vec<T>::get(raw[u], x);
#pragma unroll
      for (int e = 0; e < NP; ++e) g[u][e] = x[e];
    }
    if (wide) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < NP; ++e) g[u][e] = mul2(add2(g[u][e], ref), cc);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < NP; ++e) g[u][e] = fma2(g[u][e], cc, ref);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float2 t = unpack2(g[u][e]);
        g[u][e] = mul2(k, pack2(ex2(t.x), ex2(t.y)));
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < have) store_vec<D, Vec<T>::VE>(d + u * stride, aligned, g[u]);
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

// Loss and gradient of long rows. Cluster y takes rows y, y + gridDim.y, ...; chunk g of the CTA
// (its slices' chunks, row after row) sits in ring slot g % chunks.
//
// Per row: every consumer warp sends its statistics to all CTAs of the cluster and waits for all of
// theirs (8 warps x cl messages on barrier got). Rows alternate between two of each barrier and
// buffer (turn): a message for the next row may come before this row's last, one for the row after
// that is sent only when this CTA has sent its next, and it sends that only when its list warp too
// has read this row's (barrier taken). The list warp gives P and z[id] (barrier ready)
// before the CTA's first warp sends: no CTA stores a part of the row (dz may be z) before every
// z[id] of it is read. It stores the listed entries' gradients when the warps have stored the row's
// (barrier stored).
//
// 4096 x 128256 bf16, k = 128: 475 us, 4.4 TB/s read and written (floor 325 us; the two exponentials an
// element take 233 of their unit). Reading the row again from L2 instead of the ring took 592 us, three
// CTAs per SM with shorter rings 619.
template <typename T, typename D>
__global__ void __launch_bounds__(DS_RING_THREADS, 2)
    distill_ring_kernel(DsArgs a, int64_t n, int chunks, int* err) {
  constexpr int VE = Vec<T>::VE, U = DS_CHUNK_VECS / DS_THREADS;
  constexpr uint32_t CHUNK = DS_CHUNK_VECS * 16;
  extern __shared__ __align__(128) uint8_t ds_ring[];
  __shared__ RunSum stats[2][DS_WARPS * DS_MAX_CL];
  __shared__ float masses[2];
  __shared__ __align__(8) uint64_t full[DS_MAX_CHUNKS], empty[DS_MAX_CHUNKS], got[2], ready[2],
      taken[2], stored[2];
  __shared__ int abort_flag;
  const int part = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t step = gridDim.y;
  auto slice = [&](int64_t row) {
    return Slice<T>(static_cast<const T*>(a.z) + row * a.ld_z, a.v, part, a.per);
  };
  if (tid == 0) {
    for (int i = 0; i < chunks; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], DS_WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&got[i], a.cl > 1 ? 1 : DS_WARPS);
      mbar_init(&ready[i], 1);
      mbar_init(&taken[i], 1);
      mbar_init(&stored[i], DS_WARPS);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (a.cl > 1) {                                     // peers' barriers exist before any message
    ds_cluster_arrive();
    ds_cluster_wait();
  }
  volatile int* const aborted = &abort_flag;
  // the row's statistics from the messages
  auto joined = [&](int turn) {
    const int all = a.cl * DS_WARPS;
    RunSum r{kNegInf, 0.f}, r2{kNegInf, 0.f};
    if (lane < all) r = stats[turn][lane];
    if (lane + 32 < all) r2 = stats[turn][lane + 32];
    const float m = fmaxf(r.m, r2.m);
    const float f = r.m == m ? 1.f : ds_rescale(r.m, m, a.c);
    const float f2 = r2.m == m ? 1.f : ds_rescale(r2.m, m, a.c);
    return ds_join_lanes<32>({m, r.s * f + r2.s * f2}, a.c);
  };
  // After a wait that gave up (recorded in err) the roles run on over whatever shared memory holds:
  // every later wait returns at once.
  if (warp == DS_WARPS) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0;
      uint32_t parity = 1, issued = 0;                // a fresh barrier's previous phase is over
      bool ok = true;
      for (int64_t row = blockIdx.y; row < n && ok; row += step) {
        const Slice<T> s = slice(row);
        for (int i = s.i0; i < s.i1; i += DS_CHUNK_VECS) {
          if (!mbar_wait(&empty[slot], parity, aborted, err, DEV_ERR_TMA_WAIT)) {
            ok = false;
            break;
          }
          const uint32_t bytes = static_cast<uint32_t>(min(DS_CHUNK_VECS, s.i1 - i)) * 16;
          mbar_arrive_expect_tx(&full[slot], bytes);
          ds_bulk_load(ds_ring + slot * CHUNK, s.at(i), bytes, &full[slot]);
          ++issued;
          if (++slot == chunks) {
            slot = 0;
            parity ^= 1u;
          }
        }
      }
      if (*aborted) {                                 // copies in flight land before the CTA ends
        const uint32_t ring = chunks;
        for (uint32_t g = issued > ring ? issued - ring : 0; g < issued; ++g)
          mbar_drain(&full[g % ring], (g / ring) & 1u, 1000000000ull);
      }
    }
  } else if (warp > DS_WARPS) {
    // ------------------------------------------------------------------ the teacher's lists
    const int turn = warp - DS_WARPS - 1;             // this warp's rows
    const IdTable table(a, reinterpret_cast<int*>(ds_ring + chunks * CHUNK) +
                               turn * (id_table_words(a) + 4 * a.k));
    float* const t = table.p + a.k;                   // logits (-inf: absent), z[id]
    float* const zk = t + a.k;
    int* const own = reinterpret_cast<int*>(zk + a.k);       // id where it lies in this CTA's slice
    float* const grad = reinterpret_cast<float*>(own + a.k);
    uint32_t parity = 0;
    for (int64_t row = blockIdx.y + turn * step; row < n; row += 2 * step, parity ^= 1u) {
      const Slice<T> s = slice(row);
      const float w = a.weight ? a.weight[row] : 1.f;
      const float wt = w * a.tau;
      for (int i = lane; i <= a.hash_mask; i += 32) table.slot[i] = -1;
      RunSum ls{kNegInf, 0.f};
      constexpr int B = 4;                            // entries per lane with loads in flight
      for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
        int id[B];
        float x[B], z[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int j = j0 + 32 * b;
          id[b] = -1;
          x[b] = kNegInf;
          if (j < a.k) {
            id[b] = a.ids[row * a.ld_ids + j];
            const int64_t o = row * a.ld_top + j;
            x[b] = a.top_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.top)[o])
                              : static_cast<const float*>(a.top)[o];
          }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (id[b] < 0 || id[b] >= a.v || x[b] == kNegInf) {   // -inf counts nothing
            id[b] = -1;
            x[b] = kNegInf;
          }
          z[b] = id[b] >= 0 && (part == 0 || s.owns(id[b], part)) ? ds_ld(s.row + id[b]) : 0.f;
          ls.m = fmaxf(ls.m, x[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int j = j0 + 32 * b;
          if (j < a.k) {
            zk[j] = z[b];
            table.id[j] = id[b];
            t[j] = x[b];
            own[j] = id[b] >= 0 && s.owns(id[b], part) ? id[b] : -1;
          }
        }
      }
      // the list is worked through B entries a lane at a time, whose steps overlap
      const float lm = ls.m == kNegInf ? 0.f : ls.m;
      for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
        float x[B];
#pragma unroll
        for (int b = 0; b < B; ++b) x[b] = j0 + 32 * b < a.k ? t[j0 + 32 * b] : kNegInf;
#pragma unroll
        for (int b = 0; b < B; ++b)                   // a NaN logit makes s NaN
          if (x[b] != kNegInf) ls.s += ex2(ds_exponent(x[b], lm, a.c));
      }
      ls = ds_join_lanes<32>(ls, a.c);
      // log p_j = t_j / tau - L_t in fp64: the difference of two numbers of the logits' size
      const LogSum norm =
          a.top_lse ? LogSum{static_cast<double>(a.top_lse[row]), 0.f} : ds_lse(a, ls);
      float mass = 0.f;
      for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
        float p[B];
#pragma unroll
        for (int b = 0; b < B; ++b) p[b] = j0 + 32 * b < a.k ? t[j0 + 32 * b] : kNegInf;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          p[b] = p[b] == kNegInf ? 0.f : expf(static_cast<float>(ds_log_share(a, p[b], norm)));
          mass += p[b];
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (j0 + 32 * b < a.k) table.p[j0 + 32 * b] = p[b];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
      __syncwarp();              // every lane has its z[id]: from here on the row may be overwritten
      if (lane == 0) {
        masses[turn] = mass;
        mbar_arrive(&ready[turn]);
      }
      __syncwarp();
      bool again = false;
      for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
        int old[B];
        uint32_t h[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int j = j0 + 32 * b;
          old[b] = -1;
          if (j < a.k && table.id[j] >= 0) {
            h[b] = table.hash(j);
            old[b] = table.ask(a, j, h[b]);
          }
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (old[b] != -1) again |= table.settle(a, j0 + 32 * b, h[b], old[b]);
      }
      again = __any_sync(0xffffffffu, again);
      __syncwarp();              // the table's other lanes' entries: a vote alone orders no memory
      if (again) {
        for (int j = lane; j - lane < a.k; j += 32) {
          bool mine = j < a.k && own[j] >= 0;
          float p = mine ? table.p[j] : 0.f;
          table.join(a, j, mine, p);
          if (j < a.k) {
            if (!mine) own[j] = -1;
            grad[j] = p;
          }
        }
      }
      mbar_wait(&got[turn], parity, aborted, err, DEV_ERR_EPI_WAIT);
      const RunSum rs = joined(turn);
      __syncwarp();
      if (lane == 0) mbar_arrive(&taken[turn]);
      const float coef = ds_coef(wt, mass, rs.s);
      for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
        float p[B], z[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int j = min(j0 + 32 * b, a.k - 1);
          p[b] = again ? grad[j] : table.p[j];
          z[b] = zk[j];
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const float g = coef == 0.f ? -wt * p[b]
                                      : fmaf(coef, ex2(ds_exponent(z[b], rs.m, a.c)), -wt * p[b]);
          if (j0 + 32 * b < a.k) grad[j0 + 32 * b] = wt == 0.f ? 0.f : g;
        }
      }
      if (part == 0) {
        const LogSum lse = ds_lse(a, rs);
        double loss = 0.0;
        for (int j0 = lane; j0 < a.k; j0 += 32 * B) {
          float p[B], x[B], z[B];
#pragma unroll
          for (int b = 0; b < B; ++b) {
            const int j = min(j0 + 32 * b, a.k - 1);
            p[b] = j0 + 32 * b < a.k ? table.p[j] : 0.f;
            x[b] = t[j];
            z[b] = zk[j];
          }
#pragma unroll
          for (int b = 0; b < B; ++b)
            if (p[b] != 0.f)                          // a masked listed entry: infinite loss
              loss += z[b] == kNegInf ? static_cast<double>(INFINITY)
                                      : p[b] * (ds_log_share(a, x[b], norm) -
                                                ds_log_share(a, z[b], lse));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
        if (lane == 0) {
          a.loss[row] = w == 0.f ? 0.f
                                 : static_cast<float>(static_cast<double>(w) * a.tau * a.tau * loss);
          if (a.lse) a.lse[row] = static_cast<float>(lse.total());
        }
      }
      mbar_wait(&stored[turn], parity, aborted, err, DEV_ERR_EPI_WAIT);
      D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
#pragma unroll 4
      for (int j = lane; j < a.k; j += 32)
        if (own[j] >= 0) ds_st(dz + own[j], grad[j]);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ consumers
    int slot = 0, turn = 0;
    uint32_t full_parity = 0, parity = 0;
    for (int64_t row = blockIdx.y; row < n; row += step) {
      const Slice<T> s = slice(row);
      if (tid == 0 && a.cl > 1) mbar_arrive_expect_tx(&got[turn], 8 * DS_WARPS * a.cl);
      const float w = a.weight ? a.weight[row] : 1.f;
      const float ze = s.edge >= 0 ? ds_ld(s.row + s.edge) : kNegInf;
      const int slot0 = slot;
      RunSum rs{kNegInf, 0.f};
      for (int i = s.i0; i < s.i1; i += DS_CHUNK_VECS) {
        mbar_wait(&full[slot], full_parity, aborted, err, DEV_ERR_LOAD_WAIT);
        const uint4* ring = reinterpret_cast<const uint4*>(ds_ring + slot * CHUNK) + tid;
        uint4 raw[U];
        if (i + DS_CHUNK_VECS <= s.i1) {
#pragma unroll
          for (int u = 0; u < U; ++u) raw[u] = ring[u * DS_THREADS];
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            raw[u] = i + tid + u * DS_THREADS < s.i1 ? ring[u * DS_THREADS] : none_vec<T>();
        }
        float most = kNegInf;
#pragma unroll
        for (int u = 0; u < U; ++u) most = fmaxf(most, Vec<T>::max(raw[u]));
        // the thread's reference changes only where a sum could overflow (its first chunk, and a
        // value 2^64 above): the exponentials of a chunk need not wait for its maximum
        if ((most - rs.m) * a.c > 64.f) {
          if (rs.s != 0.f) rs.s *= ds_rescale(rs.m, most, a.c);
          rs.m = most;
        }
        const float m = rs.m == kNegInf ? 0.f : rs.m;   // nothing but -inf (or NaN) so far
        const bool mwide = ds_wide(m, a.c);
        rs.s += ds_terms<T, U>(raw, mwide, m, a.c);
        if (++slot == chunks) {
          slot = 0;
          full_parity ^= 1u;
        }
      }
      if (s.edge >= 0 && ze != kNegInf) {
        // the maximum's own term too: 2^(ze c - fl(ze c)) is not 1, and +inf makes it NaN
        const float m = fmaxf(rs.m, ze);
        rs.s = (rs.m == m ? rs.s : rs.s * ds_rescale(rs.m, m, a.c)) + ex2(ds_exponent(ze, m, a.c));
        rs.m = m;
      }
      rs = ds_join_lanes<32>(rs, a.c);
      mbar_wait(&ready[turn], parity, aborted, err, DEV_ERR_EPI_WAIT);
      // the list warp has read the row before's statistics: the next message into them can only
      // follow this row's
      if (row != blockIdx.y)
        mbar_wait(&taken[turn ^ 1], turn ? parity : parity ^ 1u, aborted, err, DEV_ERR_EPI_WAIT);
      if (a.cl > 1) {
        if (lane < a.cl) ds_send(&stats[turn][part * DS_WARPS + warp], &got[turn], lane, rs);
      } else if (lane == 0) {
        stats[turn][warp] = rs;
        mbar_arrive(&got[turn]);
      }
      mbar_wait(&got[turn], parity, aborted, err, DEV_ERR_EPI_WAIT);
      rs = joined(turn);
      const float coef = ds_coef(w * a.tau, masses[turn], rs.s);
      D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
      const bool al = store_aligned(s, dz), wide = ds_wide(rs.m, a.c);
      D* d = dz + s.head + static_cast<int64_t>(s.i0 + tid) * VE;
      int back = slot0;
      for (int i = s.i0; i < s.i1; i += DS_CHUNK_VECS, d += DS_CHUNK_VECS * VE) {
        const uint4* ring = reinterpret_cast<const uint4*>(ds_ring + back * CHUNK) + tid;
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = ring[u * DS_THREADS];
        put_gradients<T, D, U>(d, DS_THREADS * VE,
                               (s.i1 - i - tid + DS_THREADS - 1) / DS_THREADS, al, raw, wide, rs.m,
                               a.c, coef);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[back]);
        if (++back == chunks) back = 0;
      }
      put_edge(s, dz, ze, rs.m, a.c, coef);
      __syncwarp();
      if (lane == 0) mbar_arrive(&stored[turn]);
      if (turn) parity ^= 1u;
      turn ^= 1;
    }
  }
  if (a.cl > 1) {                                     // no CTA ends while a message is under way
    __syncwarp();
    ds_cluster_arrive();
    ds_cluster_wait();
  }
}

// Loss and gradient; NV vectors of z per thread stay in registers. 96 x 50001 bf16: 8.6 us of the GPU,
// the launch, one read and the barriers' latency; 256 x 128256: 40 us, 3.3 TB/s.
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
  extern __shared__ int ds_table[];
  Entries<KPT> e;
  load_entries<DS_THREADS>(a, row, e);
  gather_logits(s, part, part == 0, e);
  clear_table<DS_THREADS>(a, ds_table);
  const float tl = a.top_lse ? a.top_lse[row] : 0.f;
  const float w = a.weight ? a.weight[row] : 1.f;
  RunSum rs{ze, 0.f};
#pragma unroll
  for (int n = 0; n < NV; ++n) rs.m = fmaxf(rs.m, Vec<T>::max(raw[n]));
  // a thread whose entries are all -inf adds nothing, to any reference (NaN it adds)
  const float m = rs.m == kNegInf ? 0.f : rs.m;
  const bool mwide = ds_wide(m, a.c);
  rs.s = ex2(ds_exponent(ze, m, a.c));
#pragma unroll
  for (int n = 0; n < NV; n += 4) {
    const uint4 four[4] = {raw[n], raw[n + 1], raw[n + 2], raw[n + 3]};
    rs.s += ds_terms<T, 4>(four, mwide, m, a.c);
    asm volatile("" : "+f"(rs.s));                     // four vectors unpacked at a time
  }
  // the gradient unpacks the vectors again: nothing unpacked lives across the statistics
#pragma unroll
  for (int n = 0; n < NV; ++n)
    asm volatile("" : "+r"(raw[n].x), "+r"(raw[n].y), "+r"(raw[n].z), "+r"(raw[n].w));
  float mass;
  row_statistics<DS_THREADS, true, true, KPT>(
      a, row, part, w, tl, sh, ds_table, rs, e, mass, [] { __syncthreads(); },
      [&](RunSum r) { return exchange_cluster(a, sh, r); });
  const float wt = w * a.tau;
  const float coef = ds_coef(wt, mass, rs.s);
  float patch[KPT];
  int patch_id[KPT];
  list_gradients<DS_THREADS>(a, sh, s, e, rs, coef, wt, part, ds_table, patch, patch_id);
  D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
  const bool al = store_aligned(s, dz), wide = ds_wide(rs.m, a.c);
  const int mine = s.i1 - s.i0 - tid;                   // vectors tid, tid + 256, ... below it
  D* d = dz + s.head + static_cast<int64_t>(s.i0 + tid) * Vec<T>::VE;
#pragma unroll
  for (int n = 0; n < NV; n += 2) {
    const uint4 two[2] = {raw[n], raw[n + 1]};
    put_gradients<T, D, 2>(d + static_cast<int64_t>(n) * DS_THREADS * Vec<T>::VE,
                           DS_THREADS * Vec<T>::VE,
                           (mine + DS_THREADS - 1) / DS_THREADS - n, al, two, wide, rs.m, a.c, coef);
  }
  put_edge(s, dz, ze, rs.m, a.c, coef);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < KPT; ++i)
    if (patch_id[i] >= 0) ds_st(dz + patch_id[i], patch[i]);
  if (a.cl > 1) ds_cluster_wait();                     // a peer may still read this CTA's sums
}

// LSE: the row's statistics are taken from z (else lse_in). GRAD: dz is written. Bound by HBM on long
// rows: the loss of 4096 x 128256 bf16 at 6.4 TB/s (163 us), the gradient from lse of 1024 x 32000 fp32
// at 5.2 TB/s (50 us).
template <typename T, typename D, bool LSE, bool GRAD, int KPT>
__global__ void __launch_bounds__(DS_THREADS) distill_stream_kernel(DsArgs a) {
  __shared__ DsShared sh;
  const int64_t row = a.row0 + blockIdx.y;
  const int part = blockIdx.x;
  const int tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
  const Slice<T> s(z, a.v, part, a.per);
  extern __shared__ int ds_table[];
  Entries<KPT> e;
  load_entries<DS_THREADS>(a, row, e);
  gather_logits(s, part, LSE && part == 0, e);
  if (GRAD) clear_table<DS_THREADS>(a, ds_table);
  const float tl = a.top_lse ? a.top_lse[row] : 0.f;
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
      rs.s += ds_terms<T, U>(raw, mwide, m, a.c);
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
  row_statistics<DS_THREADS, LSE, GRAD, KPT>(
      a, row, part, w, tl, sh, ds_table, rs, e, mass, [] { __syncthreads(); },
      [&](RunSum r) { return exchange_cluster(a, sh, r); });
  if (GRAD) {
    const float wt = w * a.tau;
    const float coef = ds_coef(wt, mass, rs.s);
    float patch[KPT];
    int patch_id[KPT];
    list_gradients<DS_THREADS>(a, sh, s, e, rs, coef, wt, part, ds_table, patch, patch_id);
    D* dz = static_cast<D*>(a.dz) + row * a.ld_dz;
    const bool al = store_aligned(s, dz), wide = ds_wide(rs.m, a.c);
    // dz may be z: every entry's z[id] was read before the first barrier above
    for (int i = s.i0 + tid; i < s.i1; i += U * DS_THREADS) {
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * DS_THREADS < s.i1) raw[u] = s.load(i + u * DS_THREADS);
      put_gradients<T, D, U>(dz + s.head + static_cast<int64_t>(i) * Vec<T>::VE,
                             DS_THREADS * Vec<T>::VE, (s.i1 - i + DS_THREADS - 1) / DS_THREADS, al,
                             raw, wide, rs.m, a.c, coef);
    }
    put_edge(s, dz, ze, rs.m, a.c, coef);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (patch_id[i] >= 0) ds_st(dz + patch_id[i], patch[i]);
  }
  if (LSE && a.cl > 1) ds_cluster_wait();              // a peer may still read this CTA's sums
}

cudaLaunchConfig_t ds_config(const DsArgs& a, int64_t rows, int threads, size_t smem, bool cluster,
                             cudaLaunchAttribute* attr, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.cl, static_cast<unsigned>(rows));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(a.cl);
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster && a.cl > 1 ? 1 : 0;
  return cfg;
}

kronq_status launch_rows(void (*kern)(DsArgs), DsArgs a, int n, bool cluster, bool table,
                         const char* what, cudaStream_t stream) {
  constexpr int most = 65535;                      // rows per launch: the grid's y extent
  const size_t smem = table ? 4 * static_cast<size_t>(id_table_words(a)) : 0;
  for (a.row0 = 0; a.row0 < n; a.row0 += most) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = ds_config(a, std::min<int64_t>(most, n - a.row0), DS_THREADS,
                                             smem, cluster, &attr, stream);
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a);
    if (err != cudaSuccess) return fail(KRONQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(err));
    KQ_TRY(check_launch(what));
  }
  return KRONQ_OK;
}

// Shared memory of the ring kernel: the chunks, then for each list warp the id table and the
// entries' logits, z, ids and gradients. Two CTAs per SM where a row fits them.
size_t ring_list_bytes(const DsArgs& a) {
  return 8 * (static_cast<size_t>(id_table_words(a)) + 4 * a.k);
}
int ring_room(int ctas) { return (ctas == 2 ? 111 : 224) * 1024; }     // per CTA
int ring_chunks(const DsArgs& a, int ctas) {
  const int64_t room = ring_room(ctas) - static_cast<int64_t>(ring_list_bytes(a));
  return static_cast<int>(std::min<int64_t>(DS_MAX_CHUNKS, room / (DS_CHUNK_VECS * 16)));
}

template <typename T, typename D>
kronq_status launch_ring(const DsArgs& a, int n, int ctas, cudaStream_t stream) {
  const int chunks = ring_chunks(a, ctas);
  const size_t smem = static_cast<size_t>(chunks) * DS_CHUNK_VECS * 16 + ring_list_bytes(a);
  auto kern = distill_ring_kernel<T, D>;
  // the most of any call: calls of other threads launch this kernel with other lists
  static std::atomic<uint64_t> allowed{0};
  KQ_TRY(allow_smem(reinterpret_cast<const void*>(kern), ring_room(1), allowed));
  int* err = device_error_word();
  if (!err) return fail(KRONQ_ERR_CUDA, "device error word unavailable");
  // As many clusters as run at once: one more would start when all others have ended. The query
  // takes about 15 us, so its last answer is kept (it depends on the device, cl and smem).
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = ds_config(a, 1, DS_RING_THREADS, smem, true, &attr, stream);
  int clusters = ctas * device_sms();
  if (a.cl > 1) {
    static thread_local int64_t key = -1;
    static thread_local int answer = 0;
    int dev = 0;
    KQ_CUDA_TRY(cudaGetDevice(&dev));
    const int64_t k = (static_cast<int64_t>(dev) << 32) + (static_cast<int64_t>(a.cl) << 24) + smem;
    if (k != key) {
      KQ_CUDA_TRY(cudaOccupancyMaxActiveClusters(&answer, kern, &cfg));
      key = k;
    }
    clusters = answer;
  }
  cfg.gridDim.y = static_cast<unsigned>(std::min(n, std::max(1, clusters)));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, static_cast<int64_t>(n), chunks, err);
  if (e != cudaSuccess)
    return fail(KRONQ_ERR_CUDA, "distill_ring_kernel: %s", cudaGetErrorString(e));
  return check_launch("distill_ring_kernel");
}

template <typename T, typename D, int KPT>
kronq_status launch_distill(DsArgs a, int n, bool lse, bool grad, cudaStream_t stream) {
  constexpr int NV = 8;
  const int64_t vecs = static_cast<int64_t>(a.v) / Vec<T>::VE + 1;    // at most, and at least one
  if (!lse) {
    // the gradient alone has no statistics to exchange: any number of slices, of at least four
    // vectors per thread, but no more than give every SM twelve CTAs (each works through the list)
    const int64_t most = std::max<int64_t>(1, (12LL * device_sms() + n - 1) / n);
    a.cl = static_cast<int>(std::max<int64_t>(1, std::min((vecs + 4 * DS_THREADS - 1) / (4 * DS_THREADS), most)));
    a.per = static_cast<int>((vecs + a.cl - 1) / a.cl);
    return launch_rows(distill_stream_kernel<T, D, false, true, KPT>, a, n, false, true,
                       "distill_stream_kernel", stream);
  }
  auto cut = [&] { return static_cast<int>((vecs + a.cl - 1) / a.cl); };
  if (grad) {
    // Long rows, at least two per cluster: the fewest CTAs that hold a row with two chunks to spare.
    // Two CTAs per SM, unless the list takes so much of their memory that a row needs four times the
    // CTAs, each of which works through the list (1024 rows, us with two and with one: 128256 wide,
    // k = 256 (8 and 2 CTAs) 254 and 158, k = 512 408 and 203; 50001 wide, k = 256 (4 and 1) 127 and 78;
    // 128256 wide, k = 128 (4 and 2) 128 and 154).
    int cl[3] = {0, 0, 0};                       // by CTAs per SM; 0: a row does not fit
    for (int ctas = 1; ctas <= 2; ++ctas) {
      const int64_t hold = static_cast<int64_t>(ring_chunks(a, ctas) - 2) * DS_CHUNK_VECS;
      for (int c = 1; c <= DS_MAX_CL && cl[ctas] == 0; c *= 2)
        if ((vecs + c - 1) / c <= hold) cl[ctas] = c;
    }
    const int ctas = cl[2] == 0 || cl[2] >= 4 * cl[1] ? 1 : 2;
    // A list of 1 / 8 of a slice's vectors or more takes the list warps longer than the slice takes the
    // others; the kernels below work through it with all of theirs (1024 rows, us, ring and below: 32000
    // wide, k = 300 74 and 66, 512 111 and 72; 50001 wide, 512 117 and 125, 700 137 and 131, 1024 195 and
    // 158; 128256 wide, 700 246 and 295, 1024 348 and 340; 300000 wide, 512 453 and 547, 700 990 and 567).
    if (vecs > DS_RING_MIN_VECS && cl[ctas] > 0 && 8 * a.k < (vecs + cl[ctas] - 1) / cl[ctas] &&
        static_cast<int64_t>(n) * cl[ctas] >= 2 * ctas * device_sms()) {
      a.cl = cl[ctas];
      a.per = cut();
      return launch_ring<T, D>(a, n, ctas, stream);
    }
  }
  // Slices: enough to give every SM two CTAs when rows are few, none shorter than one vector per
  // thread.
  a.cl = 1;
  while (a.cl < DS_MAX_CL && static_cast<int64_t>(n) * a.cl < 2 * device_sms() &&
         vecs > static_cast<int64_t>(a.cl) * DS_THREADS)
    a.cl *= 2;
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
  return a.k <= DS_THREADS
             ? launch_distill<T, D, 1>(a, n, lse, grad, stream)
             : launch_distill<T, D, kMaxDistillTop / DS_THREADS>(a, n, lse, grad, stream);
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
