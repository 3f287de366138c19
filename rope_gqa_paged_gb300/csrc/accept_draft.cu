// rra_accept_draft: which drafted tokens the target keeps, and the token that follows them.
//
// Token x_j, drafted with probability q_j(x_j), is kept while u_j q_j(x_j) < p_j(x_j), that is with
// probability min(1, p_j / q_j). The first token that is not kept, at n, is replaced by a draw from
// the normalised rest max(p_n - q_n, 0); when all are kept one more is drawn from p_n. So every token
// follows the target's distribution ("Transformer架构优化实战2026：注意力机制、KV Cache与推理加速完整指南"
// §五 names the method). The draw inverts the cumulative distribution: the lowest index v with
// r_0 + ... + r_v > u (r_0 + ... + r_(V-1)).
//
// Exactness: u q and p are compared as float64 products (24 x 24 bits fit 53). With every
// probability a whole number of units (2^-60 for float32; 2^-45 for bf16, whose 8 bits it holds
// exactly from 2^-38 up), r = p - min(p, q) is one too, and the sums are 64-bit integers. They do not
// depend on their order, so any split of the vocabulary over lanes, warps and CTAs gives the same
// token, and a float64 cumulative sum does unless u falls within rounding of a border.
// The integers come from float32 additions: x + 2 rounds x to a multiple of 2^-22 and holds that
// multiple in its low bits, so adding up the bit patterns adds up the integers; x minus the rounded
// part is exact and goes through the same step with the next smaller constant (unit 2^-45, then
// 2^-60). (The 64-bit conversion instruction runs at a small fraction of that: 64 rows of 128000
// float32 values 54 us with it, 36 us with 64-bit shifts, 33 us with these additions.)
//
// Bound: HBM (one row of p, and one of q where a token was rejected) for large batches, latency for
// small ones. One cluster of CTAs takes a sequence: each CTA decides n for itself (two dependent
// loads), sums its part of the vocabulary, and the CTAs exchange their sums through distributed
// shared memory: one launch, no workspace, no atomics. The CTA whose part holds the border looks for it again
// in the run of the warp that holds it, one to four vectors per thread, then in one thread's values. (64 rows of
// 128000 float32 values: 33 us with one warp going through the run 32 values a step, 19.3 with the run split
// among the warps until 256 values are left and 8 of them per lane, 19.1 so; 256 rows of 100003 bf16 values 29.8
// and 28.5. The sums without any search: 16.0 and 23.2.)
// Rows of any alignment load in aligned 16-byte vectors of p; where q's rows lie at another offset its
// two vectors are shifted together. Only vectors wholly inside the row are read so.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rra_device.cuh"
#include "rra_internal.h"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;   // 64 registers
constexpr int kMaxCluster = 16;
constexpr int kMaxGamma = 32;   // one lane of a warp per drafted token
constexpr int kScan = 4;        // most vectors per thread of the last search

struct AcceptArgs {
  const void* p;                // [B, gamma + 1, V] with these strides (elements)
  int64_t p_sb, p_st;
  const void* q;                // [B, gamma, V], or nullptr: q_j(x_j) = 1
  int64_t q_sb, q_st;
  const int32_t* tokens;        // [B, gamma]
  const int32_t* lens;          // [B] or nullptr (gamma)
  const float* u_accept;        // [B, gamma]
  const float* u_sample;        // [B]
  const int32_t* positions;     // [B] or nullptr
  int32_t* tokens_out;          // [B, gamma + 1]
  int32_t* n_accepted;          // [B]
  int32_t* positions_out;       // [B] or nullptr
  int gamma, V;
  int32_t* err;
};

// Rounding constants: kM[l] + x, |x| at most half the previous unit (at most 1 for the first), stays in
// one binade, whose unit is 2^-22, 2^-45, 2^-60.
__device__ constexpr float kM0 = 2.f, kM1 = 0x1.8p-22f, kM2 = 0x1.8p-37f;

// Two float32 additions in one instruction: x.lo + y.lo and x.hi + y.hi.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) | (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t z;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ uint64_t neg2(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint32_t both(uint64_t x) { return static_cast<uint32_t>(x) + static_cast<uint32_t>(x >> 32); }

// Sums of probabilities in units, as sums of bit patterns of the rounded values. At most 256 values go
// into one (the second part of a value is up to 2^22 units of 2^-45, the first up to 2^22 of 2^-22).
template <int LEVELS>
struct UnitSum {
  uint32_t a0 = 0, a1 = 0, a2 = 0;
  __device__ __forceinline__ void add(float x, float y) {
    const uint64_t xy = pack2(x, y);
    const uint64_t t0 = add2(xy, pack2(kM0, kM0));
    a0 += both(t0);
    const uint64_t l0 = add2(xy, neg2(add2(t0, pack2(-kM0, -kM0))));
    const uint64_t t1 = add2(l0, pack2(kM1, kM1));
    a1 += both(t1);
    if constexpr (LEVELS == 3) {
      const uint64_t l1 = add2(l0, neg2(add2(t1, pack2(-kM1, -kM1))));
      a2 += both(add2(l1, pack2(kM2, kM2)));
    }
  }
  // the sum of the `count` values added, in units of 2^-60
  __device__ __forceinline__ int64_t value(uint32_t count) const {
    const auto part = [&](uint32_t a, float m) {
      return static_cast<int64_t>(static_cast<int32_t>(a - count * __float_as_uint(m)));
    };
    int64_t s = (part(a0, kM0) << 38) + (part(a1, kM1) << 15);
    if constexpr (LEVELS == 3) s += part(a2, kM2);
    return s;
  }
};

template <typename T>
constexpr int kLevels = sizeof(T) == 4 ? 3 : 2;

template <typename T>
__device__ __forceinline__ int64_t units(float x) {
  UnitSum<kLevels<T>> s;
  s.add(x, 0.f);
  return s.value(2);
}

// NaN: 0; outside [0, 1]: the nearer end.
template <typename T>
__device__ __forceinline__ float load_prob(const T* p) {
  return __saturatef(Elem<T>::load(p));
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int64_t ld_cluster(const int64_t* local, uint32_t rank) {
  uint32_t addr;
  int64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// 16 bytes of p at element offset v of a row, as probabilities; values outside [0, V) are 0.
template <typename T, int E>
__device__ __forceinline__ void unpack_probs(const uint4& w, float (&x)[E]) {
  Elem<T>::unpack(w, x);
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __saturatef(x[e]);
}

// The 16 bytes that start `bytes` (a multiple of the element size) into the 32 of (a, b).
template <typename T>
__device__ __forceinline__ uint4 shift_vectors(const uint4& a, const uint4& b, uint32_t bytes) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (bytes & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (bytes & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// How q's row lies: there is none, at the offset of p's row within 16 bytes, at another one.
enum class Rows { kOne, kAligned, kShifted };

// One lane's part of the sum of p - min(p, q) over the vectors [n0, n1), all of them wholly inside the
// row (kShifted: the two vectors of q as well).
template <typename T, Rows ROWS>
__device__ __forceinline__ int64_t sum_vectors(const T* p, const T* q, int head, uint32_t off, int n0, int n1, int lane) {
  constexpr int E = Elem<T>::kPerChunk;
  constexpr int kBatch = ROWS == Rows::kShifted ? 2 : 4;  // vectors of each row in flight per lane (64 registers)
  constexpr int kVectors = 256 / E;                       // between two flushes of the 32-bit sums
  static_assert(kVectors % kBatch == 0, "whole batches");
  const uint4* pv = reinterpret_cast<const uint4*>(p - head);
  const uint4* qv = reinterpret_cast<const uint4*>(q - head - static_cast<int>(off));
  int64_t sum = 0;
  int n = n0 + lane;
  while (n < n1) {
    UnitSum<kLevels<T>> sp, sm;
    uint32_t count = 0;
    auto add = [&](const uint4& a, const uint4& b) {
      float x[E];
      unpack_probs<T, E>(a, x);
#pragma unroll
      for (int e = 0; e < E; e += 2) sp.add(x[e], x[e + 1]);
      if constexpr (ROWS != Rows::kOne) {
        float y[E];
        unpack_probs<T, E>(b, y);
#pragma unroll
        for (int e = 0; e < E; e += 2) sm.add(fminf(x[e], y[e]), fminf(x[e + 1], y[e + 1]));
      }
    };
    const int stop = min(n1, n + 32 * kVectors);
    for (; n + 32 * (kBatch - 1) < stop; n += 32 * kBatch, count += kBatch * E) {
      uint4 a[kBatch], b[kBatch], c[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        a[k] = pv[n + 32 * k];
        if constexpr (ROWS != Rows::kOne) b[k] = qv[n + 32 * k];
        if constexpr (ROWS == Rows::kShifted) c[k] = qv[n + 32 * k + 1];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if constexpr (ROWS == Rows::kShifted) b[k] = shift_vectors<T>(b[k], c[k], off * sizeof(T));
        add(a[k], b[k]);
      }
    }
    if constexpr (kBatch > 1) {
      for (; n < stop; n += 32, count += E) {
        const uint4 a = pv[n];
        uint4 b;
        if constexpr (ROWS != Rows::kOne) b = qv[n];
        if constexpr (ROWS == Rows::kShifted) b = shift_vectors<T>(b, qv[n + 1], off * sizeof(T));
        add(a, b);
      }
    }
    sum += sp.value(count);
    if constexpr (ROWS != Rows::kOne) sum -= sm.value(count);
  }
  return sum;
}

// Vector n of a row holds its elements n E - head .. n E - head + E - 1, 16-byte aligned in p; those of
// [lo, hi) lie wholly inside the row, in q as well, whose vectors have them from element `off` on.
template <typename T>
struct Layout {
  int head, lo, hi;
  uint32_t off;
  __device__ __forceinline__ Layout(const T* p, const T* q, int V) {
    constexpr int E = Elem<T>::kPerChunk;
    head = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    off = q == nullptr ? 0u
                       : static_cast<uint32_t>(((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) & 15) /
                                               sizeof(T));
    // n E - head >= 0 (>= off) and n E - head + E (- off + 2 E) <= V
    lo = (head + static_cast<int>(off) + E - 1) / E;
    hi = max((V + head - (off != 0 ? E - static_cast<int>(off) : 0)) / E, 0);
  }
};

// Sum of p - min(p, q) over vector n of a row; element `skip` counts as 0 (there is no q then).
template <typename T>
__device__ __forceinline__ int64_t vector_rest(const T* p, const T* q, int V, const Layout<T>& at, int n, int skip) {
  constexpr int E = Elem<T>::kPerChunk;
  const int v0 = n * E - at.head;
  float x[E], y[E];
  if (n >= at.lo && n < at.hi) {
    unpack_probs<T, E>(*reinterpret_cast<const uint4*>(p + v0), x);
    if (q != nullptr) {
      const uint4* qv = reinterpret_cast<const uint4*>(q + v0 - static_cast<int>(at.off));
      unpack_probs<T, E>(at.off != 0 ? shift_vectors<T>(qv[0], qv[1], at.off * sizeof(T)) : qv[0], y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = v0 + e >= 0 && v0 + e < V;
      x[e] = in ? load_prob(p + v0 + e) : 0.f;
      y[e] = in && q != nullptr ? load_prob(q + v0 + e) : 0.f;
    }
  }
  UnitSum<kLevels<T>> sp, sm;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if (v0 + e == skip) x[e] = 0.f;
    if (v0 + e + 1 == skip) x[e + 1] = 0.f;
    sp.add(x[e], x[e + 1]);
    if (q != nullptr) sm.add(fminf(x[e], y[e]), fminf(x[e + 1], y[e + 1]));
  }
  return sp.value(E) - (q != nullptr ? sm.value(E) : 0);
}

// One lane's part of the sum of p - min(p, q) over the vectors [n0, n1) of a row, in units of 2^-60; q may be
// nullptr (the sum of p). The vectors that reach over the row's ends go value by value.
template <typename T>
__device__ __forceinline__ int64_t sum_rest(const T* p, const T* q, int V, int n0, int n1, int lane) {
  constexpr int E = Elem<T>::kPerChunk;
  const Layout<T> at(p, q, V);
  const int head = at.head, i0 = min(max(n0, at.lo), n1), i1 = max(min(n1, at.hi), i0);
  const uint32_t off = at.off;
  const bool shifted = off != 0;
  int64_t sum = 0;
  if (q == nullptr)
    sum = sum_vectors<T, Rows::kOne>(p, q, head, 0, i0, i1, lane);
  else if (!shifted)
    sum = sum_vectors<T, Rows::kAligned>(p, q, head, 0, i0, i1, lane);
  else
    sum = sum_vectors<T, Rows::kShifted>(p, q, head, off, i0, i1, lane);
  const int before = (i0 - n0) * E, ends = before + (n1 - i1) * E;  // values of the other vectors
  for (int i = lane; i < ends; i += 32) {
    const int v = (i < before ? n0 * E + i : i1 * E + i - before) - head;
    if (v >= 0 && v < V) {
      const float x = load_prob(p + v);
      sum += units<T>(x);
      if (q != nullptr) sum -= units<T>(fminf(x, load_prob(q + v)));
    }
  }
  return sum;
}

struct Shared {
  int64_t warp_sums[2][kWarps], cta_sum[2], scan_sums[kWarps], hit_before;
  int hit;
};

// This warp's sum over the vectors [n0, n1), to every lane.
template <typename T>
__device__ __forceinline__ int64_t run_sum(const T* p, const T* q, int V, int skip, int head, int n0, int n1, int lane) {
  constexpr int E = Elem<T>::kPerChunk;
  int64_t s = warp_sum(sum_rest<T>(p, q, V, n0, n1, lane));
  if (skip >= 0 && skip >= n0 * E - head && skip < n1 * E - head) s -= units<T>(load_prob(p + skip));
  return s;
}

// The lowest token whose inclusive sum exceeds `border`, by the CTA whose part holds it: its warps' runs of
// `step` vectors start at f0 and end before f1, `before` is the sum of what precedes them. The run of the warp that
// holds the border is split among the warps until a thread has at most kScan vectors; the threads' sums then
// give the thread, and one warp looks through its values. (Its own function, so that the sums' loop keeps the
// registers to itself.)
template <typename T>
__device__ __noinline__ void find_border(const T* p, const T* q, int V, int skip, int f0, int step, int f1, int64_t before,
                                         int64_t border, int32_t* token_out, Shared& sh) {
  constexpr int E = Elem<T>::kPerChunk;
  static_assert(kScan * E <= 32, "a lane per value of a thread's vectors");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Layout<T> at(p, q, V);
  for (int level = 0;; ++level) {
    // (sums are never negative, so the first warp whose inclusive sum exceeds the border holds it)
    const int64_t* sums = sh.warp_sums[level & 1];
    int w = 0;
    for (; w < kWarps - 1 && border >= before + sums[w]; ++w) before += sums[w];
    f0 = min(f0 + w * step, f1);
    f1 = min(f0 + step, f1);
    if (f1 - f0 <= kScan * kThreads) break;
    step = (f1 - f0 + kWarps - 1) / kWarps;
    const int n0 = min(f0 + warp * step, f1);
    const int64_t s = run_sum<T>(p, q, V, skip, at.head, n0, min(n0 + step, f1), lane);
    if (lane == 0) sh.warp_sums[(level & 1) ^ 1][warp] = s;
    __syncthreads();
  }
  const int c = (f1 - f0 + kThreads - 1) / kThreads;  // consecutive vectors per thread
  const int m0 = f0 + static_cast<int>(threadIdx.x) * c, m1 = min(m0 + c, f1);
  int64_t mine = 0;
  for (int n = m0; n < m1; ++n) mine += vector_rest<T>(p, q, V, at, n, skip);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sh.scan_sums[warp] = incl;
  if (threadIdx.x == 0) sh.hit = -1;
  __syncthreads();
  int64_t excl = before + incl - mine;
  for (int w = 0; w < warp; ++w) excl += sh.scan_sums[w];
  if (excl <= border && border < excl + mine) {
    sh.hit = m0;
    sh.hit_before = excl;
  }
  __syncthreads();
  if (warp == 0 && sh.hit >= 0) {
    const int v = sh.hit * E - at.head + lane;
    int64_t val = 0;
    if (lane < c * E && v >= 0 && v < V && v != skip) {
      const float pv = load_prob(p + v);
      val = units<T>(pv) - (q != nullptr ? units<T>(fminf(pv, load_prob(q + v))) : 0);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, val, d);
      if (lane >= d) val += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, sh.hit_before + val > border);
    if (over != 0 && lane == __ffs(over) - 1) *token_out = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) accept_draft_kernel(const AcceptArgs a) {
  constexpr int E = Elem<T>::kPerChunk;
  __shared__ Shared sh;
  const int b = blockIdx.y, C = gridDim.x;
  const int rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gamma = a.gamma, V = a.V;

  pdl_wait();
  pdl_launch_dependents();
  const bool scribe = rank == 0 && warp == 0;  // the warp that writes what does not depend on the draw

  // ---- how many tokens are kept (every warp finds it for itself: lane j has token j)
  int len = a.lens != nullptr ? a.lens[b] : gamma;
  const float u_last = a.u_sample[b];
  int x = -1;
  float u = 0.f;
  if (lane < gamma) {
    x = a.tokens[static_cast<size_t>(b) * gamma + lane];
    u = a.u_accept[static_cast<size_t>(b) * gamma + lane];
  }
  if (len < 0 || len > gamma) {
    if (scribe && lane == 0) flag_error(a.err, RRA_ERR_SEQ_LEN);
    len = min(max(len, 0), gamma);
  }
  const T* prow = static_cast<const T*>(a.p) + b * a.p_sb;
  const T* qrow = static_cast<const T*>(a.q) + b * a.q_sb;
  bool keep = false;
  if (lane < len) {
    if (x < 0 || x >= V) {
      if (scribe) flag_error(a.err, RRA_ERR_TOKEN);
    } else {
      const float px = load_prob(prow + lane * a.p_st + x);
      const float qx = a.q != nullptr ? load_prob(qrow + lane * a.q_st + x) : 1.f;
      keep = static_cast<double>(u) * static_cast<double>(qx) < static_cast<double>(px);
    }
  }
  const uint32_t dropped = ~__ballot_sync(0xffffffffu, keep);
  const int n = min(dropped != 0 ? __ffs(dropped) - 1 : 32, len);
  const int at = __shfl_sync(0xffffffffu, x, n & 31);  // the rejected token (n < len)
  const T* p = prow + n * a.p_st;
  const T* q = n < len && a.q != nullptr ? qrow + n * a.q_st : nullptr;
  // without the drafter's probabilities the rejected token alone is taken out of p
  int skip = n < len && a.q == nullptr && at >= 0 && at < V ? at : -1;
  if (scribe) {  // (V - 1 until the draw replaces it, behind the cluster's barrier: always a token)
    for (int j = lane; j <= gamma; j += 32)
      a.tokens_out[static_cast<size_t>(b) * (gamma + 1) + j] = j < n ? x : j == n ? V - 1 : -1;
    if (lane == 0) {
      a.n_accepted[b] = n;
      if (a.positions_out != nullptr) a.positions_out[b] = a.positions[b] + n + 1;
    }
  }

  // ---- sums of r over this warp's run of the vocabulary, the CTA's and the sequence's
  const int head = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
  const int vecs = (V + head + E - 1) / E;
  const int per_warp = (vecs + C * kWarps - 1) / (C * kWarps);
  int64_t total, before, own;
  // a second time, over p itself, where nothing is left (p <= q everywhere, by rounding)
  for (int pass = 0;; ++pass) {
    const int n0 = min((rank * kWarps + warp) * per_warp, vecs);
    const int64_t run = run_sum<T>(p, q, V, skip, head, n0, min(n0 + per_warp, vecs), lane);
    if (lane == 0) sh.warp_sums[0][warp] = run;
    __syncthreads();
    if (threadIdx.x == 0) {
      int64_t s = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sh.warp_sums[0][w];
      sh.cta_sum[pass] = s;
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    const int64_t c = lane < C ? ld_cluster(&sh.cta_sum[pass], lane) : 0;
    total = warp_sum(c);
    before = warp_sum(lane < rank ? c : 0);
    own = __shfl_sync(0xffffffffu, c, rank);
    if (total > 0 || pass == 1) break;
    q = nullptr;
    skip = -1;
  }
  cluster_arrive();  // this CTA has read the others' sums

  // ---- the border u * total, and the CTA whose part holds it
  if (total <= 0) {
    if (scribe && lane == 0) flag_error(a.err, RRA_ERR_PROBS);
  } else {
    const float uc = fminf(fmaxf(u_last, 0.f), 1.f - 0x1p-24f);
    const int64_t border = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(total), __float2ull_rz(uc * 0x1p64f)));
    if (before <= border && border < before + own)
      find_border<T>(p, q, V, skip, rank * kWarps * per_warp, per_warp, vecs, before, border,
                     a.tokens_out + static_cast<size_t>(b) * (gamma + 1) + n, sh);
  }
  cluster_wait();  // no CTA's sums go away while another may still read them
}

template <typename T>
cudaError_t launch_accept(const AcceptArgs& a, int B, int clusters, cudaStream_t stream) {
  static int done[64] = {0};
  auto kern = accept_draft_kernel<T>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {  // clusters of 16 CTAs are opt-in
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clusters, B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = clusters;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace
}  // namespace rra

extern "C" int rra_accept_draft(const void* target_probs, int64_t target_stride_b, int64_t target_stride_t,
                                const void* draft_probs, int64_t draft_stride_b, int64_t draft_stride_t,
                                const int32_t* draft_tokens, const int32_t* draft_lens, const float* u_accept,
                                const float* u_sample, const int32_t* positions, int32_t* tokens_out,
                                int32_t* n_accepted, int32_t* positions_out, int B, int gamma, int V, rra_dtype dt,
                                int32_t* err_flag, void* stream) {
  if (dt != RRA_F32 && dt != RRA_BF16) return RRA_EUNSUPPORTED;
  if (B < 0 || gamma < 1 || V < 1) return RRA_EINVAL;
  if (gamma > rra::kMaxGamma) return RRA_EUNSUPPORTED;
  if (B > 65535 || V > (1 << 30)) return RRA_ERANGE;
  if (B == 0) return RRA_OK;
  if (!target_probs || !draft_tokens || !u_accept || !u_sample || !tokens_out || !n_accepted) return RRA_EINVAL;
  if (positions_out != nullptr && positions == nullptr) return RRA_EINVAL;
  const uintptr_t mask = dt == RRA_BF16 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(target_probs) & mask) || (reinterpret_cast<uintptr_t>(draft_probs) & mask))
    return RRA_EINVAL;
  if (target_stride_b < 0 || target_stride_t < 0 || draft_stride_b < 0 || draft_stride_t < 0) return RRA_EINVAL;
  // A sequence's inputs are read by every CTA of its cluster, its outputs written by one of them: none may lie over another
  // array (positions_out over positions, element on element, is one thread's).
  {
    struct Range {
      const void* p;
      size_t n;
    };
    const size_t b = size_t(B) * 4, bg = b * gamma;
    const Range outs[] = {{tokens_out, b + bg}, {n_accepted, b}, {positions_out, b}};
    const Range ins[] = {{draft_tokens, bg}, {u_accept, bg}, {draft_lens, b}, {u_sample, b}, {positions, b}};
    const auto meet = [](const Range& x, const Range& y) {
      const uintptr_t i = reinterpret_cast<uintptr_t>(x.p), j = reinterpret_cast<uintptr_t>(y.p);
      return i != 0 && j != 0 && i < j + y.n && j < i + x.n;
    };
    for (int i = 0; i < 3; ++i) {
      for (int j = 0; j < i; ++j)
        if (meet(outs[i], outs[j])) return RRA_EINVAL;
      for (const Range& in : ins)
        if (meet(outs[i], in) && !(i == 2 && in.p == positions && positions_out == positions)) return RRA_EINVAL;
    }
  }
  rra::AcceptArgs a{};
  a.p = target_probs;
  a.p_sb = target_stride_b;
  a.p_st = target_stride_t;
  a.q = draft_probs;
  a.q_sb = draft_stride_b;
  a.q_st = draft_stride_t;
  a.tokens = draft_tokens;
  a.lens = draft_lens;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.positions = positions;
  a.tokens_out = tokens_out;
  a.n_accepted = n_accepted;
  a.positions_out = positions_out;
  a.gamma = gamma;
  a.V = V;
  a.err = err_flag;
  // CTAs per sequence: 16 while they leave every CTA an SM of its own (one sequence of 32000 float32
  // values: 5.6 us, 1.5 us more with 8). Otherwise the largest power of two, up to 8, with which the whole grid is
  // resident at once (64 x 128000 float32: 19.1 us with 8, 4.5 more with 4, 8 more with 16, whose clusters wait
  // for 16 free places of one GPC; 256 x 100003 bf16: 28.5 us with 2, 8 more with 8 in four turns; sizes between
  // the powers gain nothing: 100 x 128000 float32 28.7 us with 4, 28.9 with 6).
  const int64_t sms = std::max(1, rra::current_sm_count());
  int clusters = int64_t(B) * rra::kMaxCluster <= sms ? rra::kMaxCluster : 8;
  while (clusters > 1 && int64_t(clusters) * B > rra::kCtasPerSm * sms) clusters /= 2;
  const cudaError_t e = dt == RRA_BF16
                            ? rra::launch_accept<__nv_bfloat16>(a, B, clusters, static_cast<cudaStream_t>(stream))
                            : rra::launch_accept<float>(a, B, clusters, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return RRA_OK;
  rra::record_cuda_error(e, "accept_draft launch");
  return RRA_ECUDA;
}
