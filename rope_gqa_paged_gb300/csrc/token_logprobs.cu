// rra_token_logprobs: log probabilities of given tokens, the entropy and the most likely tokens of rows of logits.
//
// With m the largest logit of a row, S = sum e^(x - m) and U = sum (x - m) e^(x - m):
//   log p(v) = x_v - m - ln S,   H = -sum p ln p = ln S - U / S.
// One pass keeps (m, S, U) of what a thread has seen, in float32 and units of log2; when the maximum moves by d,
// S' = 2^d S and U' = 2^d (U + d S). Logits of -inf (masked) add nothing; a row that holds a NaN or +inf, or nothing
// above -inf, has no distribution.
//
// The most likely tokens come from a second look at few values. A thread keeps the largest value of every batch (or few
// batches) of its vectors. A bound that at least k values of the CTA reach (common_bound) is no larger than the k-th largest;
// whatever reaches it lies in batches whose maxima do. Those are read again, what reaches the bound goes to the
// cluster's first CTA (about 24 values per CTA for k = 20), and the k largest are sorted by counting, for each, how many are larger.
// Where too many reach it (equal values, above all -inf; large values all with few threads) a finer bound on (value,
// index) takes over, and k searches one after the other where that does not help either.
//
// Bound: HBM (each logit read once) for many rows: 4000 x 100003 float32 with 8 alternatives 250 us (6.4 TB/s; 226 without them),
// 1024 x 128000 bf16 51.5 us (5.1 TB/s: 1.7 rows per resident CTA, issue slots half used). Latency for few: 1 x
// 32000 float32 with 5 alternatives 5.0 us, 1 x 128000 bf16 with 20 6.0 us. A feeding warp copies batches of 16 KB into a ring
// (fed by a reading thread: 302 us instead of 256 for the first); a row's parts are joined through distributed shared
// memory: one launch, no workspace; the atomics only hand out places in lists that are sorted afterwards, so results do
// not depend on their order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rra_device.cuh"
#include "rra_internal.h"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kMaxCluster = 16;
constexpr int kMaxTop = 32;
constexpr int kMaxTokens = 32;   // given tokens per row: a lane each
constexpr int kBatch = 4;        // vectors in flight per thread
constexpr int kStageBytes = kThreads * kBatch * 16;
constexpr int kRing = 2;         // batches of all threads on their way
constexpr int kEntries = 16;     // batch maxima that a thread keeps, as bf16 (rounded up)
constexpr int kMaxFound = 1024;  // values of a row that reach the bound; more of a CTA go the long way
constexpr int kMaxKeys = 512;    // of a CTA that reach the bound there; more go the longest way

struct LogprobArgs {
  const void* logits;            // [B, N, V] with these strides (elements)
  int64_t sb, st;
  const int32_t* tokens;         // [B, N, T] or nullptr
  float* logprobs;               // [B, N, T]
  float* entropy;                // [B, N] or nullptr
  float* top_logprobs;           // [B, N, top_k]
  int32_t* top_tokens;
  int64_t rows;
  int N, V, T, top_k;
  int32_t* err;
};

__device__ __forceinline__ float ex2(float x) {  // 2^x on the special-function unit (2^-inf = 0)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 operations in one instruction, on pairs (lo, hi).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) | (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}
__device__ __forceinline__ float lo2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t z;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t z;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t c) {
  uint64_t z;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(x), "l"(y), "l"(c));
  return z;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}

// What a type's vectors are worked on with: their maximum, and their values no lower than a bound.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);  // -inf
  }
  static __device__ __forceinline__ float max_of(const uint4& w, float m) {
    return max_nan(max_nan(max_nan(m, __uint_as_float(w.x)), max_nan(__uint_as_float(w.y), __uint_as_float(w.z))),
                   __uint_as_float(w.w));
  }
  static constexpr int kPairs = 2;
  using Bound = float;
  static __device__ __forceinline__ Bound make_bound(float b) { return b; }
  static __device__ __forceinline__ void clamped(const uint4& w, Bound bound, uint64_t (&x)[2]) {
    x[0] = pack2(max_nan(__uint_as_float(w.x), bound), max_nan(__uint_as_float(w.y), bound));
    x[1] = pack2(max_nan(__uint_as_float(w.z), bound), max_nan(__uint_as_float(w.w), bound));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __forceinline__ float max_of(const uint4& w, float m) {
    const uint32_t x = max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w));
    return max_nan(m, max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)));
  }
  static constexpr int kPairs = 4;
  using Bound = uint32_t;  // twice
  static __device__ __forceinline__ Bound make_bound(float b) {
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rd(b))) * 0x10001u;
  }
  static __device__ __forceinline__ void clamped(const uint4& w, Bound bb, uint64_t (&x)[4]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = max_nan_bf16x2(v[i], bb);
      x[i] = pack2(__uint_as_float(c << 16), __uint_as_float(c & 0xffff0000u));
    }
  }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = -1000.f;  // a power of two that is 0, and no infinity to multiply 0 with

// (m, S, U) of a set of logits, S and U in units of 2^(m log2 e); U's factors in log2.
struct Stats {
  float m, s, u;
  __device__ __forceinline__ void move_to(float to) {
    const float d = fmaxf((m - to) * kLog2e, kFar), f = ex2(d);  // (-inf to -inf: NaN, which fmaxf drops; s is 0)
    u = f * fmaf(d, s, u);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void add(float x) {  // m is at least x
    const float d = (x - (m == -INFINITY ? 0.f : m)) * kLog2e, e = ex2(d);
    s += e;
    u = fmaf(fmaxf(d, kFar), e, u);
  }
};

// The order of the logits, the largest key first: value, then the lower index. 0 is below every logit's.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 counts as 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ Key make_key(float x, int index) {
  return (static_cast<Key>(ordered(x)) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ int key_index(Key k) { return static_cast<int>(~static_cast<uint32_t>(k)); }
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t b = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ Key warp_max(Key k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<Key>(hi) << 32) | lo;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_addr(const void* local, uint32_t rank) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(rank));
  return addr;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, Key v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The warp's statistics together, the same in every lane (the sums are over pairs, so their order does not show).
__device__ __forceinline__ Stats join_warp(Stats s) {
  const uint32_t m = __reduce_max_sync(0xffffffffu, ordered(s.m));  // (a NaN counts as the largest)
  s.move_to(__uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s.s += __shfl_xor_sync(0xffffffffu, s.s, d);
    s.u += __shfl_xor_sync(0xffffffffu, s.u, d);
  }
  return s;
}

struct Shared {
  Stats stats[kMaxCluster * kWarps];              // of every CTA's warps (in the first CTA)
  alignas(16) uint32_t groups[kThreads / 4];      // the largest values of groups of four threads
  uint32_t bound;
  Key top[kMaxTop];                               // this CTA's, sorted; 0 past the end
  Key best[kWarps];
  uint64_t full[kRing], empty[kRing];
  int counts[kMaxCluster];                        // keys that the CTAs found (in the first CTA)
  int count, kept;
};

// Dynamic shared memory: the ring of vectors on their way in, the batch maxima, the keys found here and in all CTAs.
constexpr int kOffMaxima = kRing * kStageBytes;
constexpr int kOffFound = kOffMaxima + kEntries * kThreads * 2;
constexpr int kOffAll = kOffFound + kMaxKeys * 8;  // (in the first CTA: kMaxFound / C places for each CTA)
constexpr int kSmemBytes = kOffAll + kMaxFound * 8;
static_assert(kCtasPerSm * (kSmemBytes + sizeof(Shared) + 1024) <= 228 * 1024, "shared memory of the SM");
static_assert(kMaxFound >= kMaxCluster * kMaxTop, "every CTA's k largest fit");

// A thread's part of the row: vectors v0 + thread, + kThreads, ... below v1, whose first element is head + E v, and at
// most one element in front of or behind the vectors. kBatch of its vectors are a batch; `per_entry` batches share an
// entry of the maxima. `in`: the vectors from v0 on, in shared memory where they all are still there.
template <typename T>
struct Part {
  static constexpr int E = Elem<T>::kPerChunk;
  const T* row;
  const uint4* in;
  int head, v0, v1, single;       // single: its index, -1: none
  int per_entry;
  template <typename F>
  __device__ __forceinline__ void vector(int v, const uint4& w, F&& f) const {  // f(value, index)
    float x[E];
    Elem<T>::unpack(w, x);
#pragma unroll
    for (int e = 0; e < E; ++e) f(x[e], head + E * v + e);
  }
  // f of the values of entry e's vectors of this thread, but for vectors that hold nothing as large as `bound`.
  template <typename F>
  __device__ __forceinline__ void entry(int e, float bound, F&& f) const {
    constexpr int kLoads = 2 * kBatch;
    const int first = v0 + e * per_entry * kBatch * kThreads + static_cast<int>(threadIdx.x);
    const int end = min(v1, first + per_entry * kBatch * kThreads);
    for (int v = first; v < end; v += kLoads * kThreads) {
      uint4 w[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) w[i] = v + i * kThreads < end ? in[v + i * kThreads - v0] : Vec<T>::none();
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) hits |= !(Vec<T>::max_of(w[i], -INFINITY) < bound) && v + i * kThreads < end ? 1u << i : 0u;
      for (; hits != 0; hits &= hits - 1) {
        const int at = v + (__ffs(hits) - 1) * kThreads;
        vector(at, in[at - v0], f);  // (read again: picked out of registers it takes more of them than there are)
      }
    }
  }
  __device__ __forceinline__ float single_value() const { return Elem<T>::load(row + single); }
};

// The barrier of the warps that read (the one that feeds the ring leaves by itself).
__device__ __forceinline__ void sync_readers() { named_barrier_sync(1, kThreads); }

// The CTA's k largest keys by taking the largest below the last one, k times.
template <typename T>
__device__ __noinline__ void top_slowly(const Part<T> part, int k, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Key last = ~Key(0);
  for (int r = 0; r < k; ++r) {
    Key mine = 0;
    auto look = [&](float x, int i) {
      const Key key = make_key(x, i);
      if (key < last && key > mine) mine = key;
    };
    for (int e = 0; e < kEntries; ++e) part.entry(e, -INFINITY, look);
    if (part.single >= 0) look(part.single_value(), part.single);
    mine = warp_max(mine);
    if (lane == 0) sh.best[warp] = mine;
    sync_readers();
    last = 0;
    for (int w = 0; w < kWarps; ++w) last = max(last, sh.best[w]);
    if (threadIdx.x == 0) sh.top[r] = last;
    sync_readers();
  }
}

// A bound that at least k of the values that the threads hold (0: none) reach, sh.bound as it was if there are not k: the k-th largest
// of the maxima of groups of four threads. (The k-th largest of all is no smaller; of values in no order about
// 64 (1/64 + 1/63 + ... , k terms) reach it: 24 for k = 20.) Every thread ranks one maximum against a quarter of the
// others.
constexpr int kGroups = kThreads / 4;
__device__ __forceinline__ uint32_t common_bound(uint32_t x, int k, Shared& sh) {
  const int t = threadIdx.x;
  x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
  x = max(x, __shfl_xor_sync(0xffffffffu, x, 2));
  if (t % 4 == 0) sh.groups[t / 4] = x;
  sync_readers();
  int larger = 0, as_large = 0;
#pragma unroll
  for (int j = 0; j < kGroups / 4; j += 4) {
    const uint4 y = *reinterpret_cast<const uint4*>(&sh.groups[t % 4 * (kGroups / 4) + j]);
    larger += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
    as_large += (y.x >= x) + (y.y >= x) + (y.z >= x) + (y.w >= x);
  }
  int both = larger | as_large << 16;
  both += __shfl_xor_sync(0xffffffffu, both, 1);
  both += __shfl_xor_sync(0xffffffffu, both, 2);
  if ((both & 0xffff) < k && both >> 16 >= k) sh.bound = x;  // (equal ones write the same)
  sync_readers();
  return sh.bound;
}

// This CTA's k largest keys, sorted into sh.top, where too many values reach a bound on the value alone: equal ones (ruled out
// tokens, a row of one value), or an order that puts large ones with few threads. First by a bound on keys, which
// differ by their index.
template <typename T>
__device__ __noinline__ void top_of_many(const Part<T> part, const __nv_bfloat16* maxima, float largest, bool some, int k, Key* found, Shared& sh) {
  const int per_warp = min(kMaxTop, 2 * ((k + kWarps - 1) / kWarps));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = threadIdx.x;
  Key mine = 0;  // the thread's largest
  for (int e = 0; some && e < kEntries; ++e) {
    if (part.v0 + e * part.per_entry * kBatch * kThreads + t >= part.v1) break;
    if (static_cast<uint32_t>(mine >> 32) == ordered(largest)) break;  // (the first entry that has it holds its lowest index)
    if (ordered(__bfloat162float(maxima[e * kThreads + t])) >= ordered(largest))
      part.entry(e, largest, [&](float x, int index) { mine = max(mine, make_key(x, index)); });
  }
  if (part.single >= 0) mine = max(mine, make_key(part.single_value(), part.single));
  Key left = mine;
  Key* held = found;  // the largest keys of each warp's threads
  static_assert(kMaxKeys >= kWarps * kMaxTop, "they fit");
  sync_readers();
  for (int i = 0; i < per_warp; ++i) {
    const Key top = warp_max(left);
    if (lane == 0) held[warp * per_warp + i] = top;
    if (left == top) left = 0;  // (keys differ, but for 0)
  }
  if (t == 0) sh.count = 0;
  sync_readers();
  Key bound = 0;
  for (int i = lane; i < kWarps * per_warp; i += 32) {
    int larger = 0;
    for (int j = 0; j < kWarps * per_warp; ++j) larger += held[j] > held[i];
    if (larger == k - 1) bound = held[i];
  }
  bound = warp_max(bound);
  sync_readers();
  auto put = [&](float x, int i) {
    const Key key = make_key(x, i);
    if (key >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kMaxKeys) found[at] = key;
    }
  };
  if (mine != 0 && mine >= bound) {
    for (int e = 0; some && e < kEntries && part.v0 + e * part.per_entry * kBatch * kThreads + t < part.v1; ++e)
      if (ordered(__bfloat162float(maxima[e * kThreads + t])) >= static_cast<uint32_t>(bound >> 32)) part.entry(e, key_value(bound), put);
    if (part.single >= 0) put(part.single_value(), part.single);
  }
  if (t < k) sh.top[t] = 0;
  sync_readers();
  const int n = sh.count;
  if (n > kMaxKeys) {
    top_slowly(part, k, sh);
  } else {
    for (int i = t; i < n; i += kThreads) {
      const Key key = found[i];
      int larger = 0;
      for (int j = 0; j < n; ++j) larger += found[j] > key;
      if (larger < k) sh.top[larger] = key;
    }
  }
  sync_readers();
}

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, kCtasPerSm) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int E = Elem<T>::kPerChunk;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  __nv_bfloat16* maxima = reinterpret_cast<__nv_bfloat16*>(smem + kOffMaxima);  // [kEntries][kThreads]
  Key* found = reinterpret_cast<Key*>(smem + kOffFound);
  Key* all = reinterpret_cast<Key*>(smem + kOffAll);
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;  // row b N + t
  if (r >= a.rows) return;  // (the whole cluster)
  const int C = gridDim.x, rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kWarps);
    }
    sh.count = sh.kept = 0;
    sh.bound = 0;
    fence_barrier_init();
  }
  cluster_arrive();  // (waited for before the first CTA's memory is written to)
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = r / a.N;
  const T* row = static_cast<const T*>(a.logits) + b * a.sb + (r - b * a.N) * a.st;
  const int V = a.V, k = a.top_k;

  Part<T> part;
  part.row = row;
  part.head = min(V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
  const uint4* vec = reinterpret_cast<const uint4*>(row + part.head);
  const int vecs = (V - part.head) / E, tail = V - part.head - vecs * E;
  const int per = (vecs + C - 1) / C;
  part.v0 = min(rank * per, vecs);
  part.v1 = min(part.v0 + per, vecs);
  const int batches = (part.v1 - part.v0 + kBatch * kThreads - 1) / (kBatch * kThreads);
  part.per_entry = (batches + kEntries - 1) / kEntries;
  part.single = -1;
  part.in = batches <= kRing ? reinterpret_cast<const uint4*>(smem) : vec + part.v0;
  const bool ringed = batches > 1;  // (one batch is loaded as it is: 4000 x 1000 bf16 37 us, 42 through the ring)
  __syncthreads();
  if (warp == kWarps) {  // the warp that feeds the ring: one copy per batch
    if (ringed && lane == 0) {
      int n = 0;
      for (; n < batches; ++n) {
        const int s = n % kRing;
        if (n >= kRing && !mbar_wait(&sh.empty[s], ((n / kRing) & 1) ^ 1)) {
          flag_error(a.err, RRA_ERR_TIMEOUT);
          break;
        }
        const int v = part.v0 + n * kBatch * kThreads;
        const uint32_t bytes = 16u * static_cast<uint32_t>(min(kBatch * kThreads, part.v1 - v));
        mbar_arrive_expect_tx(&sh.full[s], bytes);
        bulk_g2s(smem + s * kStageBytes, vec + v, bytes, &sh.full[s]);
      }
      for (int i = max(n - kRing, 0); i < n; ++i) mbar_wait(&sh.full[i % kRing], (i / kRing) & 1);  // none still on its way
    }
    __syncwarp();
    cluster_wait();
    return;  // (barriers count the threads that are left)
  }

  const int t = threadIdx.x;
  // the given tokens' logits
  int token = -1;
  float x_token = 0.f;
  const bool asks = rank == 0 && warp == 1 && lane < a.T;
  if (asks) {
    token = a.tokens[r * a.T + lane];
    if (token >= 0 && token < V) x_token = Elem<T>::load(row + token);
  }
  part.single = rank != 0 ? -1 : t < part.head ? t : t >= E && t - E < tail ? V - tail + t - E : -1;

  // ---- (m, S, U), one pass
  Stats st{-INFINITY, 0.f, 0.f};
  int entry = t, in_entry = 0;
  bool plain = true;
  uint64_t minus_m = 0;
  typename Vec<T>::Bound bound{};
  auto batch = [&](const uint4 (&w)[kBatch]) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) mx = Vec<T>::max_of(w[i], mx);
    if (k > 0) {
      maxima[entry] = __float2bfloat16_ru(in_entry == 0 ? mx : max_nan(mx, __bfloat162float(maxima[entry])));
      if (++in_entry == part.per_entry) {
        in_entry = 0;
        entry += kThreads;
      }
    }
    if (!(mx <= st.m)) {  // (a NaN too: it makes m and the sums NaN)
      st.move_to(mx);
      // A logit far below m adds 0 to both sums, wherever it is: held at a bound, so that -inf is no infinity to
      // multiply 0 with. (e^-150 is 0 in float32; |m| / 16 so that the bound is another number than m.)
      const float low = mx - fmaf(fabsf(mx), 0x1p-4f, 150.f);
      plain = !(low > -1e38f);
      bound = Vec<T>::make_bound(low);
      minus_m = pack2(-mx, -mx);
    }
    if (!plain) {
      const uint64_t log2e = pack2(kLog2e, kLog2e);
      uint64_t s2[2] = {0, 0}, u2[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        uint64_t x[Vec<T>::kPairs];
        Vec<T>::clamped(w[i], bound, x);
#pragma unroll
        for (int p = 0; p < Vec<T>::kPairs; ++p) {
          const uint64_t d = mul2(add2(x[p], minus_m), log2e), e = pack2(ex2(lo2(d)), ex2(hi2(d)));
          s2[p & 1] = add2(s2[p & 1], e);
          u2[p & 1] = fma2(d, e, u2[p & 1]);
        }
      }
      const uint64_t s = add2(s2[0], s2[1]), u = add2(u2[0], u2[1]);
      st.s += lo2(s) + hi2(s);
      st.u += lo2(u) + hi2(u);
    } else {  // (nothing but -inf, or values near the type's lowest, so far; or a NaN)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[E];
        Elem<T>::unpack(w[i], x);
#pragma unroll
        for (int e = 0; e < E; ++e) st.add(x[e]);
      }
    }
  };
  const bool some = part.v0 + t < part.v1;
  if (ringed) {
    int n = 0;
    for (; n < batches; ++n) {
      const int s = n % kRing, v = part.v0 + n * kBatch * kThreads + t;
      if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[s], (n / kRing) & 1))) break;
      const uint4* in = reinterpret_cast<const uint4*>(smem + s * kStageBytes) + t;
      uint4 w[kBatch];
      if (n + 1 < batches) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = in[i * kThreads];
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = v + i * kThreads < part.v1 ? in[i * kThreads] : Vec<T>::none();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
      batch(w);
    }
    if (n < batches) flag_error(a.err, RRA_ERR_TIMEOUT);
  } else if (some) {
    uint4 w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w[i] = part.v0 + t + i * kThreads < part.v1 ? vec[part.v0 + t + i * kThreads] : Vec<T>::none();
    if (k > 0) {  // (for a second look)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) reinterpret_cast<uint4*>(smem)[t + i * kThreads] = w[i];
    }
    batch(w);
  }
  const float largest = st.m;  // of the vectors
  uint32_t mine = some ? ordered(largest) : 0u;
  if (part.single >= 0) {
    const float x = part.single_value();
    if (!(x <= st.m)) st.move_to(x);
    st.add(x);
    mine = max(mine, ordered(x));
  }
  st = join_warp(st);
  cluster_wait();
  if (lane == 0) {
    const uint32_t to = cluster_addr(&sh.stats[rank * kWarps + warp], 0);
    st_cluster(to, st.m);
    st_cluster(to + 4, st.s);
    st_cluster(to + 8, st.u);
  }

  // ---- this CTA's k largest, and what else reaches a bound below them: to the first CTA, which has places for them
  const int places = kMaxFound / C;  // (at least kMaxTop)
  if (k > 0) {
    const uint32_t bound = common_bound(mine, k, sh);
    const float bound_x = bound != 0 ? key_value(static_cast<Key>(bound) << 32) : -INFINITY;
    const uint32_t to = cluster_addr(all + rank * places, 0);
    auto put = [&](float x, int i) {
      if (x >= bound_x) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < places) st_cluster(to + 8 * at, make_key(x, i));
      }
    };
    if (some && largest >= bound_x)  // the thread's batches that reach the bound
      for (int e = 0; e < kEntries && part.v0 + e * part.per_entry * kBatch * kThreads + t < part.v1; ++e)
        if (__bfloat162float(maxima[e * kThreads + t]) >= bound_x) part.entry(e, bound_x, put);
    if (part.single >= 0) put(part.single_value(), part.single);
    sync_readers();
    int n = sh.count;
    if (n > places) {
      sync_readers();
      top_of_many(part, maxima, largest, some, k, found, sh);
      if (t < k) st_cluster(to + 8 * t, sh.top[t]);
      n = k;
    }
    if (t == 0) st_cluster(cluster_addr(&sh.counts[rank], 0), n);
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  } else {
    sync_readers();
  }

  // ---- the row's statistics, by every warp; the results
  Stats s{-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kMaxCluster * kWarps / 32; ++i) {
    if (32 * i + lane < C * kWarps) {
      Stats o = sh.stats[32 * i + lane];
      const float m = max_nan(s.m, o.m);
      s.move_to(m);
      o.move_to(m);
      s.s += o.s;
      s.u += o.u;
    }
  }
  s = join_warp(s);
  const bool good = s.s > 0.f && s.s < INFINITY;  // (NaN: no)
  const float nan = __int_as_float(0x7fc00000), log_s = good ? logf(s.s) : nan;
  if (t == 0) {
    if (!good) flag_error(a.err, RRA_ERR_PROBS);
    if (a.entropy != nullptr) a.entropy[r] = good ? fmaxf(log_s - kLn2 * (s.u / s.s), 0.f) : nan;
  }
  if (asks) {
    float lp = 0.f;  // (-1: no token)
    if (token < -1 || token >= V) {
      flag_error(a.err, RRA_ERR_TOKEN);
      lp = nan;
    } else if (token >= 0) {
      lp = (x_token - s.m) - log_s;
    }
    a.logprobs[r * a.T + lane] = lp;
  }
  if (k == 0) return;
  if (!good) {
    if (t < k) {
      a.top_tokens[r * k + t] = -1;
      a.top_logprobs[r * k + t] = nan;
    }
    return;
  }
  // the k largest of all keys, sorted by counting; of several CTAs' those that reach a bound made in the same way
  const Key* kept = all;
  int n = sh.counts[0];
  if (C > 1) {
    Key* list = reinterpret_cast<Key*>(smem);  // (the ring is done)
    static_assert(kRing * kStageBytes >= kMaxFound * 8, "they fit");
    Key mine_of[kMaxFound / kThreads];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kMaxFound / kThreads; ++i) {
      const int at = t + i * kThreads, c = at / places;
      mine_of[i] = c < C && at - c * places < sh.counts[c] ? all[at] : 0;
      best = max(best, static_cast<uint32_t>(mine_of[i] >> 32));
    }
    const uint32_t bound32 = common_bound(best, k, sh);  // (where too few threads have keys, this CTA's own stands: a lower one)
#pragma unroll
    for (int i = 0; i < kMaxFound / kThreads; ++i)
      if (mine_of[i] != 0 && static_cast<uint32_t>(mine_of[i] >> 32) >= bound32) list[atomicAdd(&sh.kept, 1)] = mine_of[i];
    sync_readers();
    kept = list;
    n = sh.kept;
  }
  for (int i = t; i < n; i += kThreads) {
    const Key key = kept[i];
    int larger = 0;
    for (int j = 0; j < n; ++j) larger += kept[j] > key;
    if (key != 0 && larger < k) {
      a.top_tokens[r * k + larger] = key_index(key);
      a.top_logprobs[r * k + larger] = (key_value(key) - s.m) - log_s;
    }
  }
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs& a, int clusters, cudaStream_t stream) {
  static int done[64] = {0};
  auto kern = token_logprobs_kernel<T>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {  // clusters of 16 CTAs are opt-in
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  cudaLaunchConfig_t cfg{};
  const unsigned y = static_cast<unsigned>(std::min<int64_t>(a.rows, 65535));
  cfg.gridDim = dim3(clusters, y, static_cast<unsigned>((a.rows + y - 1) / y));
  cfg.blockDim = dim3(kThreads + 32);
  cfg.dynamicSmemBytes = kSmemBytes;
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

extern "C" int rra_token_logprobs(const void* logits, int64_t stride_b, int64_t stride_t, const int32_t* tokens, int T,
                                  float* logprobs, float* entropy, int top_k, float* top_logprobs, int32_t* top_tokens,
                                  int B, int N, int V, rra_dtype dt, int32_t* err_flag, void* stream) {
  if (dt != RRA_F32 && dt != RRA_BF16) return RRA_EUNSUPPORTED;
  if (B < 0 || N < 1 || V < 1 || T < 0 || top_k < 0 || top_k > V) return RRA_EINVAL;
  if (T > rra::kMaxTokens || top_k > rra::kMaxTop) return RRA_EUNSUPPORTED;
  if (V > (1 << 30) || int64_t(B) * N > INT32_MAX) return RRA_ERANGE;
  if (B == 0) return RRA_OK;
  if (!logits || (T > 0 && (!tokens || !logprobs)) || (top_k > 0 && (!top_logprobs || !top_tokens))) return RRA_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) & (dt == RRA_BF16 ? 1 : 3)) return RRA_EINVAL;
  if (stride_b < 0 || stride_t < 0) return RRA_EINVAL;
  {  // an output over another one, over the tokens or over the logits: some row would read what another row wrote
    struct Range {
      const void* p;
      size_t n;
    };
    const size_t rows = size_t(B) * N * 4;
    const size_t es = dt == RRA_BF16 ? 2 : 4, span = (size_t(B - 1) * stride_b + size_t(N - 1) * stride_t + V) * es;
    const Range all[] = {{logprobs, rows * T}, {entropy, rows}, {top_logprobs, rows * top_k}, {top_tokens, rows * top_k}, {tokens, rows * T},
                         {logits, span}};
    for (int i = 0; i < 4; ++i)
      for (int j = i + 1; j < 6; ++j) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(all[i].p), y = reinterpret_cast<uintptr_t>(all[j].p);
        if (x != 0 && y != 0 && all[i].n > 0 && all[j].n > 0 && x < y + all[j].n && y < x + all[i].n) return RRA_EINVAL;
      }
  }
  rra::LogprobArgs a{};
  a.logits = logits;
  a.sb = stride_b;
  a.st = stride_t;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_logprobs = top_logprobs;
  a.top_tokens = top_tokens;
  a.rows = int64_t(B) * N;
  a.N = N;
  a.V = V;
  a.T = T;
  a.top_k = top_k;
  a.err = err_flag;
  // CTAs per row: the most (a power of two up to 16) that leave no SM more than two (64 x 128000 float32 14.7 us with 4,
  // 16.9 with 8, 17.3 with 2; 256 x 128256 bf16 21.2 with 1, 22.2 with 2; 1024 x 128000 bf16 51.5 with 1, 66 with 2, 79 with 4: clusters
  // wait for places side by side, and every CTA looks twice), and no more than one where their parts are short (32 x
  // 32000 bf16 6.5 us with 4, 8.7 with 8; 16 x 128000 bf16 7.7 with 16, 9.6 with 8; 1 x 128000 6.1 with 16, 8.3 with 8).
  const int64_t sms = std::max(1, rra::current_sm_count()), vecs = V / (dt == RRA_BF16 ? 8 : 4);
  int clusters = rra::kMaxCluster;
  while (clusters > 1 && (a.rows * clusters > 2 * sms ||
                          (a.rows * clusters > sms && vecs / clusters < 3 * rra::kThreads)))
    clusters /= 2;
  const cudaError_t e = dt == RRA_BF16 ? rra::launch_logprobs<__nv_bfloat16>(a, clusters, static_cast<cudaStream_t>(stream))
                                       : rra::launch_logprobs<float>(a, clusters, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return RRA_OK;
  rra::record_cuda_error(e, "token_logprobs launch");
  return RRA_ECUDA;
}
