// rra_token_logprobs: log probabilities of given tokens, the entropy and the most likely tokens of rows of logits.
//
// With m the largest logit of a row, S = sum e^(x - m) and U = sum (x - m) e^(x - m):
//   log p(v) = x_v - m - ln S,   H = -sum p ln p = ln S - U / S.
// One pass keeps (m, S, U) of what a thread has seen, in float32 and units of log2; when the maximum moves by d,
// S' = 2^d S and U' = 2^d (U + d S). Logits of -inf (masked) add nothing; a row that holds a NaN or +inf, or nothing
// above -inf, has no distribution.
//
// The most likely tokens come from a second look at few values. Order all logits by (value, lower index first). A thread
// keeps its largest. The k-th largest T of what the threads hold is no larger than the k-th largest of the part that the
// CTA has, and whatever is as large lies with threads whose largest is: so only those look through their values
// again and put down what reaches T (some 2 k values where a row is in no order), and the k largest are sorted by
// counting, for each, how many are larger. T is taken from the largest few of each warp.
//
// Bound: HBM (each logit read once) for many rows; latency for few. One cluster of CTAs takes a row and joins its
// parts through distributed shared memory: one launch, no workspace; the atomics only hand out places in a list that is
// sorted afterwards, so results do not depend on their order.
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
constexpr int kMaxFound = 1024;  // values that reach T; more go the long way

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
  __device__ __forceinline__ void join(const Stats& o) {
    const float to = fmaxf(m, o.m);
    Stats b = o;
    move_to(to);
    b.move_to(to);
    s += b.s;
    u += b.u;
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
__device__ __forceinline__ Key ld_cluster_key(uint32_t addr) {
  Key v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct Shared {
  Stats warp_stats[kWarps], stats;
  Key held[kWarps * kMaxTop];     // the largest keys of each warp's threads
  Key found[kMaxFound];
  Key top[kMaxTop];               // this CTA's, sorted; 0 past the end
  Key all[kMaxCluster * kMaxTop];
  Key best[kWarps];
  int count;
};

// A thread's part of the row: vectors v0 + threadIdx.x, + kThreads, ... below v1, whose first element is
// head + E v, and at most one element in front of or behind the vectors.
template <typename T>
struct Part {
  const T* row;
  int head, v0, v1, single;       // single: its index, -1: none
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {  // f(value, index), indexes ascending but for the single one
    constexpr int E = Elem<T>::kPerChunk;
    const uint4* vec = reinterpret_cast<const uint4*>(row + head);
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kThreads) {
      float x[E];
      Elem<T>::unpack(vec[v], x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e], head + E * v + e);
    }
    if (single >= 0) f(Elem<T>::load(row + single), single);
  }
};

// The CTA's k largest keys by taking the largest below the last one, k times.
template <typename T>
__device__ __noinline__ void top_slowly(const Part<T>& part, int k, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Key last = ~Key(0);
  for (int r = 0; r < k; ++r) {
    Key mine = 0;
    part.each([&](float x, int i) {
      const Key key = make_key(x, i);
      if (key < last && key > mine) mine = key;
    });
    mine = warp_max(mine);
    if (lane == 0) sh.best[warp] = mine;
    __syncthreads();
    last = 0;
    for (int w = 0; w < kWarps; ++w) last = max(last, sh.best[w]);
    if (threadIdx.x == 0) sh.top[r] = last;
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int E = Elem<T>::kPerChunk;
  __shared__ Shared sh;
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;  // row b N + t
  if (r >= a.rows) return;  // (the whole cluster)
  const int C = gridDim.x, rank = static_cast<int>(cluster_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = r / a.N;
  const T* row = static_cast<const T*>(a.logits) + b * a.sb + (r - b * a.N) * a.st;
  const int V = a.V, k = a.top_k;
  // the given tokens' logits
  int token = -1;
  float x_token = 0.f;
  const bool asks = rank == 0 && warp == 1 && lane < a.T;
  if (asks) {
    token = a.tokens[r * a.T + lane];
    if (token >= 0 && token < V) x_token = Elem<T>::load(row + token);
  }

  // ---- (m, S, U), one pass
  Part<T> part;
  part.row = row;
  part.head = static_cast<int>(min(static_cast<uint32_t>(V), static_cast<uint32_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / static_cast<uint32_t>(sizeof(T))));
  const int vecs = (V - part.head) / E, tail = V - part.head - vecs * E;
  const int per = (vecs + C - 1) / C;
  part.v0 = min(rank * per, vecs);
  part.v1 = min(part.v0 + per, vecs);
  const int t = threadIdx.x;
  part.single = rank != 0 ? -1 : t < part.head ? t : t >= E && t - E < tail ? V - tail + t - E : -1;
  Stats st{-INFINITY, 0.f, 0.f};
  int best = -1;  // first vector of the batch that raised the maximum last
  const uint4* vec = reinterpret_cast<const uint4*>(row + part.head);
  for (int v = part.v0 + t; v < part.v1; v += kBatch * kThreads) {
    uint4 w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (v + i * kThreads < part.v1) w[i] = vec[v + i * kThreads];
    float x[kBatch][E];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (v + i * kThreads < part.v1) {
        Elem<T>::unpack(w[i], x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) mx = fmaxf(mx, x[i][e]);
    }
    if (mx > st.m || best < 0) {
      st.move_to(fmaxf(mx, st.m));
      best = v;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) st.add(x[i][e]);
  }
  Key mine = 0;  // the thread's largest
  if (k > 0 && best >= 0) {
    for (int i = 0; i < kBatch; ++i) {
      const int v = best + i * kThreads;
      if (v < part.v1) {
        float x[E];
        Elem<T>::unpack(vec[v], x);
#pragma unroll
        for (int e = 0; e < E; ++e) mine = max(mine, make_key(x[e], part.head + E * v + e));
      }
    }
  }
  if (part.single >= 0) {
    const float x = Elem<T>::load(row + part.single);
    if (x > st.m) st.move_to(x);
    st.add(x);
    mine = max(mine, make_key(x, part.single));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Stats o;
    o.m = __shfl_xor_sync(0xffffffffu, st.m, d);
    o.s = __shfl_xor_sync(0xffffffffu, st.s, d);
    o.u = __shfl_xor_sync(0xffffffffu, st.u, d);
    st.join(o);
  }
  if (lane == 0) sh.warp_stats[warp] = st;

  // ---- this CTA's k largest
  if (k > 0) {
    const int per_warp = min(kMaxTop, 2 * ((k + kWarps - 1) / kWarps));
    Key left = mine;
    for (int i = 0; i < per_warp; ++i) {
      const Key top = warp_max(left);
      if (lane == 0) sh.held[warp * per_warp + i] = top;
      if (left == top) left = 0;  // (keys differ, but for 0)
    }
    if (t == 0) sh.count = 0;
    __syncthreads();
    // T: the k-th largest of what the warps hold (0 where the CTA has fewer values)
    const int held = kWarps * per_warp;
    Key T_key = 0;
    for (int i = lane; i < held; i += 32) {
      const Key key = sh.held[i];
      int larger = 0;
      for (int j = 0; j < held; ++j) larger += sh.held[j] > key;
      if (larger == k - 1) T_key = key;
    }
    T_key = warp_max(T_key);
    if (mine >= T_key && mine != 0)
      part.each([&](float x, int i) {
        const Key key = make_key(x, i);
        if (key >= T_key) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kMaxFound) sh.found[at] = key;
        }
      });
    for (int i = t; i < k; i += kThreads) sh.top[i] = 0;
    __syncthreads();
    const int found = sh.count;
    if (found > kMaxFound) {
      top_slowly(part, k, sh);
    } else {
      for (int i = t; i < found; i += kThreads) {
        const Key key = sh.found[i];
        int larger = 0;
        for (int j = 0; j < found; ++j) larger += sh.found[j] > key;
        if (larger < k) sh.top[larger] = key;
      }
    }
  }
  __syncthreads();
  if (t == 0) {
    Stats s = sh.warp_stats[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s.join(sh.warp_stats[w]);
    sh.stats = s;
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    // ---- the row's statistics, by every warp; the results
    Stats s{-INFINITY, 0.f, 0.f};
    if (lane < C) {
      const uint32_t at = cluster_addr(&sh.stats, lane);
      s.m = ld_cluster_f32(at);
      s.s = ld_cluster_f32(at + 4);
      s.u = ld_cluster_f32(at + 8);
    }
    for (int i = t; i < C * k; i += kThreads) sh.all[i] = ld_cluster_key(cluster_addr(&sh.top[i % k], i / k));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      Stats o;
      o.m = __shfl_xor_sync(0xffffffffu, s.m, d);
      o.s = __shfl_xor_sync(0xffffffffu, s.s, d);
      o.u = __shfl_xor_sync(0xffffffffu, s.u, d);
      s.join(o);
    }
    __syncthreads();
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
    for (int i = t; i < C * k; i += kThreads) {
      const Key key = sh.all[i];
      int larger = 0;
      for (int j = 0; j < C * k; ++j) larger += sh.all[j] > key;
      if (key != 0 && larger < k) {
        a.top_tokens[r * k + larger] = good ? key_index(key) : -1;
        a.top_logprobs[r * k + larger] = good ? (key_value(key) - s.m) - log_s : nan;
      }
    }
  }
  cluster_arrive();  // no CTA's lists go away while another may still read them
  cluster_wait();
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
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = 1;
  }
  cudaLaunchConfig_t cfg{};
  const unsigned y = static_cast<unsigned>(std::min<int64_t>(a.rows, 65535));
  cfg.gridDim = dim3(clusters, y, static_cast<unsigned>((a.rows + y - 1) / y));
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
  {  // an output over another one or over the tokens: some row would read what another row wrote
    struct Range {
      const void* p;
      size_t n;
    };
    const size_t rows = size_t(B) * N * 4;
    const Range all[] = {{logprobs, rows * T}, {entropy, rows}, {top_logprobs, rows * top_k}, {top_tokens, rows * top_k}, {tokens, rows * T}};
    for (int i = 0; i < 4; ++i)
      for (int j = i + 1; j < 5; ++j) {
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
  const int64_t sms = std::max(1, rra::current_sm_count());
  int clusters = a.rows * rra::kMaxCluster <= sms ? rra::kMaxCluster : 8;
  while (clusters > 1 && int64_t(clusters) * a.rows > rra::kCtasPerSm * sms) clusters /= 2;
  const cudaError_t e = dt == RRA_BF16 ? rra::launch_logprobs<__nv_bfloat16>(a, clusters, static_cast<cudaStream_t>(stream))
                                       : rra::launch_logprobs<float>(a, clusters, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return RRA_OK;
  rra::record_cuda_error(e, "token_logprobs launch");
  return RRA_ECUDA;
}
