// rra_accept_draft: which drafted tokens the target keeps, and the token that follows them.
//
// Token x_j, drafted with probability q_j(x_j), is kept while u_j q_j(x_j) < p_j(x_j), that is with
// probability min(1, p_j / q_j). The first token that is not kept, at n, is replaced by a draw from
// the normalised rest max(p_n - q_n, 0); when all are kept one more is drawn from p_n. So every token
// follows the target's distribution ("Transformer架构优化实战2026：注意力机制、KV Cache与推理加速完整指南"
// §五 names the method). The draw inverts the cumulative distribution: the lowest index v with
// r_0 + ... + r_v > u (r_0 + ... + r_(V-1)).
//
// Exactness: u q and p are compared as float64 products (24 x 24 bits fit 53). The r_v are summed as
// 64-bit integers in units of 2^-60, each probability cut to a whole number of units: integer
// sums do not depend on their order, so any split of the vocabulary over lanes, warps and CTAs
// gives the same token, and a float64 cumulative sum does unless u falls within ~V 2^-53 of a border.
//
// Bound: HBM (one row of p, and one of q where a token was rejected) for large batches, latency for
// small ones. One cluster of CTAs takes a sequence: each CTA decides n for itself (two
// dependent loads), sums its part of the vocabulary (a contiguous run per warp, lanes on
// consecutive values, so rows of any alignment and stride load in whole lines), and the CTAs exchange
// their sums through distributed shared memory: one launch, no workspace, no atomics. The warp whose
// run holds the border reads it again (from L1 or L2) and scans it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rra_device.cuh"
#include "rra_internal.h"

namespace rra {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxGamma = 32;   // one lane of a warp per drafted token
constexpr int kBatch = 8;       // groups of 32 values whose loads a warp has in flight together

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

// A probability as a whole number of 2^-60 units (NaN: 0; outside [0, 1]: the nearer end).
__device__ __forceinline__ uint64_t units(float x) {
  return __float2ull_rz(fminf(fmaxf(x, 0.f), 1.f) * 0x1p60f);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
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
__device__ __forceinline__ uint64_t ld_cluster(const uint64_t* local, uint32_t rank) {
  uint32_t addr;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// The rest of one sequence's distribution at the decisive row: r_v and p_v in units.
template <typename T>
struct Rest {
  const T* p;
  const T* q;      // nullptr: nothing is taken off, but from `skip`
  int skip;        // token whose p counts as taken off entirely (no draft probabilities), or -1
  __device__ __forceinline__ uint64_t rest(float pv, float qv, int v) const {
    const uint64_t a = units(pv), b = units(qv);
    return v == skip || a <= b ? 0 : a - b;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) accept_draft_kernel(const AcceptArgs a) {
  __shared__ uint64_t warp_sums[2][kWarps];
  __shared__ uint64_t cta_sums[2];
  const int b = blockIdx.y, C = gridDim.x;
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gamma = a.gamma, V = a.V;

  pdl_wait();
  pdl_launch_dependents();
  const bool scribe = rank == 0 && warp == 0;  // the warp that writes what does not depend on the draw

  // ---- how many tokens are kept (every warp finds it for itself: lane j has token j)
  int len = a.lens != nullptr ? a.lens[b] : gamma;
  if (len < 0 || len > gamma) {
    if (scribe && lane == 0) flag_error(a.err, RRA_ERR_SEQ_LEN);
    len = min(max(len, 0), gamma);
  }
  const T* prow = static_cast<const T*>(a.p) + b * a.p_sb;
  const T* qrow = static_cast<const T*>(a.q) + b * a.q_sb;
  int x = -1;
  bool keep = false;
  if (lane < len) {
    x = a.tokens[static_cast<size_t>(b) * gamma + lane];
    const float u = a.u_accept[static_cast<size_t>(b) * gamma + lane];
    if (x < 0 || x >= V) {
      if (scribe) flag_error(a.err, RRA_ERR_TOKEN);
    } else {
      const float px = Elem<T>::load(prow + lane * a.p_st + x);
      const float qx = a.q != nullptr ? Elem<T>::load(qrow + lane * a.q_st + x) : 1.f;
      keep = static_cast<double>(u) * static_cast<double>(qx) < static_cast<double>(px);
    }
  }
  const uint32_t dropped = ~__ballot_sync(0xffffffffu, keep);
  const int n = min(dropped != 0 ? __ffs(dropped) - 1 : 32, len);
  const int at = __shfl_sync(0xffffffffu, x, n & 31);  // the rejected token (n < len)
  const Rest<T> rest{prow + n * a.p_st, n < len && a.q != nullptr ? qrow + n * a.q_st : nullptr,
                     n < len && a.q == nullptr ? at : -1};
  if (scribe) {
    for (int j = lane; j <= gamma; j += 32) {
      if (j != n) a.tokens_out[static_cast<size_t>(b) * (gamma + 1) + j] = j < n ? x : -1;
    }
    if (lane == 0) {
      a.n_accepted[b] = n;
      if (a.positions_out != nullptr) a.positions_out[b] = a.positions[b] + n + 1;
    }
  }

  // ---- sums of r and p over this warp's run of the vocabulary
  const int groups = (V + 31) / 32;                             // of 32 values
  const int per_warp = (groups + C * kWarps - 1) / (C * kWarps);
  const int g0 = min((static_cast<int>(rank) * kWarps + warp) * per_warp, groups);
  const int g1 = min(g0 + per_warp, groups);
  uint64_t sr = 0, sp = 0;
  for (int g = g0; g < g1; g += kBatch) {
    float pv[kBatch], qv[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int v = (g + k) * 32 + lane;
      const bool in = g + k < g1 && v < V;
      pv[k] = in ? Elem<T>::load(rest.p + v) : 0.f;
      qv[k] = in && rest.q != nullptr ? Elem<T>::load(rest.q + v) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      sr += rest.rest(pv[k], qv[k], (g + k) * 32 + lane);
      sp += units(pv[k]);
    }
  }
  sr = warp_sum(sr);
  sp = warp_sum(sp);
  if (lane == 0) {
    warp_sums[0][warp] = sr;
    warp_sums[1][warp] = sp;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    uint64_t s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += warp_sums[threadIdx.x][w];
    cta_sums[threadIdx.x] = s;
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();

  // ---- the border u * total, and the warp whose run holds it
  const uint64_t cr = lane < C ? ld_cluster(&cta_sums[0], lane) : 0;
  const uint64_t cp = lane < C ? ld_cluster(&cta_sums[1], lane) : 0;
  cluster_arrive();  // this CTA has read the others' sums
  const uint64_t total_r = warp_sum(cr), total_p = warp_sum(cp);
  // nothing is left (p <= q everywhere, by rounding): draw from p itself
  const int which = total_r > 0 ? 0 : 1;
  const uint64_t total = which == 0 ? total_r : total_p;
  const float u = fminf(fmaxf(a.u_sample[b], 0.f), 1.f - 0x1p-24f);
  const uint64_t border = __umul64hi(total, __float2ull_rz(u * 0x1p64f));  // floor(u * total)
  uint64_t before = warp_sum(lane < static_cast<int>(rank) ? (which == 0 ? cr : cp) : 0);
  before += warp_sum(lane < warp ? warp_sums[which][lane & (kWarps - 1)] : 0);
  const uint64_t mine = warp_sums[which][warp];
  int32_t* token_out = a.tokens_out + static_cast<size_t>(b) * (gamma + 1) + n;
  if (total == 0) {
    if (scribe && lane == 0) {
      flag_error(a.err, RRA_ERR_PROBS);
      *token_out = V - 1;
    }
  } else if (before <= border && border < before + mine) {
    bool found = false;
    for (int g = g0; g < g1 && !found; g += kBatch) {
      uint64_t val[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int v = (g + k) * 32 + lane;
        const bool in = g + k < g1 && v < V;
        const float pv = in ? Elem<T>::load(rest.p + v) : 0.f;
        const float qv = in && rest.q != nullptr ? Elem<T>::load(rest.q + v) : 0.f;
        val[k] = which == 0 ? rest.rest(pv, qv, v) : units(pv);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        uint64_t c = val[k];  // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, c, d);
          if (lane >= d) c += y;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, before + c > border);
        if (!found && over != 0) {
          found = true;
          if (lane == 0) *token_out = (g + k) * 32 + __ffs(over) - 1;
        }
        before += __shfl_sync(0xffffffffu, c, 31);
      }
    }
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
  const int clusters = rra::kMaxCluster;
  const cudaError_t e = dt == RRA_BF16
                            ? rra::launch_accept<__nv_bfloat16>(a, B, clusters, static_cast<cudaStream_t>(stream))
                            : rra::launch_accept<float>(a, B, clusters, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) return RRA_OK;
  rra::record_cuda_error(e, "accept_draft launch");
  return RRA_ECUDA;
}
