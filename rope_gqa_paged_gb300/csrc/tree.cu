// A tree of drafted tokens: RoPE and append of its nodes, and the launches of its attention (tree.cuh).
#include "tree.cuh"

namespace rra {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAhead = 2;  // pairs of vectors that a thread loads before it knows where the node is
static_assert(kAppendThreads >= kTreeMaxNodes && kAppendThreads >= kMaxDecodeHeadDim / 2, "a thread per node, per frequency");

// One CTA per node: its depth, the sines and cosines of its position (cached tokens + depth; rope_cos_sin), then
// q and k of every head in pairs of 16-byte vectors, turned with the error-free rotation of the other appends (the
// same bits), and v as it is. Bound: latency for few nodes, HBM (and L2) for many. The first vectors of each thread are on
// their way while the depth and the angles are found.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) tree_append_kernel(const __grid_constant__ TreeAppendArgs a) {
  constexpr int HALF = D / 2, kPairs = D / 16;  // pairs of vectors per head
  __shared__ float cs[4][HALF];
  __shared__ int parents[kTreeMaxNodes];
  __shared__ long long slot_sh;
  const int j = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  const size_t node = static_cast<size_t>(b) * a.N + j;
  const int items = (a.Hq + a.Hkv) * kPairs;
  pdl_wait();
  pdl_launch_dependents();  // (only now: see tree_attn_kernel)
  const int p = __ldcg(a.positions + b);
  int n = a.lens != nullptr ? __ldcg(a.lens + b) : a.N;
  int up = t <= j ? __ldcg(a.parents + static_cast<size_t>(b) * a.N + t) : -1;
  // half-split pairs: dims 8c .. and D/2 + 8c ..; interleaved: the 16 dims from 16c on
  const int step0 = a.rope_style == 1 ? 16 : 8, step1 = a.rope_style == 1 ? 8 : HALF;
  auto source = [&](int i) {
    const int h = i / kPairs, c = i - h * kPairs;
    return (h < a.Hq ? static_cast<const __nv_bfloat16*>(a.q) + (node * a.Hq + h) * D
                     : static_cast<const __nv_bfloat16*>(a.k_new) + (node * a.Hkv + h - a.Hq) * D) + step0 * c;
  };
  uint4 x0[kAhead], x1[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (t + k * kAppendThreads < items) {
      const __nv_bfloat16* src = source(t + k * kAppendThreads);
      x0[k] = *reinterpret_cast<const uint4*>(src);
      x1[k] = *reinterpret_cast<const uint4*>(src + step1);
    }
  if (n < 0 || n > a.N) {
    if (j == 0 && t == 0) flag_error(a.err, RRA_ERR_SEQ_LEN);
    n = min(max(n, 0), a.N);
  }
  if (n > 0 && (p < 0 || p > a.capacity - n)) {
    if (j == 0 && t == 0) flag_error(a.err, RRA_ERR_POSITION);
    return;
  }
  if (j >= n) return;
  if (t <= j) {
    if (up < -1 || up >= t) {
      if (t == j) flag_error(a.err, RRA_ERR_TREE);
      up = -1;
    }
    parents[t] = up;
  }
  if (t == kAppendThreads - 1) {  // where k and v of KV head 0 go (rows), -1: nowhere
    const int slot = p + j;
    long long row = static_cast<long long>(b) * a.Hkv * a.capacity + slot;
    if (a.block_table != nullptr) {
      const int phys = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks_per_seq + (slot >> a.log2_bs));
      if (phys < 0 || phys >= a.num_blocks) {
        flag_error(a.err, RRA_ERR_BLOCK_ID);
        row = -1;
      } else {
        row = ((static_cast<long long>(phys) << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1))) * a.Hkv;
      }
    }
    slot_sh = row;
  }
  __syncthreads();
  if (t < HALF) {
    int depth = 0;
    for (int x = parents[j]; x >= 0; x = parents[x]) ++depth;
    rope_cos_sin(p + depth, a.rope_phi[t], cs[0][t], cs[1][t], cs[2][t], cs[3][t]);
  }
  __syncthreads();
  const size_t head_stride = a.block_table != nullptr ? 1 : a.capacity;
  const long long slot = slot_sh;
  auto turn = [&](int i, const uint4& w0, const uint4& w1) {
    const int h = i / kPairs, c = i - h * kPairs;
    if (h >= a.Hq && slot < 0) return;
    __nv_bfloat16* dst = (h < a.Hq ? static_cast<__nv_bfloat16*>(a.q_out) + (node * a.Hq + h) * D
                                   : static_cast<__nv_bfloat16*>(a.k_cache) + (slot + (h - a.Hq) * head_stride) * D) + step0 * c;
    float x[8], y[8], u[8], v[8];
    Elem<__nv_bfloat16>::unpack(w0, x);
    Elem<__nv_bfloat16>::unpack(w1, y);
    if (a.rope_style == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int f = 8 * c + e, f2 = f + 4;
        u[2 * e] = rotate_diff(x[2 * e], x[2 * e + 1], cs[0][f], cs[1][f], cs[2][f], cs[3][f]);
        u[2 * e + 1] = rotate_diff(x[2 * e + 1], -x[2 * e], cs[0][f], cs[1][f], cs[2][f], cs[3][f]);
        v[2 * e] = rotate_diff(y[2 * e], y[2 * e + 1], cs[0][f2], cs[1][f2], cs[2][f2], cs[3][f2]);
        v[2 * e + 1] = rotate_diff(y[2 * e + 1], -y[2 * e], cs[0][f2], cs[1][f2], cs[2][f2], cs[3][f2]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int f = 8 * c + e;
        u[e] = rotate_diff(x[e], y[e], cs[0][f], cs[1][f], cs[2][f], cs[3][f]);
        v[e] = rotate_diff(y[e], -x[e], cs[0][f], cs[1][f], cs[2][f], cs[3][f]);
      }
    }
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
    *reinterpret_cast<uint4*>(dst + step1) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (t + k * kAppendThreads < items) turn(t + k * kAppendThreads, x0[k], x1[k]);
  for (int i = t + kAhead * kAppendThreads; i < items; i += kAppendThreads) {
    const __nv_bfloat16* src = source(i);
    const uint4 w0 = *reinterpret_cast<const uint4*>(src), w1 = *reinterpret_cast<const uint4*>(src + step1);
    turn(i, w0, w1);
  }
  if (slot < 0) return;
  for (int i = t; i < a.Hkv * (D / 8); i += kAppendThreads) {
    const int g = i / (D / 8), c = i - g * (D / 8);
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v_new) + (node * a.Hkv + g) * D + 8 * c);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_cache) + (slot + g * head_stride) * D + 8 * c) = x;
  }
}

template <int D, int NQ>
cudaError_t launch_nq(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  return a.block_table != nullptr ? tree::launch_attn<D, NQ, true>(a, km, vm, st) : tree::launch_attn<D, NQ, false>(a, km, vm, st);
}

}  // namespace

cudaError_t launch_tree_attn(const TreeArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  if (a.D == 128) return a.nq == 2 ? launch_nq<128, 2>(a, k_map, v_map, stream) : launch_nq<128, 1>(a, k_map, v_map, stream);
  return a.nq == 2 ? launch_nq<64, 2>(a, k_map, v_map, stream) : launch_nq<64, 1>(a, k_map, v_map, stream);
}

cudaError_t launch_tree_append(const TreeAppendArgs& a, cudaStream_t stream) {
  const dim3 grid(a.N, a.B);
  return a.D == 128 ? launch_pdl(tree_append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, a)
                    : launch_pdl(tree_append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, a);
}

}  // namespace rra
