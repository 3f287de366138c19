// rra_tree_keep: which path of a tree of drafted tokens the target keeps, and its keys and values moved together in the
// caches of all layers.
//
// The path starts at node 0 and goes on from node x to its child with the token that the target chose after x (the
// lowest such child), until there is none. The i-th kept node, at cache slot p + node, belongs at slot p + i. Nodes come
// after their parents, so node >= i: moving them in order never writes a slot that a later one is still to be read from.
//
// Bound: latency (the walk: loads, then one step of a warp per kept node; the move: loads, then stores) for a few
// sequences; HBM for many, with each kept row that is not in place read and written once per layer. One CTA per
// sequence and pair of caches (a layer's K and V, as a rule): it walks for itself, then its threads take 16-byte columns of the
// kept rows. Every cache is in one pair, once: two CTAs that move the same rows would read what the other has written.
#include <cuda_runtime.h>

#include <algorithm>
#include <functional>

#include "rra_device.cuh"
#include "rra_internal.h"

namespace rra {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // rows that a thread loads before it stores them
constexpr int kMaxLayers = 128;

struct KeepArgs {
  const int32_t* tokens;         // [B, N]
  const int32_t* parents;        // [B, N]
  const int32_t* choices;        // [B, N], choice_stride elements apart
  int64_t choice_stride;
  const int32_t* lens;           // [B] or nullptr (N)
  const int32_t* positions;      // [B]
  const int32_t* block_table;    // nullptr: contiguous caches
  int max_blocks_per_seq, log2_bs, num_blocks, capacity;
  int32_t *tokens_out, *n_kept, *nodes_out, *positions_out;
  int B, N, pairs, Hkv, row_vecs;  // pairs of caches; 16-byte vectors of a head's row
  int32_t* err;
  void* caches[2 * kMaxLayers];  // different ones; the last one nullptr where their number is odd
};

__global__ void __launch_bounds__(kThreads) tree_keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int parent[kTreeMaxNodes], token[kTreeMaxNodes], choice[kTreeMaxNodes], path[kTreeMaxNodes];
  __shared__ long long src_row[kTreeMaxNodes], dst_row[kTreeMaxNodes];
  __shared__ int kept_sh, moves_sh;
  const int b = blockIdx.y, pair = blockIdx.x, t = threadIdx.x, lane = t & 31;
  pdl_wait();
  pdl_launch_dependents();
  const bool scribe = pair == 0;
  int n = a.lens != nullptr ? a.lens[b] : a.N;
  if (n < 0 || n > a.N) {
    if (scribe && t == 0) flag_error(a.err, RRA_ERR_SEQ_LEN);
    n = min(max(n, 0), a.N);
  }
  const int p = a.positions[b];
  const bool refused = n > 0 && (p < 0 || p > a.capacity - n);
  if (scribe && refused && t == 0) flag_error(a.err, RRA_ERR_POSITION);
  if (t < n) {
    const size_t at = static_cast<size_t>(b) * a.N + t;
    int up = a.parents[at];
    if (up < -1 || up >= t) {
      if (scribe) flag_error(a.err, RRA_ERR_TREE);
      up = -1;
    }
    parent[t] = up;
    token[t] = a.tokens[at];
    choice[t] = a.choices[static_cast<int64_t>(at) * a.choice_stride];
  }
  __syncthreads();
  if (t < 32) {  // the walk: lane l looks at nodes l, l + 32, ...
    int count = 0;
    for (int x = n > 0 ? 0 : -1; x >= 0;) {
      if (lane == 0) path[count] = x;
      ++count;
      const int want = choice[x];
      int next = -1;
#pragma unroll
      for (int w = kTreeMaxNodes / 32 - 1; w >= 0; --w) {
        const int j = 32 * w + lane;
        const uint32_t hit = __ballot_sync(0xffffffffu, j < n && parent[j] == x && token[j] == want && want >= 0);
        if (hit != 0) next = 32 * w + __ffs(hit) - 1;
      }
      x = next;  // (children come after their parents, so this ends)
    }
    if (lane == 0) kept_sh = count;
  }
  __syncthreads();
  const int kept = kept_sh;
  if (scribe) {
    for (int i = t; i < a.N; i += kThreads) {
      a.tokens_out[static_cast<size_t>(b) * a.N + i] = i < kept ? choice[path[i]] : -1;
      a.nodes_out[static_cast<size_t>(b) * a.N + i] = i < kept ? path[i] : -1;
    }
    if (t == 0) {
      a.n_kept[b] = kept;
      a.positions_out[b] = refused ? p : p + kept;
    }
  }
  if (refused || a.pairs == 0) return;
  // ---- the rows to move (path[i] = i from the start: in place)
  if (t == 0) {
    int first = 0;
    while (first < kept && path[first] == first) ++first;
    moves_sh = first;
  }
  __syncthreads();
  const int first = moves_sh;
  if (first == kept) return;
  if (t < 2 * kTreeMaxNodes) {  // cache rows of KV head 0, -1: none
    const int i = t >> 1;
    if (i >= first && i < kept) {
      const int slot = p + (t & 1 ? i : path[i]);
      long long row = static_cast<long long>(b) * a.Hkv * a.capacity + slot;
      if (a.block_table != nullptr) {
        const int phys = a.block_table[static_cast<size_t>(b) * a.max_blocks_per_seq + (slot >> a.log2_bs)];
        if (phys < 0 || phys >= a.num_blocks) {
          if (scribe) flag_error(a.err, RRA_ERR_BLOCK_ID);
          row = -1;
        } else {
          row = ((static_cast<long long>(phys) << a.log2_bs) + (slot & ((1 << a.log2_bs) - 1))) * a.Hkv;
        }
      }
      (t & 1 ? dst_row : src_row)[i] = row;
    }
  }
  __syncthreads();
  const long long head_stride = a.block_table != nullptr ? 1 : a.capacity;
  const int columns = a.Hkv * a.row_vecs, caches = a.caches[2 * pair + 1] != nullptr ? 2 : 1;
  for (int c = t; c < caches * columns; c += kThreads) {  // a column of one cache, then of the other: moved by one thread, in order
    const bool second = c >= columns;
    const int g = (second ? c - columns : c) / a.row_vecs, x = (second ? c - columns : c) - g * a.row_vecs;
    uint4* cache = static_cast<uint4*>(a.caches[2 * pair + (second ? 1 : 0)]) + x;
    for (int i = first; i < kept; i += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + k < kept && src_row[i + k] >= 0) v[k] = cache[(src_row[i + k] + g * head_stride) * a.row_vecs];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + k < kept && src_row[i + k] >= 0 && dst_row[i + k] >= 0) cache[(dst_row[i + k] + g * head_stride) * a.row_vecs] = v[k];
    }
  }
}

bool meet(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != 0 && y != 0 && an > 0 && bn > 0 && x < y + bn && y < x + an;
}

}  // namespace
}  // namespace rra

extern "C" int rra_tree_keep(const int32_t* draft_tokens, const int32_t* parents, const int32_t* choices, int64_t choice_stride,
                             const int32_t* tree_lens, const int32_t* positions, void* const* k_caches,
                             void* const* v_caches, int n_layers, const int32_t* block_table, int max_blocks_per_seq,
                             int block_size, int num_blocks, int max_len, int32_t* tokens_out, int32_t* n_kept,
                             int32_t* nodes_out, int32_t* positions_out, int B, int N, int Hkv, int D, rra_dtype dt,
                             int32_t* err_flag, void* stream) {
  using namespace rra;
  if (dt != RRA_F32 && dt != RRA_BF16) return RRA_EUNSUPPORTED;
  if (B < 0 || N < 1 || Hkv < 1 || n_layers < 0 || choice_stride < 0) return RRA_EINVAL;
  if (D != 64 && D != 128) return RRA_EUNSUPPORTED;
  if (N > kTreeMaxNodes || n_layers > kMaxLayers) return RRA_EUNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return RRA_ERANGE;
  int64_t capacity = max_len;
  int log2_bs = 0;
  if (block_table != nullptr) {
    if (block_size <= 0 || max_blocks_per_seq < 1 || num_blocks < 1) return RRA_EINVAL;
    if ((block_size & (block_size - 1)) != 0) return RRA_EUNSUPPORTED;
    while ((1 << log2_bs) < block_size) ++log2_bs;
    capacity = int64_t(max_blocks_per_seq) * block_size;
  } else if (max_len < 1) {
    return RRA_EINVAL;
  }
  if (capacity > (int64_t(1) << 30)) return RRA_ERANGE;
  if (B == 0) return RRA_OK;
  if (!draft_tokens || !parents || !choices || !positions || !tokens_out || !n_kept || !nodes_out || !positions_out)
    return RRA_EINVAL;
  if (n_layers > 0 && (!k_caches || !v_caches)) return RRA_EINVAL;
  KeepArgs a{};
  for (int l = 0; l < n_layers; ++l) {
    a.caches[2 * l] = k_caches[l];
    a.caches[2 * l + 1] = v_caches[l];
    for (const void* c : {k_caches[l], v_caches[l]})
      if (c == nullptr || (reinterpret_cast<uintptr_t>(c) & 15) != 0) return RRA_EINVAL;
  }
  // Each cache once (layers may share one); others must not meet.
  std::sort(a.caches, a.caches + 2 * n_layers, std::less<void*>());
  const int n_caches = static_cast<int>(std::unique(a.caches, a.caches + 2 * n_layers) - a.caches);
  std::fill(a.caches + n_caches, a.caches + 2 * n_layers, nullptr);
  const unsigned __int128 all_rows = block_table != nullptr ? static_cast<unsigned __int128>(num_blocks) << log2_bs
                                                            : static_cast<unsigned __int128>(B) * max_len;
  const size_t cache_bytes = static_cast<size_t>(
      std::min<unsigned __int128>(all_rows * Hkv * D * (dt == RRA_BF16 ? 2 : 4), size_t(1) << 62));
  for (int i = 0; i + 1 < n_caches; ++i)
    if (meet(a.caches[i], cache_bytes, a.caches[i + 1], cache_bytes)) return RRA_EINVAL;
  // Every pair's CTA reads the inputs, one of them writes the outputs, and all write to the caches meanwhile.
  const size_t s = size_t(B) * 4, sn = s * N, choice_bytes = ((size_t(B) * N - 1) * choice_stride + 1) * 4;
  const struct {
    const void* p;
    size_t n;
  } outs[] = {{tokens_out, sn}, {n_kept, s}, {nodes_out, sn}, {positions_out, s}},
    ins[] = {{draft_tokens, sn}, {parents, sn}, {choices, choice_bytes}, {tree_lens, s}, {positions, s},
           {block_table, s * max_blocks_per_seq}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return RRA_EINVAL;
    for (const auto& in : ins)
      if (meet(outs[i].p, outs[i].n, in.p, in.n)) return RRA_EINVAL;
  }
  for (int i = 0; i < n_caches; ++i) {
    for (const auto& out : outs)
      if (meet(a.caches[i], cache_bytes, out.p, out.n)) return RRA_EINVAL;
    for (const auto& in : ins)
      if (meet(a.caches[i], cache_bytes, in.p, in.n)) return RRA_EINVAL;
  }
  a.tokens = draft_tokens;
  a.parents = parents;
  a.choices = choices;
  a.choice_stride = choice_stride;
  a.lens = tree_lens;
  a.positions = positions;
  a.block_table = block_table;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.log2_bs = log2_bs;
  a.num_blocks = num_blocks;
  a.capacity = static_cast<int>(capacity);
  a.tokens_out = tokens_out;
  a.n_kept = n_kept;
  a.nodes_out = nodes_out;
  a.positions_out = positions_out;
  a.B = B;
  a.N = N;
  a.pairs = (n_caches + 1) / 2;
  a.Hkv = Hkv;
  a.row_vecs = D * (dt == RRA_BF16 ? 2 : 4) / 16;
  a.err = err_flag;
  const cudaError_t e = launch_pdl(tree_keep_kernel, dim3(std::max(1, a.pairs), B), dim3(kThreads), 0,
                                   static_cast<cudaStream_t>(stream), a);
  if (e == cudaSuccess) return RRA_OK;
  record_cuda_error(e, "tree_keep launch");
  return RRA_ECUDA;
}
