// The launches of shared-prefix attention: the prefix for all rows (shared_prefix.cuh), each sequence's
// own tokens (own_tokens.cuh), the merge.
#include "own_tokens.cuh"
#include "shared_prefix.cuh"

namespace rra {
namespace {

// SHORT_PREFIX: of at most kShortRow tokens, whose pass holds P to 2^-16 for every row. Behind a longer one, short
// sequences are the own-token kernel's alone.
template <int D, bool SHORT_PREFIX>
cudaError_t launch_d(const DecodeArgs& a, const SharedMaps& m, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.prefix_splits > 0)
    e = shared_prefix_nq(int64_t(a.B) * a.gamma * (a.Hq / a.Hkv)) == 2
            ? spx::launch_prefix<D, 2, SHORT_PREFIX>(a, m.k_prefix, m.v_prefix, st)
            : spx::launch_prefix<D, 1, SHORT_PREFIX>(a, m.k_prefix, m.v_prefix, st);
  if (e != cudaSuccess) return e;
  e = a.hpc * a.gamma > 8 ? own::launch<D, 2, !SHORT_PREFIX>(a, m.k_own, m.v_own, st)
                          : own::launch<D, 1, !SHORT_PREFIX>(a, m.k_own, m.v_own, st);
  if (e != cudaSuccess || a.num_splits == 1) return e;
  return spx::launch_merge<D>(a, st);
}

template <int D>
cudaError_t launch_d(const DecodeArgs& a, const SharedMaps& m, cudaStream_t st) {
  return a.prefix_splits > 0 && a.prefix_len <= spx::kShortRow ? launch_d<D, true>(a, m, st) : launch_d<D, false>(a, m, st);
}

}  // namespace

cudaError_t launch_shared_prefix(const DecodeArgs& a, const SharedMaps& maps, cudaStream_t stream) {
  return a.D == 128 ? launch_d<128>(a, maps, stream) : launch_d<64>(a, maps, stream);
}

}  // namespace rra
