// The launches of shared-prefix attention: the prefix for all rows (shared_prefix.cuh), each
// sequence's own tokens (decode_mma.cuh for one new token, verify.cuh for more), the merge.
#include "shared_prefix.cuh"
#include "verify.cuh"

namespace rra {
namespace {

template <int D>
cudaError_t launch_d(const DecodeArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, const CUtensorMap& k_groups,
                     const CUtensorMap& v_groups, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.prefix_splits > 0)
    e = shared_prefix_nq(int64_t(a.B) * a.gamma * (a.Hq / a.Hkv)) == 2 ? spx::launch_prefix<D, 2>(a, k_groups, v_groups, st)
                                                                       : spx::launch_prefix<D, 1>(a, k_groups, v_groups, st);
  if (e != cudaSuccess) return e;
  if (a.gamma > 1)
    e = launch_decode_verify_t<D, true, false, true>(a, k_map, v_map, st);
  else if (a.hpc > 8)
    e = launch_decode_mma_nt<D, true, false, 2, false, true>(a, k_map, v_map, a.hpc, st);
  else
    e = launch_decode_mma_nt<D, true, false, 1, false, true>(a, k_map, v_map, a.hpc, st);
  if (e != cudaSuccess || a.num_splits == 1) return e;
  return spx::launch_merge<D>(a, st);
}

}  // namespace

cudaError_t launch_shared_prefix(const DecodeArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                 const CUtensorMap& k_groups, const CUtensorMap& v_groups, cudaStream_t stream) {
  return a.D == 128 ? launch_d<128>(a, k_map, v_map, k_groups, v_groups, stream)
                    : launch_d<64>(a, k_map, v_map, k_groups, v_groups, stream);
}

}  // namespace rra
