// The two launches of shared-prefix attention: the prefix for all rows (shared_prefix.cuh), then
// each sequence's own tokens and the merge (verify.cuh).
#include "shared_prefix.cuh"
#include "verify.cuh"

namespace rra {

cudaError_t launch_shared_prefix(const DecodeArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                 cudaStream_t stream) {
  if (a.prefix_splits > 0) {
    const cudaError_t e = a.D == 128 ? spx::launch_prefix<128>(a, k_map, v_map, stream)
                                     : spx::launch_prefix<64>(a, k_map, v_map, stream);
    if (e != cudaSuccess) return e;
  }
  return a.D == 128 ? launch_decode_verify_t<128, true, false, true>(a, k_map, v_map, stream)
                    : launch_decode_verify_t<64, true, false, true>(a, k_map, v_map, stream);
}

}  // namespace rra
