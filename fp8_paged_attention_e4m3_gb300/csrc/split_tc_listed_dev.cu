// The tcgen05 split kernel over visit lists of a block-scaled cache, device-side plan: its
// instantiations, in a translation unit of their own so they compile in
// parallel.
#include "split_tc.cuh"

namespace vae4 {

cudaError_t launch_split_tc_listed_dev(const SplitParams &p, const TcArgs &a, int n,
                                       const CUtensorMap &map_k, const CUtensorMap &map_v,
                                       cudaStream_t stream) {
  return launch_tc_any<kPlanDevice, false, kListed>(p, a, n, map_k, map_v, stream);
}

}  // namespace vae4
