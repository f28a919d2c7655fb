// The tcgen05 split kernel over visit lists of a block-scaled cache, static grid: its
// instantiations, in a translation unit of their own so they compile in
// parallel.
#include "split_tc.cuh"

namespace vae4 {

cudaError_t launch_split_tc_listed_len(const SplitParams &p, const TcArgs &a, int n,
                                       const CUtensorMap &map_k, const CUtensorMap &map_v,
                                       cudaStream_t stream) {
  return launch_tc_any<kPlanFromLen, false, kListed>(p, a, n, map_k, map_v, stream);
}

}  // namespace vae4
