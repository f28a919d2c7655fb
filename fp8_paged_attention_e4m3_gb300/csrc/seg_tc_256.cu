// The split kernel over block-scaled caches, head dim 256: its instantiations,
// in a translation unit of their own so they compile in parallel.
#include "seg_tc.cuh"

namespace vae4 {
namespace seg {

cudaError_t launch_256(const SegParams &p, const CUtensorMap &k, const CUtensorMap &v,
                      cudaStream_t s) {
  return p.list ? launch_d<256, true>(p, k, v, s) : launch_d<256, false>(p, k, v, s);
}

}  // namespace seg
}  // namespace vae4
