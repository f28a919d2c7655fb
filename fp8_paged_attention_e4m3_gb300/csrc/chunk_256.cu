// Chunk attention, head dim 256 (see chunk.cuh).
#include "chunk.cuh"

namespace vae4 {
namespace chunk {
cudaError_t launch_256(const ChunkParams &p, cudaStream_t s) { return launch_d<256>(p, s); }
}  // namespace chunk
}  // namespace vae4
