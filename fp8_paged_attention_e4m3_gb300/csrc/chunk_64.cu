// Chunk attention, head dim 64 (see chunk.cuh).
#include "chunk.cuh"

namespace vae4 {
namespace chunk {
cudaError_t launch_64(const ChunkParams &p, cudaStream_t s) { return launch_d<64>(p, s); }
}  // namespace chunk
}  // namespace vae4
