// Chunk attention, head dim 128 (see chunk.cuh).
#include "chunk.cuh"

namespace vae4 {
namespace chunk {
cudaError_t launch_128(const ChunkParams &p, cudaStream_t s) { return launch_d<128>(p, s); }
}  // namespace chunk
}  // namespace vae4
