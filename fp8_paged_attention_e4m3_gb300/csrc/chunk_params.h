// Launch parameters of chunk attention, shared by the host entry point and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vae4 {

constexpr int kMaxChunkCtas = 1024;
constexpr int kMaxChunk = 65536;  // new tokens of a sequence

// A unit that several CTAs share: where its parts lie and which rows it holds.
struct alignas(16) ChunkSplit {
  int32_t b, h, row0, parts;  // parts = 0: none starts in this CTA
  int32_t rows, pad[3];       // live rows from row0 on
};

// Strides are in elements (bytes for the caches).
struct ChunkParams {
  const void *q;               // f16 or bf16 [B][Qmax][Hq][D]
  int64_t q_sb, q_si, q_sh;
  void *out;                   // the same type and shape
  int64_t o_sb, o_si, o_sh;
  const uint8_t *k_base, *v_base;
  int64_t k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;
  int64_t n_pages;
  int32_t wide;                // bases and strides are multiples of 16
  const int32_t *bt;
  int64_t bt_sb;
  const int32_t *seq;          // i32 [B] or [B][2]
  int32_t seq_sb, seq_has_qlen;
  int32_t capacity;            // most tokens of a sequence
  const float *scales;         // of page ph, K | V w, head h, block x: ph s_page + w s_kv + h s_head + x
  int64_t s_page, s_kv, s_head;
  int32_t page_blocks;         // page / blk
  unsigned long long page_m, blk_m;  // reciprocals of page and block (div16)
  float *ws_ml;                // f32 [2 ctas][R][2]
  float *ws_o;                 // f32 [2 ctas][R][D]
  ChunkSplit *split;           // [ctas]
  uint32_t *status;
  int32_t B, Qmax, Hkv, G, D, page;
  int32_t bf16, e5m2;
  int32_t ctas;                // groups of CTAs (chunk_group)
  float alpha;                 // softmax_scale log2(e) = alpha 2^alpha_e, 1 <= alpha <= 2
  int32_t alpha_e;
  long long wait_limit, drain_limit;  // SM cycles
};

// CTAs that share a unit, and its rows: each CTA has two tiles of 128, one where a key's
// head is 256 wide.
__host__ __device__ constexpr int chunk_group(int D) { return D == 64 ? 1 : 2; }
__host__ __device__ constexpr int chunk_rows(int D) { return (D <= 128 ? 256 : 128) * chunk_group(D); }

cudaError_t launch_chunk(const ChunkParams &p, cudaStream_t stream);
cudaError_t launch_chunk_combine(const ChunkParams &p, cudaStream_t stream);

}  // namespace vae4
