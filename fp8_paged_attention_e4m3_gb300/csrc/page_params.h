// Launch parameters of the kernels that copy, fork, resize and compact the pages of a
// cache, shared by the host entry points and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vae4 {

constexpr int kMaxForkRows = 8192;     // a column tile of the table is held in shared memory
constexpr int kMaxResizeRows = 16384;  // (pages, first written page) of every row are held there

// CTAs of 1024 threads that share a large pool (256 rows of 2048, 246 thousand pages: 39.6 us
// with 32, 30.3 with 64, 29.3 with 128 and 152)
constexpr int kPoolGrid = 128;

// What a page holds of one tensor: n[0] x n[1] x n[2] runs of `run` vectors of
// `vec` bytes, the runs' starts s[0 .. 2] bytes apart; neighbouring dimensions that
// lie end to end are merged.
struct PageSlab {
  uint8_t *base;
  int64_t ps;       // bytes from page to page
  int64_t s[3];
  int32_t n[3];     // n[0] outermost
  int32_t run;      // vectors per run
  int32_t first;    // the slab's first vector in the page's numbering, a multiple of 32
  int32_t vecs;     // n[0] n[1] n[2] run
};

struct CopyParams {
  PageSlab slab[4];        // K, V, bounds, scales (the last two may be empty)
  int32_t vec[4];          // bytes of a vector: 16, 8 or 4
  int32_t vecs;            // of all slabs, with the gaps
  const int32_t *pairs;    // i32 [n][2]: source, destination
  int64_t pair_sb;
  int32_t n;
  int64_t n_pages;
  uint32_t *status;        // may be null
};

// A pool: its block table and the count of entries of every page.
struct PoolParams {
  int32_t *bt;             // i32 [B][cols]
  int64_t bt_sb;
  int32_t B, cols;
  int32_t *counts;         // i32 [n_pages]
  int32_t n_pages;
  uint32_t *status;        // may be null
};

struct ForkParams {
  PoolParams pool;
  const int32_t *parents;  // i32 [B]
  int32_t width;           // columns per CTA (set at the launch)
};

struct ResizeParams {
  PoolParams pool;
  const int32_t *seq;      // i32 [B] or [B][2]
  int32_t seq_sb, seq_has_qlen;
  int32_t page;
  int32_t *copies;         // i32 [B][2]
  int64_t copies_sb;
  int32_t *list;           // i32 [n_pages]: scratch
  int2 *sums;              // [kPoolGrid * 32]: scratch
};

struct CompactParams {
  PoolParams pool;
  int32_t *moves;          // i32 [n][2]
  int64_t moves_sb;
  int32_t n;
};

cudaError_t launch_copy_pages(const CopyParams &p, cudaStream_t stream);
cudaError_t launch_fork_pages(const ForkParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_resize_pages(const ResizeParams &p, cudaStream_t stream);
cudaError_t launch_compact_pages(const CompactParams &p, cudaStream_t stream);

}  // namespace vae4
