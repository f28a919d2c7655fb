// The pages' lives: copying pages of a cache, and a pool's fork, resize and compaction.
//
// A pool is a block table and a count for every page of the table entries that hold
// it (0: free, below 0: kept).  Everything that a call decides follows from the pool
// alone, in one order (sequences ascending, then places, then page ids), so that its
// results do not depend on how the threads run: counts are changed by integer
// additions, and ranks come from prefix sums.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "block_common.cuh"
#include "kernels.h"
#include "page_params.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// copy: every pair's pages, all slabs.
//
// One CTA per pair and 1024 vectors of 16 bytes: four loads per thread in flight
// before the first store.  The slabs of a page are numbered one after another (from
// multiples of 32, so that a warp copies from one slab).  Bound by memory: 901 pages of
// 128 KB with scales and bounds, 240 MB read and written, 37.6 us, 0.94 of the rate of a
// plain copy; a single page of 2 KB, a launch.
constexpr int kCopyThreads = 256, kCopyUnroll = 4;

__device__ __forceinline__ int64_t slab_offset(const PageSlab &s, int v, int vec) {
  if (s.n[2] == 1) return (int64_t)v * vec;
  const int r = v / s.run, c = v - r * s.run;
  const int r1 = r / s.n[2], i2 = r - r1 * s.n[2];
  const int i0 = r1 / s.n[1], i1 = r1 - i0 * s.n[1];
  return i0 * s.s[0] + i1 * s.s[1] + i2 * s.s[2] + (int64_t)c * vec;
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  await_previous();
  const int32_t *pr = p.pairs + (int64_t)blockIdx.x * p.pair_sb;
  const int src = load_dep(pr), dst = load_dep(pr + 1);
  if (src == dst) return;  // padding (-1, -1) too
  if (src < 0 || dst < 0 || src >= p.n_pages || dst >= p.n_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    return;
  }
  for (int v0 = blockIdx.y * (kCopyThreads * kCopyUnroll); v0 < p.vecs;
       v0 += gridDim.y * (kCopyThreads * kCopyUnroll)) {
    uint4 x[kCopyUnroll];
    uint8_t *to[kCopyUnroll];
    int size[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const int v = v0 + u * kCopyThreads + (int)threadIdx.x;
      int k = 0;
#pragma unroll
      for (int t = 1; t < 4; ++t)
        if (v >= p.slab[t].first) k = t;
      const PageSlab &s = p.slab[k];
      size[u] = 0;
      if (v - s.first < s.vecs) {
        const int vec = p.vec[k];
        const int64_t off = slab_offset(s, v - s.first, vec);
        const uint8_t *from = s.base + src * s.ps + off;
        to[u] = s.base + dst * s.ps + off;
        size[u] = vec;
        if (vec == 16)
          x[u] = load_dep(reinterpret_cast<const uint4 *>(from));
        else if (vec == 8)
          *reinterpret_cast<uint2 *>(&x[u]) = load_dep(reinterpret_cast<const uint2 *>(from));
        else
          x[u].x = load_dep(reinterpret_cast<const uint32_t *>(from));
      }
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      if (size[u] == 16)
        *reinterpret_cast<uint4 *>(to[u]) = x[u];
      else if (size[u] == 8)
        *reinterpret_cast<uint2 *>(to[u]) = make_uint2(x[u].x, x[u].y);
      else if (size[u] == 4)
        *reinterpret_cast<uint32_t *>(to[u]) = x[u].x;
    }
  }
}

// ---------------------------------------------------------------------------
// counts

// A page's count, changed by others of this grid meanwhile.
__device__ __forceinline__ int count_of(const PoolParams &p, int e) { return __ldcg(p.counts + e); }

// One entry of page e less; what is kept stays, and a count that is zero although an
// entry holds the page is reported and left.  Every thread that finds no count to take
// undoes its own step, so that a count ends right however many are at it: of those that
// are too many for it, the first finds the zero.  (No count is above 2^30: such a value
// is the lowest number, less the steps under way.)
__device__ __forceinline__ int take_count(const PoolParams &p, int e) { return atomicAdd(p.counts + e, -1); }
__device__ __forceinline__ void taken(const PoolParams &p, int e, int c, unsigned &bad) {
  if (c > 0 && c <= 1 << 30) return;
  atomicAdd(p.counts + e, 1);
  if (c == 0) bad |= VAE4_STATUS_BAD_COUNT;
}
__device__ __forceinline__ void drop_count(const PoolParams &p, int e, unsigned &bad) {
  taken(p, e, take_count(p, e), bad);
}

// The same for `by` entries more, where the count was c.
__device__ __forceinline__ void add_count(const PoolParams &p, int e, int c, int by, unsigned &bad) {
  if (c > 0 && c <= 1 << 30)
    atomicAdd(p.counts + e, by);
  else if (c == 0)
    bad |= VAE4_STATUS_BAD_COUNT;
}

__device__ __forceinline__ void report(uint32_t *status, unsigned bad) {
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad && status && (threadIdx.x & 31) == 0) atomicOr(status, bad);
}

// ---------------------------------------------------------------------------
// fork: row b <- row parents[b].
//
// A CTA takes all rows of some columns into shared memory before it writes any, so
// rows may change places.  An entry of a row with m children counts m - 1 more.
constexpr int kForkThreads = 512;

__global__ void __launch_bounds__(kForkThreads) fork_pages_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int smem[];
  const PoolParams &o = p.pool;
  const int W = p.width, B = o.B, tid = threadIdx.x;
  int *parent = smem, *kids = smem + B, *tile = smem + 2 * B;  // [B][W]
  for (int b = tid; b < B; b += kForkThreads) kids[b] = 0;
  __syncthreads();
  await_previous();
  unsigned bad = 0;
  const int c0 = blockIdx.x * W, log_w = __ffs(W) - 1;
  for (int x = tid; x < B << log_w; x += kForkThreads) {
    const int b = x >> log_w, c = c0 + (x & (W - 1));
    tile[x] = c < o.cols ? load_dep(o.bt + b * o.bt_sb + c) : -1;
  }
  for (int b = tid; b < B; b += kForkThreads) {
    int from = load_dep(p.parents + b);
    if (from < -1 || from >= B) {
      bad |= VAE4_STATUS_BAD_PARENT;
      from = b;  // the row stays
    }
    parent[b] = from;
    if (from >= 0) atomicAdd(kids + from, 1);
  }
  __syncthreads();
  // (counts of four entries per thread are on their way at once: one entry after another,
  // 256 rows of 2047 entries took 12.9 us instead of 10.9)
  for (int x0 = tid; x0 < B << log_w; x0 += 4 * kForkThreads) {
    int c[4], e[4], more[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = x0 + u * kForkThreads;
      e[u] = -1;
      if (x < B << log_w) {
        e[u] = tile[x];
        more[u] = kids[x >> log_w] - 1;
        if (e[u] < -1 || e[u] >= o.n_pages) {
          bad |= VAE4_STATUS_BAD_BLOCK;
          e[u] = -1;
        }
        if (more[u] == 0) e[u] = -1;
      }
      if (e[u] >= 0) c[u] = more[u] < 0 ? take_count(o, e[u]) : count_of(o, e[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e[u] >= 0) {
        if (more[u] < 0)
          taken(o, e[u], c[u], bad);
        else
          add_count(o, e[u], c[u], more[u], bad);
      }
  }
  for (int x = tid; x < B << log_w; x += kForkThreads) {
    const int b = x >> log_w, c = c0 + (x & (W - 1)), from = parent[b];
    if (from != b && c < o.cols) o.bt[b * o.bt_sb + c] = from >= 0 ? tile[(from << log_w) + (x & (W - 1))] : -1;
  }
  report(o.status, bad);
}

// ---------------------------------------------------------------------------
// resize and compact: one cluster, whose warps share the table's entries and the
// pages evenly in ascending ranges.  Between steps that read what others wrote the
// cluster meets (its barrier orders their memory); ranks across the cluster are
// exchanged through distributed shared memory.  A small pool is a chain of reads, meetings
// and atomics: 13 us for 8 rows of 64 entries, 11 to 13 for 64 moves.
constexpr int kPoolThreads = 1024, kPoolCtas = 8;
constexpr int kPoolWarps = kPoolThreads / 32 * kPoolCtas;
// Entries and pages (compaction: entries) up to which a cluster takes all steps.  Resize, a page
// more for each row: 17 us against 31 at 2^15 entries and pages, 25 against 31 at 2^16, 25 against
// 29 at 2^17, 40 against 31 at 2^18.  Compaction, an eighth of the pages at most: 15.0 against
// 15.0 at 2^14 entries beside as many pages, 17 against 16 at 2^15, 21 against 18 at 2^16.
constexpr int64_t kSmallPool = 1 << 15;

struct ClusterSums {
  int2 warp[kPoolThreads / 32];
  int2 cta[kPoolCtas];
};

// Sums of a pair over all warps of the cluster (returned), and over those before
// this one (*before).  Every thread calls it; `s` is used once.
__device__ __forceinline__ int2 cluster_sums(ClusterSums &s, int2 mine, int2 *before) {
  cg::cluster_group cl = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)cl.block_rank();
  if (lane == 0) s.warp[warp] = mine;
  __syncthreads();
  const int2 w = s.warp[lane];
  if (warp == 0) {
    const int2 t = make_int2((int)__reduce_add_sync(0xffffffffu, (unsigned)w.x),
                             (int)__reduce_add_sync(0xffffffffu, (unsigned)w.y));
    if (lane < kPoolCtas) *cl.map_shared_rank(&s.cta[rank], lane) = t;
  }
  cl.sync();
  const int2 c = lane < kPoolCtas ? s.cta[lane] : make_int2(0, 0);
  const int2 bw = lane < warp ? w : make_int2(0, 0), bc = lane < rank ? c : make_int2(0, 0);
  before->x = (int)__reduce_add_sync(0xffffffffu, (unsigned)(bw.x + bc.x));
  before->y = (int)__reduce_add_sync(0xffffffffu, (unsigned)(bw.y + bc.y));
  return make_int2((int)__reduce_add_sync(0xffffffffu, (unsigned)c.x),
                   (int)__reduce_add_sync(0xffffffffu, (unsigned)c.y));
}

// The warp's share of n things: [x, y), x and y multiples of 32 (but for y = n).
__device__ __forceinline__ int2 share(int64_t n, int gwarp, int warps = kPoolWarps) {
  const int64_t per = (n + warps * 32 - 1) / (warps * 32) * 32;
  return make_int2((int)min(n, gwarp * per), (int)min(n, (gwarp + 1) * per));
}

// f(index, value) over the warp's share of the table's entries, row after row;
// every lane calls it, an index past the share with value -2
constexpr int kBatch = 8;  // loads in flight per thread
template <class F>
__device__ __forceinline__ void each_entry(const PoolParams &o, int2 part, F f) {
  const int lane = threadIdx.x & 31;
  for (int x0 = part.x; x0 < part.y; x0 += 32 * kBatch) {
    int e[kBatch], b[kBatch], j[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int x = x0 + 32 * u + lane;
      b[u] = (int)((unsigned)x / (unsigned)o.cols);
      j[u] = x - b[u] * o.cols;
      e[u] = x < part.y ? __ldcg(o.bt + b[u] * o.bt_sb + j[u]) : -2;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (x0 + 32 * u < part.y) f(b[u], j[u], e[u], x0 + 32 * u + lane < part.y);
  }
}
// f(page, count, in the share) over the warp's share of the pages
template <class F>
__device__ __forceinline__ void each_page(const PoolParams &o, int2 part, F f) {
  const int lane = threadIdx.x & 31;
  for (int x0 = part.x; x0 < part.y; x0 += 32 * kBatch) {
    int c[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int x = x0 + 32 * u + lane;
      c[u] = x < part.y ? count_of(o, x) : 0;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (x0 + 32 * u < part.y) f(x0 + 32 * u + lane, c[u], x0 + 32 * u + lane < part.y);
  }
}

// resize: pages past a row's length go back; then entries without a page and
// written entries of pages that others hold too get the lowest free ones.
//
// The steps, each of which needs what all warps did in the one before.  A small pool
// takes them in one launch of a cluster, a large one in a chain of dependent launches of
// the whole GPU.
struct Resize {
  const ResizeParams &p;
  const int2 *row;  // (pages, first page written) of each row; pages = -1: the row stays
  int2 part, ids;   // the warp's entries and pages
  int lane;
  unsigned below;

  __device__ __forceinline__ Resize(const ResizeParams &q, const int2 *r, int gwarp, int warps)
      : p(q), row(r), part(share((int64_t)q.pool.B * q.pool.cols, gwarp, warps)),
        ids(share(q.pool.n_pages, gwarp, warps)), lane(threadIdx.x & 31), below((1u << lane) - 1u) {}

  // Rows of the table into shared memory; with `copies`, the list of copies is emptied.
  static __device__ __forceinline__ void rows(const ResizeParams &p, int2 *row, bool copies, unsigned &bad) {
    for (int b = threadIdx.x; b < p.pool.B; b += kPoolThreads) {
      const int32_t *s = p.seq + (int64_t)b * p.seq_sb;
      const int L = load_dep(s), q = p.seq_has_qlen ? load_dep(s + 1) : 0;
      int2 r = make_int2(-1, 0);
      if (L < 0 || L > p.pool.cols * p.page)
        bad |= VAE4_STATUS_BAD_LENGTH;
      else if (q < 0 || q > L)
        bad |= VAE4_STATUS_BAD_QLEN;
      else
        r = make_int2((L + p.page - 1) / p.page, q > 0 ? (L - q) / p.page : p.pool.cols);
      row[b] = r;
      if (copies) {
        p.copies[b * p.copies_sb] = -1;
        p.copies[b * p.copies_sb + 1] = -1;
      }
    }
    __syncthreads();
  }

  __device__ __forceinline__ void release(unsigned &bad) const {
    each_entry(p.pool, part, [&](int b, int j, int e, bool in) {
      if (!in) return;
      if (e < -1 || e >= p.pool.n_pages) {
        bad |= VAE4_STATUS_BAD_BLOCK;
      } else if (row[b].x >= 0 && j >= row[b].x && e >= 0) {
        p.pool.bt[b * p.pool.bt_sb + j] = -1;
        drop_count(p.pool, e, bad);
      }
    });
  }

  // Does the entry need a page?  Evaluated twice, with no count changed in between that
  // an entry of the table holds.
  __device__ __forceinline__ bool needs(int b, int j, int e, bool in) const {
    if (!in || j >= row[b].x) return false;
    if (e == -1) return true;
    if (e < 0 || e >= p.pool.n_pages || j < row[b].y) return false;
    const int c = count_of(p.pool, e);
    return c > 1 || c < 0;
  }

  __device__ __forceinline__ int2 count() const {  // (entries that need one, free pages)
    int2 mine = make_int2(0, 0);
    each_entry(p.pool, part, [&](int b, int j, int e, bool in) {
      mine.x += __popc(__ballot_sync(0xffffffffu, needs(b, j, e, in)));
    });
    each_page(p.pool, ids, [&](int, int c, bool in) {
      mine.y += __popc(__ballot_sync(0xffffffffu, in && c == 0));
    });
    return mine;
  }

  // The free pages in order, as many as are needed.
  __device__ __forceinline__ void list(int at, int served) const {
    if (at >= served) return;
    each_page(p.pool, ids, [&](int x, int c, bool in) {
      const unsigned m = __ballot_sync(0xffffffffu, in && c == 0);
      const int r = at + __popc(m & below);
      if (in && c == 0 && r < served) __stcg(p.list + r, x);
      at += __popc(m);
    });
  }

  __device__ __forceinline__ void assign(int at, int served, int mine) const {
    if (mine == 0 || at >= served) return;
    each_entry(p.pool, part, [&](int b, int j, int e, bool in) {
      const bool want = needs(b, j, e, in);
      const unsigned m = __ballot_sync(0xffffffffu, want);
      const int r = at + __popc(m & below);
      at += __popc(m);
      if (!want || r >= served) return;
      const int id = __ldcg(p.list + r);
      __stcg(p.list + r, e);  // the page that it gives up, counted down by settle()
      p.pool.bt[b * p.pool.bt_sb + j] = id;
      __stcg(p.pool.counts + id, 1);
      if (e < 0 || j != row[b].y) return;
      const int32_t *s = p.seq + (int64_t)b * p.seq_sb;
      if ((load_dep(s) - load_dep(s + 1)) % p.page != 0) {
        p.copies[b * p.copies_sb] = e;
        p.copies[b * p.copies_sb + 1] = id;
      }
    });
  }

  static __device__ __forceinline__ void settle(const ResizeParams &p, int thread, int threads, int served,
                                                unsigned &bad) {
    for (int r = thread; r < served; r += threads) {
      const int e = __ldcg(p.list + r);
      if (e >= 0) drop_count(p.pool, e, bad);
    }
  }
};

__global__ void __launch_bounds__(kPoolThreads, 1)
    resize_pages_kernel(const __grid_constant__ ResizeParams p) {
  extern __shared__ int2 row[];
  __shared__ ClusterSums sums;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cl.block_rank();
  await_previous();
  unsigned bad = 0;
  Resize::rows(p, row, rank == 0, bad);
  const Resize x(p, row, rank * (kPoolThreads / 32) + (tid >> 5), kPoolWarps);
  x.release(bad);
  cl.sync();
  const int2 mine = x.count();
  int2 before;
  const int2 total = cluster_sums(sums, mine, &before);
  const int served = min(total.x, total.y);
  if (total.x > total.y) bad |= VAE4_STATUS_NO_PAGES;
  x.list(before.y, served);
  cl.sync();
  x.assign(before.x, served, mine.x);
  cl.sync();
  Resize::settle(p, rank * kPoolThreads + tid, kPoolCtas * kPoolThreads, served, bad);
  report(p.pool.status, bad);
}

// The same steps, a launch each.  Sums of the warps' pairs over the grid (returned), and
// over the warps before this one.
__device__ __forceinline__ int2 grid_sums(const int2 *sums, int2 *before) {
  __shared__ int4 red[kPoolThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = gridDim.x * (kPoolThreads / 32), first = blockIdx.x * (kPoolThreads / 32);
  int4 v = make_int4(0, 0, 0, 0);  // all, those of earlier CTAs
  for (int w = tid; w < n; w += kPoolThreads) {
    const int2 t = __ldcg(sums + w);
    v.x += t.x;
    v.y += t.y;
    if (w < first) {
      v.z += t.x;
      v.w += t.y;
    }
  }
  auto sum = [](int x) -> int { return (int)__reduce_add_sync(0xffffffffu, (unsigned)x); };
  v = make_int4(sum(v.x), sum(v.y), sum(v.z), sum(v.w));
  if (lane == 0) red[warp] = v;
  const int2 own = __ldcg(sums + first + lane);
  __syncthreads();
  const int4 r = red[lane];
  const int2 b = lane < warp ? own : make_int2(0, 0);
  *before = make_int2(sum(r.z + b.x), sum(r.w + b.y));
  return make_int2(sum(r.x), sum(r.y));
}

template <int STEP>
__global__ void __launch_bounds__(kPoolThreads, 1)
    resize_step_kernel(const __grid_constant__ ResizeParams p) {
  extern __shared__ int2 row[];
  const int gwarp = blockIdx.x * (kPoolThreads / 32) + ((int)threadIdx.x >> 5);
  await_previous();
  unsigned bad = 0, seen = 0;
  if (STEP == 0 || STEP == 1 || STEP == 3) Resize::rows(p, row, STEP == 0 && blockIdx.x == 0, seen);
  if (STEP == 0 && blockIdx.x == 0) bad = seen;
  const Resize x(p, row, gwarp, (int)gridDim.x * (kPoolThreads / 32));
  if (STEP == 0) x.release(bad);
  if (STEP == 1) {
    const int2 mine = x.count();
    if ((threadIdx.x & 31) == 0) __stcg(p.sums + gwarp, mine);
  }
  if (STEP >= 2) {
    int2 before;
    const int2 total = grid_sums(p.sums, &before);
    const int served = min(total.x, total.y);
    if (STEP == 2) {
      if (total.x > total.y) bad |= VAE4_STATUS_NO_PAGES;
      x.list(before.y, served);
    }
    if (STEP == 3) x.assign(before.x, served, __ldcg(p.sums + gwarp).x);
    if (STEP == 4)
      Resize::settle(p, blockIdx.x * kPoolThreads + threadIdx.x, gridDim.x * kPoolThreads, served, bad);
  }
  report(p.pool.status, bad);
}

// compact: with n pages in use, the highest pages with id >= n go to the lowest free
// ones below n.  A page that moves leaves its rank in the place of its count until
// the table's entries have been looked up there: by the same cluster, or (SPLIT, for a
// large table) by launches of the whole GPU behind it.
__device__ __forceinline__ void look_up(const CompactParams &p, int b, int j, int e, int moved, unsigned &bad) {
  if (e < -1 || e >= p.pool.n_pages) {
    bad |= VAE4_STATUS_BAD_BLOCK;
  } else if (e >= 0) {
    const int r = (int)((unsigned)count_of(p.pool, e) ^ 0x80000000u);
    // (a kept page's count may look like a rank)
    if (r >= 0 && r < moved && __ldcg(p.moves + r * p.moves_sb) == e)
      p.pool.bt[b * p.pool.bt_sb + j] = __ldcg(p.moves + r * p.moves_sb + 1);
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kPoolThreads, 1)
    compact_pages_kernel(const __grid_constant__ CompactParams p) {
  __shared__ ClusterSums sums[2];
  cg::cluster_group cl = cg::this_cluster();
  const PoolParams &o = p.pool;
  const int tid = threadIdx.x, lane = tid & 31, rank = (int)cl.block_rank();
  const int gwarp = rank * (kPoolThreads / 32) + (tid >> 5);
  const unsigned below = (1u << lane) - 1u;
  cl.sync();  // every CTA of the cluster runs, before any is written to
  await_previous();
  const int2 ids = share(o.n_pages, gwarp);
  int2 mine = make_int2(0, 0), before;  // (pages in use, pages that may move)
  each_page(o, ids, [&](int, int c, bool in) {
    mine.x += __popc(__ballot_sync(0xffffffffu, in && c != 0));
    mine.y += __popc(__ballot_sync(0xffffffffu, in && c > 0));
  });
  const int n = cluster_sums(sums[0], mine, &before).x;
  // holes below n and pages to move from n on
  if (ids.y <= n) {
    mine = make_int2(ids.y - ids.x - mine.x, 0);
  } else if (ids.x >= n) {
    mine.x = 0;
  } else {
    mine = make_int2(0, 0);
    each_page(o, ids, [&](int x, int c, bool in) {
      mine.x += __popc(__ballot_sync(0xffffffffu, in && c == 0 && x < n));
      mine.y += __popc(__ballot_sync(0xffffffffu, in && c > 0 && x >= n));
    });
  }
  const int2 total = cluster_sums(sums[1], mine, &before);
  const int moved = min(p.n, total.y);  // (no fewer holes than pages to move)
  if (mine.x > 0 && before.x < moved) {
    int at = before.x;
    each_page(o, ids, [&](int x, int c, bool in) {
      const bool hole = in && c == 0 && x < n;
      const unsigned m = __ballot_sync(0xffffffffu, hole);
      const int r = at + __popc(m & below);
      if (hole && r < moved) __stcg(p.moves + r * p.moves_sb + 1, x);
      at += __popc(m);
    });
  }
  if (mine.y > 0 && total.y - before.y - mine.y < moved) {
    int at = total.y - before.y;  // ranks descend with the id
    each_page(o, ids, [&](int x, int c, bool in) {
      const bool goes = in && c > 0 && x >= n;
      const unsigned m = __ballot_sync(0xffffffffu, goes);
      const int r = at - 1 - __popc(m & below);
      if (goes && r < moved) __stcg(p.moves + r * p.moves_sb, x);
      at -= __popc(m);
    });
  }
  const int first = rank * kPoolThreads + tid;
  for (int r = moved + first; r < p.n; r += kPoolCtas * kPoolThreads) {
    __stcg(p.moves + r * p.moves_sb, -1);
    __stcg(p.moves + r * p.moves_sb + 1, -1);
  }
  // (the same for the whole cluster, and no remote access is left; without moves the
  // table's entries are looked at for the status alone)
  if (moved == 0 && (SPLIT || !o.status)) return;
  cl.sync();
  for (int r = first; r < moved; r += kPoolCtas * kPoolThreads) {
    const int from = __ldcg(p.moves + r * p.moves_sb), to = __ldcg(p.moves + r * p.moves_sb + 1);
    __stcg(o.counts + to, count_of(o, from));
    __stcg(o.counts + from, INT32_MIN + r);
  }
  if (SPLIT) return;
  cl.sync();
  unsigned bad = 0;
  each_entry(o, share((int64_t)o.B * o.cols, gwarp), [&](int b, int j, int e, bool in) {
    if (in) look_up(p, b, j, e, moved, bad);
  });
  report(o.status, bad);
  cl.sync();
  for (int r = first; r < moved; r += kPoolCtas * kPoolThreads)
    __stcg(o.counts + __ldcg(p.moves + r * p.moves_sb), 0);
}

__global__ void __launch_bounds__(kPoolThreads) compact_table_kernel(const __grid_constant__ CompactParams p) {
  await_previous();
  // nothing moves, and nobody asks for invalid entries
  if (!p.pool.status && (p.n == 0 || load_dep(p.moves) < 0)) return;
  unsigned bad = 0;
  const int warps = gridDim.x * (kPoolThreads / 32), gwarp = blockIdx.x * (kPoolThreads / 32) + (threadIdx.x >> 5);
  each_entry(p.pool, share((int64_t)p.pool.B * p.pool.cols, gwarp, warps), [&](int b, int j, int e, bool in) {
    if (in) look_up(p, b, j, e, p.n, bad);
  });
  report(p.pool.status, bad);
}

__global__ void __launch_bounds__(256) compact_counts_kernel(const __grid_constant__ CompactParams p) {
  await_previous();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= p.n) return;
  const int e = load_dep(p.moves + r * p.moves_sb);
  if (e >= 0) p.pool.counts[e] = 0;
}

// The limit of a kernel's dynamic shared memory, raised once per context to the most
// that any call needs (as for the visit lists).  The 48 KB that every launch may have are
// for a kernel's static arrays too.
constexpr size_t kStaticSmem = 1024;  // at least what any of them declares
static_assert(sizeof(ClusterSums) + 64 <= kStaticSmem && kPoolThreads / 32 * sizeof(int4) <= kStaticSmem,
              "static shared memory");
template <auto Kernel>
cudaError_t allow_smem(size_t most, size_t smem) {
  if (smem + kStaticSmem <= 48 * 1024) return cudaSuccess;
  constexpr int kDevs = 64;
  static std::atomic<unsigned long long> configured[kDevs] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const unsigned long long ctx = current_context_id();
  if (dev >= 0 && dev < kDevs && ctx != 0 && configured[dev].load(std::memory_order_acquire) == ctx)
    return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess && dev >= 0 && dev < kDevs)
    configured[dev].store(current_context_id(), std::memory_order_release);
  return e;
}

template <class P>
cudaError_t launch_cluster(void (*kernel)(P), size_t smem, cudaStream_t stream, const P &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPoolCtas);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPoolCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyParams &p, cudaStream_t stream) {
  const int per = kCopyThreads * kCopyUnroll;
  const int parts = std::min((p.vecs + per - 1) / per, 65535);
  return launch_dependent(copy_pages_kernel, dim3((unsigned)p.n, (unsigned)parts), kCopyThreads, 0,
                          stream, p);
}

cudaError_t launch_fork_pages(const ForkParams &in, int num_sms, cudaStream_t stream) {
  constexpr int kMost = kMaxForkRows * (4 * 4 + 8);
  ForkParams p = in;
  const int B = p.pool.B;
  // 128-byte pieces of rows, but narrower ones until every SM has a CTA (32 bytes at
  // least) or the tile fits
  p.width = 32;
  while (p.width > 8 && (p.pool.cols + p.width - 1) / p.width < num_sms) p.width /= 2;
  while (p.width > 4 && B * (4 * p.width + 8) > kMost) p.width /= 2;
  const size_t smem = (size_t)B * (4 * p.width + 8);
  const cudaError_t e = allow_smem<fork_pages_kernel>(kMost, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(fork_pages_kernel, dim3((unsigned)((p.pool.cols + p.width - 1) / p.width)),
                          kForkThreads, smem, stream, p);
}

cudaError_t launch_resize_pages(const ResizeParams &p, cudaStream_t stream) {
  const size_t smem = (size_t)p.pool.B * sizeof(int2), most = kMaxResizeRows * sizeof(int2);
  cudaError_t e;
  // (256 rows of 2047 entries, 246 thousand pages: 29 us, on a cluster 93)
  if ((int64_t)p.pool.B * p.pool.cols + p.pool.n_pages <= kSmallPool) {
    if ((e = allow_smem<resize_pages_kernel>(most, smem)) != cudaSuccess) return e;
    return launch_cluster(resize_pages_kernel, smem, stream, p);
  }
  if ((e = allow_smem<resize_step_kernel<0>>(most, smem)) != cudaSuccess) return e;
  if ((e = allow_smem<resize_step_kernel<1>>(most, smem)) != cudaSuccess) return e;
  if ((e = allow_smem<resize_step_kernel<3>>(most, smem)) != cudaSuccess) return e;
  const dim3 grid(kPoolGrid);
  if ((e = launch_dependent(resize_step_kernel<0>, grid, kPoolThreads, smem, stream, p)) != cudaSuccess) return e;
  if ((e = launch_dependent(resize_step_kernel<1>, grid, kPoolThreads, smem, stream, p)) != cudaSuccess) return e;
  if ((e = launch_dependent(resize_step_kernel<2>, grid, kPoolThreads, 0, stream, p)) != cudaSuccess) return e;
  if ((e = launch_dependent(resize_step_kernel<3>, grid, kPoolThreads, smem, stream, p)) != cudaSuccess) return e;
  return launch_dependent(resize_step_kernel<4>, grid, kPoolThreads, 0, stream, p);
}

cudaError_t launch_compact_pages(const CompactParams &p, cudaStream_t stream) {
  if (p.n == 0) return launch_dependent(compact_table_kernel, dim3(kPoolGrid), kPoolThreads, 0, stream, p);
  // (32 rows of 16384 entries, 16384 moves: 34 us, on a cluster 70)
  if ((int64_t)p.pool.B * p.pool.cols <= kSmallPool)
    return launch_cluster(compact_pages_kernel<false>, 0, stream, p);
  cudaError_t e = launch_cluster(compact_pages_kernel<true>, 0, stream, p);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(compact_table_kernel, dim3(kPoolGrid), kPoolThreads, 0, stream, p)) != cudaSuccess)
    return e;
  return launch_dependent(compact_counts_kernel, dim3((unsigned)((p.n + 255) / 256)), 256, 0, stream, p);
}

}  // namespace vae4
