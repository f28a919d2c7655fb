// Choice of blocks: for query i and KV head h with v visible blocks, the k
// blocks to attend to, in ascending order: the first `sink` and the last
// `local` of the visible ones, then the highest scores among the others,
// ties by the lowest index (a NaN ranks with -inf).  All v blocks if v <= k;
// places past the last choice hold -1.
//
// Radix selection, one CTA per row: scores map to unsigned keys of the same
// order; up to three passes over the candidates (11, 11 and 10 bits)
// histogram the keys that agree with the digits found so far and find the
// digit in which the m-th largest lies, so that at the end the m-th largest
// key itself and the number of its equals to take are known (a pass that
// leaves no choice ends the search).  Then the chosen indices are written in
// order.
//
// A warp owns a contiguous segment of the row and each of its lanes every
// 32nd key of it, in registers where the row allows (up to kKeys per lane):
// the row is then read once, and votes leave one bit per place in shared
// memory, whose words a thread each counts and writes.  Longer rows are read
// again in each pass, and every warp counts and then writes its segment.
//
// The steps of the search bound it, not the bytes (4 per score): histogram,
// scan over the bins, next digit, each behind a barrier and each over all keys
// of the row.  16 rows of 4096 blocks take 4.8 us, 256 rows of up to 16384 blocks
// 14.6 us (of which reading the row is a third).  Rows past 16384 blocks are read
// again in each pass: 256 rows of 16384 13.7 us, of 16400 29.2, of 25000 43.2; two
// rows 8.6, 17.0 and 22.6, of 100000 97.
#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kBins = 2048;

// unsigned keys in the order of the scores; -0 and 0 are equal, NaN = -inf
__device__ __forceinline__ uint32_t score_key(float x) {
  x = x == x ? x + 0.f : -__int_as_float(0x7f800000);
  const int u = __float_as_int(x);
  return (uint32_t)(u ^ (u >> 31 | (int)0x80000000));
}

// kKeys > 0: rows of up to kThreads * kKeys blocks, in registers; 0: any row
template <int kThreads, int kKeys, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) select_blocks_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kOwn = kBins / kThreads;  // bins per thread
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wsum[kWarps], weq[kWarps];
  __shared__ uint32_t pick[3];  // digit of the m-th largest, rank left in it, its count
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int32_t *ids = p.ids + (int64_t)b * p.i_sb + (int64_t)i * p.i_si + (int64_t)h * p.i_sh;
  await_previous();
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool bad_l = L < 0 || (L > 0 && (L - 1) / p.blk >= p.cols);
  const bool bad = bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L);
  if (bad && i == 0 && h == 0 && tid == 0 && p.status)
    atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
  const int v = bad || L == 0 || i >= n ? 0 : (L - n + i) / p.blk + 1;  // visible blocks
  if (v <= p.k) {
    for (int x = tid; x < p.k; x += kThreads) ids[x] = x < v ? x : -1;
    return;
  }
  const float *sc = p.scores + (int64_t)b * p.s_sb + (int64_t)i * p.s_si + (int64_t)h * p.s_sh;
  const int c0 = p.sink, c1 = v - p.local;  // candidates
  const int seg = ((v + kWarps - 1) / kWarps + 31) & ~31;  // a warp's segment
  const int x0 = min(warp * seg, v), x1 = min(x0 + seg, v);
  // key of a candidate; all ones for a forced place, 0 past the row's end (no
  // score maps to either)
  auto key_of = [&](int x, float score) -> uint32_t {
    return x >= x1 ? 0u : x >= c0 && x < c1 ? score_key(score) : 0xFFFFFFFFu;
  };
  uint32_t key[kKeys > 0 ? kKeys : 1];
  if constexpr (kKeys > 0) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e)  // all under way together
      key[e] = __float_as_uint(load_dep(sc + min(x0 + 32 * e + lane, v - 1)));
    if (x0 >= c0 && x0 + 32 * kKeys <= min(x1, c1)) {  // candidates alone
#pragma unroll
      for (int e = 0; e < kKeys; ++e) key[e] = score_key(__uint_as_float(key[e]));
    } else {
#pragma unroll
      for (int e = 0; e < kKeys; ++e) key[e] = key_of(x0 + 32 * e + lane, __uint_as_float(key[e]));
    }
  }
  auto each_key = [&](auto &&f) {
    if constexpr (kKeys > 0) {
#pragma unroll
      for (int e = 0; e < kKeys; e += 4) {
        if (32 * e >= x1 - x0) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) f(x0 + 32 * (e + k) + lane, key[e + k]);
      }
    } else {
      for (int x = x0; x < x1; x += 32) f(x + lane, key_of(x + lane, load_dep(sc + min(x + lane, v - 1))));
    }
  };
  uint32_t m = (uint32_t)(p.k - p.sink - p.local);  // how many of them (fewer than there are)
  uint32_t prefix = 0u, mask = 0u;
  bool all_equal = m == 0;  // m == 0: no candidate is chosen
  for (int pass = 0; pass < 3 && !all_equal; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 0x3FFu : 0x7FFu;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) hist[tid + e * kThreads] = 0u;
    __syncthreads();
    if (pass == 0)
      each_key([&](int, uint32_t u) {
        if (u + 1u > 1u) atomicAdd(&hist[u >> 21], 1u);  // a candidate
      });
    else  // (the first digits of the two other values are no score's)
      each_key([&](int, uint32_t u) {
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & digits], 1u);
      });
    __syncthreads();
    // thread t owns kOwn bins; counts of all higher bins by a suffix scan
    uint32_t own[kOwn], sum = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) sum += own[e] = hist[kOwn * tid + e];
    uint32_t suf = sum;  // over this and the higher lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_down_sync(0xffffffffu, suf, o);
      if (lane + o < 32) suf += t;
    }
    if (lane == 0) wsum[warp] = suf;
    __syncthreads();
    // (the sums of the higher warps, one per lane)
    suf += __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? wsum[lane] : 0u);
    uint32_t above = suf - sum;  // candidates in bins past the thread's
#pragma unroll
    for (int e = kOwn - 1; e >= 0; --e) {
      if (above < m && m <= above + own[e]) {
        pick[0] = kOwn * tid + e;
        pick[1] = m - above;
        pick[2] = own[e];
      }
      above += own[e];
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    mask |= digits << shift;
    m = pick[1];
    all_equal = pick[2] == m;  // every key of the digit is chosen
    __syncthreads();
  }
  // chosen: the forced places and the keys above the digits found, and of those
  // that agree with them the first m.  (With no place for candidates, mask = 0,
  // only the forced places.)  Few places of a row are chosen, so one vote passes
  // over most of it.
  if (mask == 0u) {
    mask = prefix = 0xFFFFFFFFu;
    m = 0xFFFFFFFFu;
  }
  if constexpr (kKeys > 0) {
    // a bit per place, chosen or agreeing, 32 places of a warp's segment a
    // word; then a thread per word counts, and the words' bits are written
    // behind what the scan over the CTA says
    constexpr int kWords = kThreads * kKeys / 32;
    static_assert(kWords <= kThreads && 2 * kWords <= kBins, "a thread per word");
    uint32_t *wg = hist, *we = hist + kWords;
    const int nw = (v + 31) / 32;
    // (lane e keeps word e of the segment)
    uint32_t bits_g = 0u, bits_e = 0u;
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      if (e % 4 == 0 && 32 * e >= x1 - x0) break;
      const uint32_t u = key[e] & mask;
      const unsigned any = __ballot_sync(0xffffffffu, u >= prefix);
      const unsigned eq = __ballot_sync(0xffffffffu, u == prefix);
      if (lane == e) {
        bits_g = any ^ eq;
        bits_e = eq;
      }
    }
    if (lane < kKeys && x0 + 32 * lane < x1) {
      wg[x0 / 32 + lane] = bits_g;
      we[x0 / 32 + lane] = bits_e;
    }
    __syncthreads();
    uint32_t bg = tid < nw ? wg[tid] : 0u, be = tid < nw ? we[tid] : 0u;
    const uint32_t ng = __popc(bg), ne = __popc(be);
    uint32_t ig = ng, ie = ne;  // over this and the lower words
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, ig, o), c = __shfl_up_sync(0xffffffffu, ie, o);
      if (lane >= o) {
        ig += a;
        ie += c;
      }
    }
    if (lane == 31) {
      wsum[warp] = ig;
      weq[warp] = ie;
    }
    __syncthreads();
    ig += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u) - ng;  // before this word
    ie += __reduce_add_sync(0xffffffffu, lane < warp ? weq[lane] : 0u) - ne;
    for (uint32_t both = bg | be; both != 0u; both &= both - 1) {
      const uint32_t bit = both & (~both + 1u);
      const bool same = (be & bit) != 0u;
      if (!same || ie < m) ids[ig + min(ie, m)] = 32 * tid + __ffs(bit) - 1;
      if (same)
        ++ie;
      else
        ++ig;
    }
    return;
  }
  uint32_t gt = 0, eq = 0;
  each_key([&](int, uint32_t u) {
    const unsigned any = __ballot_sync(0xffffffffu, (u & mask) >= prefix);
    if (any != 0u) {
      const unsigned e = __ballot_sync(0xffffffffu, (u & mask) == prefix);
      eq += __popc(e);
      gt += __popc(any ^ e);
    }
  });
  if (lane == 0) {
    wsum[warp] = gt;
    weq[warp] = eq;
  }
  __syncthreads();
  uint32_t base_gt = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u);
  uint32_t base_eq = __reduce_add_sync(0xffffffffu, lane < warp ? weq[lane] : 0u);
  each_key([&](int x, uint32_t u) {
    const bool in = (u & mask) >= prefix;
    const unsigned any = __ballot_sync(0xffffffffu, in);
    if (any != 0u) {
      const bool same = (u & mask) == prefix;
      const unsigned be = __ballot_sync(0xffffffffu, same), bg = any ^ be;
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t gr = base_gt + __popc(bg & below), e = base_eq + __popc(be & below);
      if (in && (!same || e < m)) ids[gr + min(e, m)] = x;
      base_gt += __popc(bg);
      base_eq += __popc(be);
    }
  });
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams &p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.Qmax, (unsigned)p.Hkv, (unsigned)p.B);
  // a row has at most `cols` blocks: a CTA that holds it in registers, of threads
  // enough that each has few keys and few enough that a scan's barriers are short
  // (16 rows of 4096 blocks: 5.7 us with 256 threads, 4.7 with 512, 4.8 to 5.2 with
  // 1024; 256 rows of 16384: 14.5 with 512, 16 and more with 1024)
  if (p.cols <= 256 * 8)
    return launch_dependent(select_blocks_kernel<256, 8, 4>, grid, 256, 0, stream, p);
  if (p.cols <= 512 * 8)
    return launch_dependent(select_blocks_kernel<512, 8, 2>, grid, 512, 0, stream, p);
  if (p.cols <= 1024 * 8)
    return launch_dependent(select_blocks_kernel<1024, 8, 1>, grid, 1024, 0, stream, p);
  if (p.cols <= 512 * 32)
    return launch_dependent(select_blocks_kernel<512, 32, 2>, grid, 512, 0, stream, p);
  return launch_dependent(select_blocks_kernel<1024, 0, 2>, grid, 1024, 0, stream, p);
}

}  // namespace vae4
