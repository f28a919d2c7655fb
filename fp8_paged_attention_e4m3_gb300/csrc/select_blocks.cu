// Choice of blocks: for query i and KV head h with v visible blocks, the k
// blocks to attend to, in ascending order: the first `sink` and the last
// `local` of the visible ones, then the highest scores among the others,
// ties by the lowest index (a NaN ranks with -inf).  All v blocks if v <= k;
// places past the last choice hold -1.
//
// Radix selection, one CTA per row: scores map to unsigned keys of the same
// order; three passes over the candidates (11, 11 and 10 bits) histogram the
// keys that agree with the digits found so far and find the digit in which
// the m-th largest lies, so that at the end the m-th largest key itself and
// the number of its equals to take are known.  A last pass writes the chosen
// indices in order: every warp counts and then writes a contiguous segment.
#include "common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// unsigned keys in the order of the scores; -0 and 0 are equal, NaN = -inf
__device__ __forceinline__ uint32_t score_key(float x) {
  x = x == x ? x + 0.f : -__int_as_float(0x7f800000);
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wsum[kSelWarps], wgt[kSelWarps], weq[kSelWarps];
  __shared__ uint32_t pick[2];  // digit of the m-th largest, rank left below it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int32_t *ids = p.ids + (int64_t)b * p.i_sb + (int64_t)i * p.i_si + (int64_t)h * p.i_sh;
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool bad_l = L < 0 || (L > 0 && (L - 1) / p.blk >= p.cols);
  const bool bad = bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L);
  if (bad && i == 0 && h == 0 && tid == 0 && p.status)
    atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
  const int v = bad || L == 0 || i >= n ? 0 : (L - n + i) / p.blk + 1;  // visible blocks
  if (v <= p.k) {
    for (int x = tid; x < p.k; x += kSelThreads) ids[x] = x < v ? x : -1;
    return;
  }
  const float *sc = p.scores + (int64_t)b * p.s_sb + (int64_t)i * p.s_si + (int64_t)h * p.s_sh;
  const int c0 = p.sink, c1 = v - p.local;  // candidates
  uint32_t m = (uint32_t)(p.k - p.sink - p.local);  // how many of them (fewer than there are)
  uint32_t prefix = 0xFFFFFFFFu, mask = 0u;
  if (m > 0) {
    prefix = 0u;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      for (int x = tid; x < kBins; x += kSelThreads) hist[x] = 0u;
      __syncthreads();
      for (int x = c0 + tid; x < c1; x += kSelThreads) {
        const uint32_t key = score_key(sc[x]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // thread t owns bins 4t .. 4t+3; counts of all higher bins by a suffix scan
      uint32_t own[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += own[e] = hist[4 * tid + e];
      uint32_t suf = sum;  // over this and the higher lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_down_sync(0xffffffffu, suf, o);
        if (lane + o < 32) suf += t;
      }
      if (lane == 0) wsum[warp] = suf;
      __syncthreads();
      for (int k = warp + 1; k < kSelWarps; ++k) suf += wsum[k];
      uint32_t above = suf - sum;  // candidates in bins past 4t+3
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        if (above < m && m <= above + own[e]) {
          pick[0] = 4 * tid + e;
          pick[1] = m - above;
        }
        above += own[e];
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= ((1u << bits) - 1u) << shift;
      m = pick[1];
      __syncthreads();
    }
  }
  // prefix: the m-th largest key; m: how many of its equals to take
  const int seg = ((v + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int x0 = min(warp * seg, v), x1 = min(x0 + seg, v);
  auto state = [&](int x) -> int {  // 0 no, 1 equal, 2 chosen
    if (x >= x1) return 0;
    if (x < c0 || x >= c1) return 2;
    if (mask == 0u) return 0;  // no place for candidates
    const uint32_t key = score_key(sc[x]);
    return key > prefix ? 2 : key == prefix ? 1 : 0;
  };
  uint32_t gt = 0, eq = 0;
  for (int x = x0; x < x1; x += 32) {
    const int s = state(x + lane);
    gt += __popc(__ballot_sync(0xffffffffu, s == 2));
    eq += __popc(__ballot_sync(0xffffffffu, s == 1));
  }
  if (lane == 0) {
    wgt[warp] = gt;
    weq[warp] = eq;
  }
  __syncthreads();
  uint32_t base_gt = 0, base_eq = 0;
  for (int k = 0; k < warp; ++k) {
    base_gt += wgt[k];
    base_eq += weq[k];
  }
  for (int x = x0; x < x1; x += 32) {
    const int s = state(x + lane);
    const uint32_t bg = __ballot_sync(0xffffffffu, s == 2), be = __ballot_sync(0xffffffffu, s == 1);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t g = base_gt + __popc(bg & below), e = base_eq + __popc(be & below);
    if (s == 2 || (s == 1 && e < m)) ids[g + min(e, m)] = x + lane;
    base_gt += __popc(bg);
    base_eq += __popc(be);
  }
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams &p, cudaStream_t stream) {
  const dim3 grid((unsigned)p.Qmax, (unsigned)p.Hkv, (unsigned)p.B);
  select_blocks_kernel<<<grid, kSelThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vae4
