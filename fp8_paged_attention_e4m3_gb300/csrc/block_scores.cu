// Block scores: for query i and KV head h, an upper bound of the logits any
// of the group's heads can have in block j, from the block's bounds of K
// (lo_d, hi_d in the cache's codes):
//     u[g] = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d
//     score = softmax_scale * s_K[j] * max_g u[g]
// FP32 sums of exact FP16 x FP8 products.  Blocks that query i does not see
// (their first token lies past its position) score -inf.
//
// One warp per block, the lanes over the channels.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kScoreThreads = 128;

template <int D, bool E5M2>
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(const ScoreParams p) {
  constexpr int CPL = D / 32;  // channels per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool long_l = L > 0 && (L - 1) / p.blk >= p.cols;  // more blocks than columns
  const bool bad_l = L < 0 || (int64_t)L > (int64_t)p.max_pages * p.nb * p.blk || long_l;
  if (bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L)) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && p.status)
      atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
    return;
  }
  const int nblk = L > 0 ? (L - 1) / p.blk + 1 : 0;
  const float ninf = -__int_as_float(0x7f800000);
  for (int j = blockIdx.x * (kScoreThreads / 32) + warp; j < nblk;
       j += gridDim.x * (kScoreThreads / 32)) {
    const int lp = j / p.nb, sub = j - lp * p.nb;
    const int phys = p.bt[(int64_t)b * p.bt_sb + lp];
    const bool ok = phys >= 0 && phys < p.n_pages;
    if (!ok && lane == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    float lo[CPL], hi[CPL], s = 0.f;
    if (ok) {
      const uint8_t *bd = p.bounds + (int64_t)phys * p.b_page + (int64_t)h * p.b_head + (int64_t)sub * p.b_blk;
#pragma unroll
      for (int k = 0; k < CPL; ++k) {
        const uint32_t a = fp8x2_to_f16x2<E5M2>(bd[lane + 32 * k] | (uint32_t)bd[p.b_mm + lane + 32 * k] << 8);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        lo[k] = f.x;
        hi[k] = f.y;
      }
      s = p.scales[(int64_t)phys * p.s_page + (int64_t)h * p.s_head + sub] * p.sm_scale;
    }
    for (int i = 0; i < n; ++i) {
      float best = ninf;
      for (int g = 0; g < p.G; ++g) {
        const __half *q = static_cast<const __half *>(p.q) + (int64_t)b * p.q_sb + (int64_t)i * p.q_si +
                          (int64_t)(h * p.G + g) * p.q_sh;
        float u = 0.f;
        if (ok) {
#pragma unroll
          for (int k = 0; k < CPL; ++k) {
            const float f = __half2float(q[lane + 32 * k]);
            u += fmaxf(f, 0.f) * hi[k] + fminf(f, 0.f) * lo[k];
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        best = fmaxf(best, u);
      }
      if (lane == 0) {
        const bool seen = (int64_t)j * p.blk <= L - n + i;
        p.scores[(int64_t)b * p.o_sb + (int64_t)i * p.o_si + (int64_t)h * p.o_sh + j] =
            ok && seen ? best * s : ninf;
      }
    }
  }
}

}  // namespace

cudaError_t launch_block_scores(const ScoreParams &p, bool e5m2, cudaStream_t stream) {
  const int per = kScoreThreads / 32;
  const int64_t rows = (int64_t)p.Hkv * p.B;
  int64_t gx = std::min<int64_t>(((int64_t)p.cols + per - 1) / per, 65535);
  gx = std::max<int64_t>(1, std::min<int64_t>(gx, (32768 + rows - 1) / rows));
  const dim3 grid((unsigned)gx, (unsigned)p.Hkv, (unsigned)p.B);
  switch (p.D * 2 + (e5m2 ? 1 : 0)) {
    case 128: block_scores_kernel<64, false><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 129: block_scores_kernel<64, true><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 256: block_scores_kernel<128, false><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 257: block_scores_kernel<128, true><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 512: block_scores_kernel<256, false><<<grid, kScoreThreads, 0, stream>>>(p); break;
    case 513: block_scores_kernel<256, true><<<grid, kScoreThreads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace vae4
