// Block scores: for query i and KV head h, an upper bound of the logits any
// of the group's heads can have in block j, from the block's bounds of K
// (lo_d, hi_d in the cache's codes):
//     u[g] = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d
//     score = softmax_scale * s_K[j] * max_g u[g]
// FP32 sums of exact FP16 x FP8 products.  Blocks that query i does not see
// (their first token lies past its position) score -inf; a NaN or an infinite
// query gives what the sums give (NaN, mostly).  A block with an invalid page or
// scale scores -inf and is reported.
//
// u is a matrix product over 2 D channels, [hi | lo] of 16 blocks (rows of A)
// times [max(q, 0) | min(q, 0)] of the group's rows (columns of B): warp-level
// tensor-core products m16n8k16, one warp per 16 blocks.  The order of the
// channels is free as long as A and B agree, so a thread takes 16 consecutive
// bytes of a block's bounds as its share of four k-steps: A goes from memory
// to the fragments with one 16-byte load per 16 channels and no shared memory,
// and the matching share of B is 4 consecutive halves of a query's row.  With few
// rows a KV head the bytes of the bounds bound it (2 D per block and head, read
// once).  16 sequences of up to 131072 tokens, 8 heads of 128, blocks of 32: 91 MB
// in 20.1 us, 4.5 TB/s; what keeps it from the memory's rate is the start of the
// chain (page, queries and lengths, asked for together -> bounds -> products) and
// the ragged end, of a grid sized for the columns, not the lengths.  Eight queries
// of 6 heads of 256 over 262144 tokens, in blocks of 64, are that chain alone,
// 5.7 us.  More rows cost products and maxima: 16 sequences of up to 131072 tokens
// in blocks of 64, 8 KV heads of 128 with 6 query heads each, take 11.9 us with one
// query and 70.6 with sixteen (96 rows).
#include <algorithm>

#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;

// halves per row of B in shared memory: 16 bytes past a multiple of 32, so
// that the 16-byte reads of a quarter warp (2 rows, 4 chunks 32 bytes apart)
// fall on different banks
constexpr int b_stride(int D) { return D + 8; }
constexpr int score_smem(int D, int NT) {
  return 2 * NT * 8 * b_stride(D) * 2 + kScoreWarps * 16 * (NT * 8 + 1) * 4;
}

// the larger of two values; NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <int D, int NT, bool E5M2>
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(const ScoreParams p) {
  constexpr int BS = b_stride(D), RS = NT * 8 + 1;
  constexpr int NC = D / 64;  // 64-channel chunks of hi, and of lo
  extern __shared__ __align__(16) uint8_t smem[];
  __half *qs = reinterpret_cast<__half *>(smem);  // [2][NT * 8][BS]: max(q, 0), min(q, 0)
  float *us = reinterpret_cast<float *>(smem + 2 * NT * 8 * BS * 2) + (threadIdx.x >> 5) * 16 * RS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y / p.parts, b = blockIdx.z;
  const int i0 = (blockIdx.y - h * p.parts) * p.qn;  // first of the CTA's queries
  await_previous();
  // requested together: the lengths, the thread's first chunks of the queries
  // (padding rows are part of the tensor) and the page of its first block
  constexpr int kChunks = NT * 8 * (D / 8);
  auto query = [&](int x) -> uint4 {
    const int r = x / (D / 8), c = x - r * (D / 8), i = r / p.G;
    if (x >= kChunks || r >= p.qn * p.G || i0 + i >= p.Qmax) return make_uint4(0u, 0u, 0u, 0u);
    return load_dep(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p.q) + (int64_t)b * p.q_sb +
                                                 (int64_t)(i0 + i) * p.q_si +
                                                 (int64_t)(h * p.G + r - i * p.G) * p.q_sh + 8 * c));
  };
  constexpr int kQ = kChunks < 4 * kScoreThreads ? (kChunks + kScoreThreads - 1) / kScoreThreads : 4;
  uint4 qv[kQ];
#pragma unroll
  for (int e = 0; e < kQ; ++e) qv[e] = query(tid + e * kScoreThreads);
  int j0 = (blockIdx.x * kScoreWarps + warp) * 16;
  int phys = 0;
  if (const int lp = (j0 + lane) / p.nb; lane < 16 && lp < p.max_pages)
    phys = load_dep(p.bt + (int64_t)b * p.bt_sb + lp);
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool long_l = L > 0 && (L - 1) / p.blk >= p.cols;  // more blocks than columns
  const bool bad_l = L < 0 || (int64_t)L > (int64_t)p.max_pages * p.nb * p.blk || long_l;
  if (bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && p.status)
      atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
    return;
  }
  const int nblk = L > 0 && n > 0 ? (L - 1) / p.blk + 1 : 0;
  const int step = gridDim.x * kScoreWarps * 16;
  if (blockIdx.x * kScoreWarps * 16 >= nblk) return;  // (a warp past the end stores nothing)
  // the page and scale of block j0 + lane (lanes 0 .. 15)
  auto page_of = [&](int jj) -> int {
    const int j = jj + lane;
    return lane < 16 && j < nblk ? load_dep(p.bt + (int64_t)b * p.bt_sb + j / p.nb) : 0;
  };
  const int ni = min(n - i0, p.qn);
  if (ni <= 0) return;
  const float ninf = -__int_as_float(0x7f800000);
  // ---- A: rows g and g + 8 of 16 blocks, 16 bytes per 64 channels; with them
  // this lane's block's scale and the mask of valid blocks
  struct Tile {
    uint4 a[2][2][NC];  // [hi, lo][row][chunk]
    float s;
    unsigned okm;
  };
  auto load = [&](Tile &x, int jj) {
    const int j = jj + lane;
    const bool ok = lane < 16 && j < nblk && phys >= 0 && phys < p.n_pages;
    if (lane < 16 && j < nblk && !ok && p.status) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    int64_t off = 0;
    x.s = 0.f;
    if (ok) {
      const int sub = j % p.nb;
      off = (int64_t)phys * p.b_page + (int64_t)h * p.b_head + (int64_t)sub * p.b_blk;
      x.s = load_dep(p.scales + (int64_t)phys * p.s_page + (int64_t)h * p.s_head + sub);
    }
    phys = page_of(jj + step);  // in flight with this step's bounds
    x.okm = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int src = g + 8 * r;
      const int64_t o = __shfl_sync(0xffffffffu, off, src);
      const bool live = (x.okm >> src) & 1u;
      const uint8_t *base = p.bounds + o + 16 * t;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x.a[0][r][c] = live ? load_dep(reinterpret_cast<const uint4 *>(base + p.b_mm + 64 * c))
                            : make_uint4(0u, 0u, 0u, 0u);
        x.a[1][r][c] = live ? load_dep(reinterpret_cast<const uint4 *>(base + 64 * c))
                            : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  auto use = [&](const Tile &x, int jj) {
    const auto &a = x.a;
    float acc[NT][4];
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint32_t w0[4] = {a[m][0][c].x, a[m][0][c].y, a[m][0][c].z, a[m][0][c].w};
        const uint32_t w1[4] = {a[m][1][c].x, a[m][1][c].y, a[m][1][c].z, a[m][1][c].w};
        const __half *qb = qs + (m * NT * 8 + g) * BS + 64 * c + 16 * t;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // two k-steps each
          uint32_t fa[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            fa[e][0] = fp8x2_to_f16x2<E5M2>(w0[2 * hf + e]);
            fa[e][1] = fp8x2_to_f16x2<E5M2>(w1[2 * hf + e]);
            fa[e][2] = fp8x2_to_f16x2<E5M2>(w0[2 * hf + e] >> 16);
            fa[e][3] = fp8x2_to_f16x2<E5M2>(w1[2 * hf + e] >> 16);
          }
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const uint4 bq = *reinterpret_cast<const uint4 *>(qb + k * 8 * BS + 8 * hf);
            mma16816(acc[k], fa[0], bq.x, bq.y);
            mma16816(acc[k], fa[1], bq.z, bq.w);
          }
        }
      }
    }
    // ---- the maximum over each query's heads, through shared memory
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      us[g * RS + 8 * k + 2 * t] = acc[k][0];
      us[g * RS + 8 * k + 2 * t + 1] = acc[k][1];
      us[(g + 8) * RS + 8 * k + 2 * t] = acc[k][2];
      us[(g + 8) * RS + 8 * k + 2 * t + 1] = acc[k][3];
    }
    __syncwarp();
    // (the scale is looked at here, so that the bounds do not wait for it)
    const float s = __shfl_sync(0xffffffffu, x.s, lane & 15), sj = s * p.sm_scale;
    const bool page_ok = (x.okm >> (lane & 15)) & 1u;
    const bool live = page_ok && s >= kMinScale && s <= kMaxScale;
    if (page_ok && !live && lane < 16 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_SCALE);
    const int jo = jj + (lane & 15);
    for (int i = lane >> 4; i < ni; i += 2) {  // 16 blocks of two queries at a time
      float best = ninf;
      for (int k = 0; k < p.G; ++k) best = max_nan(best, us[(lane & 15) * RS + i * p.G + k]);
      if (jo < nblk) {
        const bool seen = (int64_t)jo * p.blk <= L - n + i0 + i;
        p.scores[(int64_t)b * p.o_sb + (int64_t)(i0 + i) * p.o_si + (int64_t)h * p.o_sh + jo] =
            live && seen ? best * sj : ninf;
      }
    }
  };
  Tile x;
  load(x, j0);  // (on its way while the queries are staged)
  // ---- B: the group's rows, split by sign
  const int rows = ni * p.G;
  auto stage = [&](int x, uint4 v) {
    const int r = x / (D / 8), c = x - r * (D / 8);
    if (r >= rows) v = make_uint4(0u, 0u, 0u, 0u);
    uint4 lo, hi;
    const __half2 z = __float2half2_rn(0.f);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t ph[4], nl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 w = *reinterpret_cast<const __half2 *>(&in[e]);
      const __half2 a = __hmax2_nan(w, z), m = __hmin2_nan(w, z);
      ph[e] = *reinterpret_cast<const uint32_t *>(&a);
      nl[e] = *reinterpret_cast<const uint32_t *>(&m);
    }
    hi = make_uint4(ph[0], ph[1], ph[2], ph[3]);
    lo = make_uint4(nl[0], nl[1], nl[2], nl[3]);
    *reinterpret_cast<uint4 *>(qs + r * BS + 8 * c) = hi;
    *reinterpret_cast<uint4 *>(qs + (NT * 8 + r) * BS + 8 * c) = lo;
  };
#pragma unroll
  for (int e = 0; e < kQ; ++e)
    if (tid + e * kScoreThreads < kChunks) stage(tid + e * kScoreThreads, qv[e]);
  for (int x = tid + kQ * kScoreThreads; x < kChunks; x += kScoreThreads) stage(x, query(x));
  __syncthreads();
  for (;;) {
    use(x, j0);
    if ((j0 += step) >= nblk) break;
    load(x, j0);
  }
}

template <int D, int NT, bool E5M2>
cudaError_t launch_t(const ScoreParams &p, cudaStream_t stream) {
  constexpr int smem = score_smem(D, NT);
  if (smem > 48 * 1024) {  // beyond the default dynamic shared-memory limit
    const cudaError_t e = cudaFuncSetAttribute(block_scores_kernel<D, NT, E5M2>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  // CTAs for one and a half loads of every SM (as far as shared memory allows),
  // whose warps then take several steps: each CTA reads and splits the queries,
  // and those of short sequences leave room early.  20.2 us for the batch above,
  // 21.5 with one load, 20.0 with two; the next step's bounds on their way during
  // one's products cost more registers than they gain (1 us)
  const int64_t per = kScoreWarps * 16, rows = (int64_t)p.Hkv * p.parts * p.B;
  const int64_t need = std::max<int64_t>(1, (p.cols + per - 1) / per);
  const int64_t res = std::max<int64_t>(1, std::min<int64_t>(8, 220 * 1024 / (smem + 1024)));
  const int64_t want = std::max<int64_t>(1, (3 * res * p.num_sms / 2 + rows - 1) / rows);
  const int64_t steps = (need + want - 1) / want;
  const dim3 grid((unsigned)std::min<int64_t>((need + steps - 1) / steps, 0x7fffffff),
                  (unsigned)(p.Hkv * p.parts), (unsigned)p.B);
  return launch_dependent(block_scores_kernel<D, NT, E5M2>, grid, kScoreThreads, smem, stream, p);
}

template <int D, bool E5M2>
cudaError_t launch_n(ScoreParams p, cudaStream_t stream) {
  // Few blocks: the queries are split over CTAs until there are two per SM.  The
  // eight queries above take 5.7 us by twos, 7.9 one by one, 6.8 all by one CTA;
  // by fours 5.1 now, 6.4 when the rule was made
  const int64_t ctas = (p.cols + 16 * kScoreWarps - 1) / (16 * kScoreWarps) * (int64_t)p.Hkv * p.B;
  p.parts = 1;
  p.qn = p.Qmax;
  while (p.qn > 1 && ctas * p.parts < 2ll * p.num_sms) {
    p.qn = (p.Qmax + 2 * p.parts - 1) / (2 * p.parts);
    p.parts = (p.Qmax + p.qn - 1) / p.qn;
  }
  const int nt = (p.qn * p.G + 7) / 8;
  if (nt <= 1) return launch_t<D, 1, E5M2>(p, stream);
  if (nt <= 2) return launch_t<D, 2, E5M2>(p, stream);
  if (nt <= 3) return launch_t<D, 3, E5M2>(p, stream);
  if (nt <= 6) return launch_t<D, 6, E5M2>(p, stream);
  return launch_t<D, 12, E5M2>(p, stream);
}

}  // namespace

cudaError_t launch_block_scores(const ScoreParams &p, bool e5m2, cudaStream_t stream) {
  switch (p.D * 2 + (e5m2 ? 1 : 0)) {
    case 128: return launch_n<64, false>(p, stream);
    case 129: return launch_n<64, true>(p, stream);
    case 256: return launch_n<128, false>(p, stream);
    case 257: return launch_n<128, true>(p, stream);
    case 512: return launch_n<256, false>(p, stream);
    case 513: return launch_n<256, true>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace vae4
