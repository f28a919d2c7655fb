// Combine of attention over a block-scaled cache: merges the FP32 partial
// states of the units that several CTAs of the split kernel shared,
//     M = max_p m_p,  w_p = 2^(m_p - M),  out = sum_p w_p O_p / sum_p w_p l_p
// over the parts with l_p > 0 (a NaN counts, and makes the row NaN: its query or
// its scores held one), in a fixed order, rounded once to FP16 (the
// block scales are in O and l already), and writes zeros to padding rows,
// sequences without tokens, rows without a visible key and units with an
// invalid part (l < 0).  Units finished in one CTA (parts = -1) are left.
//
// A unit's parts lie in slots first, ctas + first + 1, ctas + first + 2, ...
// Few streams (many parts each): one CTA per (row, 64 channels), 16 groups of
// 16 lanes over the parts.  Many streams: one warp per (row, 32 channels).  The
// latency of table -> parts -> sums bounds both: 152 parts of 48 rows of 256
// (7.5 MB, in L2) take 4 us after the split kernel.
#include <algorithm>

#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {


__device__ __forceinline__ bool row_live(const SegParams &p, int b, int i, uint32_t *bits) {
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int ql = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  *bits = L < 0 || L > p.seq_capacity                    ? VAE4_STATUS_BAD_LENGTH
          : ql < 0 || ql > p.Qmax || (L > 0 && ql > L) ? VAE4_STATUS_BAD_QLEN
                                                       : 0u;
  return *bits == 0u && L > 0 && i < ql;
}

__device__ __forceinline__ int64_t slot_of(const SegParams &p, int first, int k) {
  return k == 0 ? first : p.ctas + first + k;
}

__device__ __forceinline__ uint2 half4(float4 a, float l, bool ok) {
  if (!ok || l <= 0.f) return make_uint2(0u, 0u);
  return make_uint2(pack_half2(__fdiv_rn(a.x, l), __fdiv_rn(a.y, l)),
                    pack_half2(__fdiv_rn(a.z, l), __fdiv_rn(a.w, l)));
}

// ---- one CTA per (row, 64 channels)
constexpr int kRowThreads = 256, kRowLanes = 16, kRowGroups = 16;

__global__ void __launch_bounds__(kRowThreads) seg_combine_rows(const SegParams p) {
  extern __shared__ __align__(16) float wl[];  // weights, then sums, of the parts
  __shared__ float4 accs[kRowGroups][kRowLanes];
  __shared__ float red[kRowThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nd = p.D / 64, r = blockIdx.x / nd, d0 = (blockIdx.x - r * nd) * 64;
  const int h = blockIdx.y, b = blockIdx.z, i = r / p.G;
  uint32_t bits;
  const bool live = row_live(p, b, i, &bits);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (bits != 0u && blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(p.status, bits);
  __half *out = static_cast<__half *>(p.out) + (int64_t)b * p.o_sb + (int64_t)i * p.o_si +
                (int64_t)(h * p.G + r - i * p.G) * p.o_sh + d0;
  const int rg = r / p.N, rr = r - rg * p.N;
  int2 e = make_int2(0, 0);
  if (live) e = p.tab[((int64_t)b * p.Hkv + h) * p.n_rg + rg];
  if (e.y < 0) return;
  const int l4 = tid % kRowLanes, grp = tid / kRowLanes, nP = min(e.y, p.ctas);
  const float *o = p.ws_o + (int64_t)rr * p.D + d0 + 4 * l4;
  const int64_t ostride = (int64_t)p.N * p.D;
  // the first parts of this thread's group, requested with the (m, l) pairs
  constexpr int kPre = 10;  // 160 parts
  float4 pre[kPre];
#pragma unroll
  for (int k = 0; k < kPre; ++k) {
    const int x = grp + k * kRowGroups;
    pre[k] = x < nP ? __ldcg(reinterpret_cast<const float4 *>(o + slot_of(p, e.x, x) * ostride))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float ninf = -__int_as_float(0x7f800000);
  float *wm = wl, *ws = wl + p.ctas;
  float mx = ninf;
  int bad = 0;
  for (int x = tid; x < nP; x += kRowThreads) {
    const float2 v = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml) + slot_of(p, e.x, x) * p.N + rr);
    wm[x] = v.x;
    ws[x] = v.y;
    if (v.y < 0.f) bad = 1;
    if (v.y > 0.f) mx = fmaxf(mx, v.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if (lane == 0) red[warp] = mx;
  bad = __syncthreads_or(bad);
  float M = red[0];
#pragma unroll
  for (int k = 1; k < kRowThreads / 32; ++k) M = fmaxf(M, red[k]);
  __syncthreads();
  float lam = 0.f;
  for (int x = tid; x < nP; x += kRowThreads) {
    const float l = ws[x], w = l <= 0.f ? 0.f : exp2f(wm[x] - M);
    wm[x] = w;
    lam += w * l;  // (NaN if l is)
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) lam += __shfl_xor_sync(0xffffffffu, lam, off);
  if (lane == 0) red[warp] = lam;
  __syncthreads();
  lam = 0.f;
#pragma unroll
  for (int k = 0; k < kRowThreads / 32; ++k) lam += red[k];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kPre; ++k) {
    const int x = grp + k * kRowGroups;
    if (x < nP && wm[x] > 0.f) {
      const float w = wm[x];
      acc.x += w * pre[k].x;
      acc.y += w * pre[k].y;
      acc.z += w * pre[k].z;
      acc.w += w * pre[k].w;
    }
  }
  for (int x = grp + kPre * kRowGroups; x < nP; x += kRowGroups) {
    const float w = wm[x];
    if (w > 0.f) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + slot_of(p, e.x, x) * ostride));
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
  }
  accs[grp][l4] = acc;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int k = 1; k < kRowGroups; ++k) {
      const float4 v = accs[k][l4];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    *reinterpret_cast<uint2 *>(out + 4 * l4) = half4(acc, lam, !bad);
  }
}

// ---- one warp per (row, 32 channels)
constexpr int kWarpThreads = 256;

__global__ void __launch_bounds__(kWarpThreads) seg_combine_warps(const SegParams p) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int nds = p.D == 64 ? 1 : p.D == 128 ? 2 : 3;  // log2 of D / 32
  const int x = blockIdx.x * (kWarpThreads / 32) + (threadIdx.x >> 5);
  const int r = x >> nds, sl = x & ((1 << nds) - 1);
  const int h = blockIdx.y, b = blockIdx.z, i = r / p.G;
  if (i >= p.Qmax) return;
  uint32_t bits;
  const bool live = row_live(p, b, i, &bits);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (bits != 0u && r == 0 && h == 0 && sl == 0 && lane == 0) atomicOr(p.status, bits);
  const int rg = r / p.N, rr = r - rg * p.N;
  int2 e = make_int2(0, 0);
  if (live) e = p.tab[((int64_t)b * p.Hkv + h) * p.n_rg + rg];
  if (e.y < 0) return;
  const int g = lane >> 3, f = lane & 7;  // eight lanes read 128 bytes of a part; four groups
  const int nP = min(e.y, p.ctas);
  const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml) + rr;
  const float *o = p.ws_o + (int64_t)rr * p.D + 32 * sl + 4 * f;
  const float ninf = -__int_as_float(0x7f800000);
  float M = ninf, lam = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  bool bad = false;
  constexpr int NPL = 4;  // parts per lane at a time
  for (int c0 = 0; c0 < nP; c0 += 4 * NPL) {
    float2 m[NPL];
    float4 v[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      const int q = c0 + g + 4 * k;
      m[k] = make_float2(ninf, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < nP) {
        const int64_t s = slot_of(p, e.x, q);
        m[k] = __ldcg(ml + s * p.N);
        v[k] = __ldcg(reinterpret_cast<const float4 *>(o + s * p.N * p.D));
      }
    }
    float mx = M;
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      if (m[k].y > 0.f) mx = fmaxf(mx, m[k].x);
      bad |= m[k].y < 0.f;
    }
#pragma unroll
    for (int off = 8; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (mx != M) {  // this round raised the maximum
      const float c = M == ninf ? 0.f : exp2f(M - mx);
      lam *= c;
      acc.x *= c;
      acc.y *= c;
      acc.z *= c;
      acc.w *= c;
      M = mx;
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      if (!(m[k].y <= 0.f)) {
        const float w = exp2f(m[k].x - M);
        lam += w * m[k].y;
        acc.x += w * v[k].x;
        acc.y += w * v[k].y;
        acc.z += w * v[k].z;
        acc.w += w * v[k].w;
      }
    }
  }
#pragma unroll
  for (int off = 8; off < 32; off <<= 1) {
    lam += __shfl_xor_sync(0xffffffffu, lam, off);
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane < 8) {
    __half *out = static_cast<__half *>(p.out) + (int64_t)b * p.o_sb + (int64_t)i * p.o_si +
                  (int64_t)(h * p.G + r - i * p.G) * p.o_sh + 32 * sl + 4 * f;
    *reinterpret_cast<uint2 *>(out) = half4(acc, lam, !bad);
  }
}

}  // namespace

cudaError_t launch_seg_combine(const SegParams &p, cudaStream_t stream) {
  const int R = p.Qmax * p.G;
  if ((int64_t)p.B * p.Hkv < 8) {
    const dim3 grid((unsigned)(R * (p.D / 64)), (unsigned)p.Hkv, (unsigned)p.B);
    return launch_dependent(seg_combine_rows, grid, kRowThreads, (size_t)p.ctas * 2 * sizeof(float),
                            stream, p);
  }
  const int warps = R * (p.D / 32), per = kWarpThreads / 32;
  const dim3 grid((unsigned)((warps + per - 1) / per), (unsigned)p.Hkv, (unsigned)p.B);
  return launch_dependent(seg_combine_warps, grid, kWarpThreads, 0, stream, p);
}

}  // namespace vae4
