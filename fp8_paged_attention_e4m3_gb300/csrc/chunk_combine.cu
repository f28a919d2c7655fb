// Combine of chunk attention: merges the FP32 partial states of the units that several
// CTAs shared,
//     M = max_p m_p,  w_p = 2^(m_p - M),  out = sum_p w_p O_p / sum_p w_p l_p
// over the parts with l_p > 0 (a NaN counts, and makes the row NaN), in a fixed order,
// rounded once; a part with l_p < 0 (an invalid page or scale that the row sees) makes
// the row zeros.  Parts of the unit that starts in CTA c lie in slots c, ctas + c + 1,
// ctas + c + 2, ...  CTAs past those of the units report invalid lengths and zero the
// rows of sequences without tokens.
#include <algorithm>

#include "block_common.cuh"
#include "chunk_params.h"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kWarps = 8, kRowsPerCta = 8, kZeroCtas = 32;

// lane's channels of a row: VN of them from VN * lane on
template <int VN>
struct Acc {
  float v[VN];
};
template <int VN>
__device__ __forceinline__ Acc<VN> load_row(const float *o, int lane) {
  Acc<VN> a;
  const float *x = o + VN * lane;
#pragma unroll
  for (int e = 0; e < VN; e += 2) {
    const float2 t = __ldcg(reinterpret_cast<const float2 *>(x + e));
    a.v[e] = t.x;
    a.v[e + 1] = t.y;
  }
  return a;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int VN = D / 32, R = chunk_rows(D);
  __shared__ float sums[kWarps][D];
  __shared__ float2 wl[kMaxChunkCtas];  // (weight, sum) of the parts
  __shared__ float red[kWarps][2];
  await_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float ninf = -__int_as_float(0x7f800000);
  if ((int)blockIdx.x >= p.ctas) {  // lengths
    const int n = kZeroCtas * gridDim.y;
    for (int b = (blockIdx.x - p.ctas) * gridDim.y + blockIdx.y; b < p.B; b += n) {
      const int32_t *s = p.seq + (int64_t)b * p.seq_sb;
      const int L = load_dep(s), q = p.seq_has_qlen ? load_dep(s + 1) : p.Qmax;
      const uint32_t bits = L < 0 || L > p.capacity                   ? VAE4_STATUS_BAD_LENGTH
                            : q < 0 || q > p.Qmax || (L > 0 && q > L) ? VAE4_STATUS_BAD_QLEN
                                                                      : 0u;
      if (bits && tid == 0) atomicOr(p.status, bits);
      if (bits == 0u && L > 0) continue;
      const int rows = min(max(q, 0), p.Qmax), H = p.Hkv * p.G;
      for (int r = warp; r < rows * H; r += kWarps) {
        const int i = r / H;
        uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<__half *>(p.out) + b * p.o_sb + i * p.o_si +
                                                   (long long)(r - i * H) * p.o_sh);
        for (int c = lane; c < D / 2; c += 32) o[c] = 0u;
      }
    }
    return;
  }
  const ChunkSplit u = p.split[blockIdx.x];
  const int first = blockIdx.x;
  const int r0 = blockIdx.y * kRowsPerCta;
  if (u.parts <= 0 || r0 >= u.rows) return;
  const int nP = min(u.parts, p.ctas - first);
  auto slot = [&](int k) -> int64_t { return k == 0 ? first : p.ctas + first + k; };
  auto write = [&](int r, const Acc<VN> &a, float l, bool ok) {
    const int rr = u.row0 + r, i = rr / p.G;
    __half *o = static_cast<__half *>(p.out) + u.b * p.o_sb + i * p.o_si +
                (long long)(u.h * p.G + rr - i * p.G) * p.o_sh + VN * lane;
    const bool zero = !ok || l <= 0.f;
    const float inv = zero ? 0.f : __fdiv_rn(1.f, l);
#pragma unroll
    for (int e = 0; e < VN; e += 2)
      *reinterpret_cast<uint32_t *>(o + e) = zero ? 0u : pack16(a.v[e] * inv, a.v[e + 1] * inv, p.bf16);
  };
  const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
  if (nP <= 2 * kWarps) {  // a warp per row
    const int r = r0 + warp;
    if (r >= u.rows) return;
    float2 v = make_float2(ninf, 0.f);
    if (lane < nP) v = __ldcg(ml + slot(lane) * R + r);
    float M = v.y > 0.f ? v.x : ninf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const bool ok = !__any_sync(0xffffffffu, v.y < 0.f);
    float w = v.y <= 0.f ? 0.f : exp2f(v.x - M);
    float l = w * v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    Acc<VN> acc = {};
#pragma unroll 4
    for (int k = 0; k < nP; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const Acc<VN> a = load_row<VN>(p.ws_o + (slot(k) * R + r) * D, lane);
      if (wk > 0.f) {
#pragma unroll
        for (int e = 0; e < VN; ++e) acc.v[e] = fmaf(wk, a.v[e], acc.v[e]);
      }
    }
    write(r, acc, l, ok);
    return;
  }
  // many parts: the warps share them, row after row
  for (int r = r0; r < min(r0 + kRowsPerCta, u.rows); ++r) {
    float M = ninf;
    int bad = 0;
    for (int k = tid; k < nP; k += 32 * kWarps) {
      const float2 v = __ldcg(ml + slot(k) * R + r);
      wl[k] = v;
      if (v.y < 0.f) bad = 1;
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[warp][0] = M;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, red[k][0]);
    float l = 0.f;
    Acc<VN> acc = {};
#pragma unroll 4
    for (int k = warp; k < nP; k += kWarps) {
      const Acc<VN> a = load_row<VN>(p.ws_o + (slot(k) * R + r) * D, lane);
      const float2 v = wl[k];
      const float w = v.y <= 0.f ? 0.f : exp2f(v.x - M);
      l += w * v.y;
      if (w > 0.f) {
#pragma unroll
        for (int e = 0; e < VN; ++e) acc.v[e] = fmaf(w, a.v[e], acc.v[e]);
      }
    }
    if (lane == 0) red[warp][1] = l;
#pragma unroll
    for (int e = 0; e < VN; ++e) sums[warp][VN * lane + e] = acc.v[e];
    __syncthreads();
    if (warp == 0) {
      l = 0.f;
      acc = {};
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        l += red[k][1];
#pragma unroll
        for (int e = 0; e < VN; ++e) acc.v[e] += sums[k][VN * lane + e];
      }
      write(r, acc, l, bad == 0);
    }
    __syncthreads();
  }
}

}  // namespace

namespace chunk {
cudaError_t launch_64(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_128(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_256(const ChunkParams &p, cudaStream_t s);
}  // namespace chunk

cudaError_t launch_chunk(const ChunkParams &p, cudaStream_t stream) {
  switch (p.D) {
    case 64: return chunk::launch_64(p, stream);
    case 128: return chunk::launch_128(p, stream);
    case 256: return chunk::launch_256(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_chunk_combine(const ChunkParams &p, cudaStream_t stream) {
  const int rows = std::min<int64_t>(chunk_rows(p.D), (int64_t)p.Qmax * p.G);
  const dim3 grid((unsigned)(p.ctas + kZeroCtas), (unsigned)((rows + kRowsPerCta - 1) / kRowsPerCta));
  switch (p.D) {
    case 64: return launch_dependent(chunk_combine_kernel<64>, grid, 32 * kWarps, 0, stream, p);
    case 128: return launch_dependent(chunk_combine_kernel<128>, grid, 32 * kWarps, 0, stream, p);
    case 256: return launch_dependent(chunk_combine_kernel<256>, grid, 32 * kWarps, 0, stream, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace vae4
