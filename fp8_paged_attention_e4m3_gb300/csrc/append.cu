// Writer of the block-scaled FP8 cache: quantises the step's new K and V rows
// into their pages, with one power-of-two scale per block of `blk` tokens,
// KV head and K | V, and keeps each block's per-channel bounds of K.
//
// For the block's new rows x and the rows it already holds (codes c, scale
// s_old):
//     a    = max |x| over the finite values
//     need = the smallest 2^e with a <= 2^e * FPMAX, -30 <= e <= 30
//     s    = need if the block holds no earlier row, else max(s_old, need)
//     code(x) = rn(clamp(x / s)),  c <- rn(dec(c) * s_old / s) if s > s_old
// FPMAX = 1.75 * 2^8 (E4M3) or 1.75 * 2^15 (E5M2), so need follows from a's
// exponent and one comparison of its significand.  A power of two costs no
// precision (the codes are floating-point), makes x / s exact before the one
// rounding to 8 bits, and makes a later growth of s exact for every code but
// those that become subnormal.  The floor 2^-30 lies below what FP16 inputs
// can need; it is also the scale of an all-zero block, so that the next row
// of the block is free to choose.
//
// One CTA per (block, head and K | V, sequence).  The rows and their codes cross
// memory once each (a row's 16 bits in, 8 out): a thread asks for its rows before
// it knows the page and keeps them in registers between the maximum and the
// rounding, and tracks the bounds as 16-bit values, since rounding to a code is
// monotonic.  2 x 16384 new tokens, 8 heads of 128: 202 MB in 48 us, 4.2 TB/s;
// the instructions per row (rounding 8 values of a thread takes most) and the
// chain of a CTA (lengths, page, rows, maximum, store) bound it, not the bytes.
// A step of few rows is the launch and that chain: 2.8 to 3.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kCtas = 4;  // per SM; 5 leave 48 registers and spill, for the same time
constexpr int kHold = 4;  // rows a thread keeps: a block of 64 tokens at D = 128 is read once

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&v[e]));
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
}

// two floats -> two FP8 codes (a in the low byte), to nearest even, saturating
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2(float a, float b) {
  unsigned short d;
  if constexpr (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(d) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(d) : "f"(b), "f"(a));
  return d;
}
// f16x2 that holds two FP8 values -> their codes (exact)
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2_of_f16x2(uint32_t h) {
  if constexpr (E5M2) return __byte_perm(h, 0u, 0x4431) & 0xFFFFu;
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return fp8x2<false>(f.x, f.y);
}

// 8 codes -> their values
template <bool E5M2>
__device__ __forceinline__ void values8(uint2 codes, __half2 (&v)[4]) {
  const uint32_t h[4] = {fp8x2_to_f16x2<E5M2>(codes.x), fp8x2_to_f16x2<E5M2>(codes.x >> 16),
                         fp8x2_to_f16x2<E5M2>(codes.y), fp8x2_to_f16x2<E5M2>(codes.y >> 16)};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const __half2 *>(&h[e]);
}

// maximum and minimum of two pairs of 16-bit values (NAN: a NaN stays)
template <bool BF16, bool NAN_STAYS>
__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16) {
    if constexpr (NAN_STAYS)
      asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    else
      asm("max.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  } else {
    if constexpr (NAN_STAYS)
      asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    else
      asm("max.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  }
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min16(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("min.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t nan_to_zero(uint32_t v) {
  constexpr uint32_t inf = BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t l = (v & 0x7FFFu) > inf ? 0u : v & 0xFFFFu;
  const uint32_t h = ((v >> 16) & 0x7FFFu) > inf ? 0u : v & 0xFFFF0000u;
  return l | h;
}

__device__ __forceinline__ bool scale_ok(float s) { return s >= kMinScale && s <= kMaxScale; }

template <int D, bool BF16, bool E5M2>
__global__ void __launch_bounds__(kAppendThreads, kCtas) append_kernel(const AppendParams p) {
  constexpr int CH = D / 8;                    // 8-element chunks per row
  constexpr int RG = kAppendThreads / CH;      // rows per pass
  constexpr int LEAD = E5M2 ? 15 : 8;          // FPMAX = 1.75 * 2^LEAD
  __shared__ uint32_t red[kAppendThreads / 32];
  __shared__ uint4 lohi[2][kAppendThreads];
  const int tid = threadIdx.x, c = tid % CH, g = tid / CH;
  const int b = blockIdx.z, h = blockIdx.y >> 1, w = blockIdx.y & 1;
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool bad_l = L < 0 || (int64_t)L > (int64_t)p.max_pages * p.page;
  if (bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && p.status)
      atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
    return;
  }
  if (L == 0 || n == 0) return;
  const int new0 = L - n;                              // first new token
  const bool bounds = w == 0 && p.bounds != nullptr;
  const int64_t first = (new0 / p.blk + (int64_t)blockIdx.x) * p.blk;  // token of the block
  if (first >= L) return;
  const int t0 = (int)first;
  const int a = max(new0 - t0, 0);                     // rows the block holds already
  const int z = min(p.blk, L - t0);                    // rows it holds afterwards
  // the first kHold rows of a thread are requested before the page is known;
  // they stay in registers for both passes
  const int64_t x_row = p.x_si[w];
  const uint16_t *x = static_cast<const uint16_t *>(p.x[w]) + (int64_t)b * p.x_sb[w] +
                      (int64_t)h * p.x_sh[w] + (int64_t)(t0 - new0) * x_row + 8 * c;
  auto load = [&](int r) { return __ldcs(reinterpret_cast<const uint4 *>(x + r * x_row)); };
  uint4 held[kHold];
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int r = a + g + k * RG;
    held[k] = r < z ? load(r) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int lp = t0 / p.page, slot = t0 - lp * p.page;
  const int phys = p.bt[(int64_t)b * p.bt_sb + lp];
  if (phys < 0 || phys >= p.n_pages) {
    if (tid == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    return;
  }
  float *sp = p.scales + (int64_t)phys * p.s_page + w * p.s_kv + (int64_t)h * p.s_head + slot / p.blk;
  float s_old = 0.f;
  if (a > 0) {
    s_old = *sp;
    if (!scale_ok(s_old)) {  // the same for every thread
      if (tid == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_SCALE);
      return;
    }
  }
  uint8_t *dst = p.c[w] + (int64_t)phys * p.c_ps[w] + (int64_t)slot * p.c_ts[w] +
                 (int64_t)h * p.c_hs[w] + 8 * c;

  // ---- largest magnitude of the new rows (as integers the bits order alike)
  uint32_t am2 = 0u;  // two 16-bit maxima; a NaN stays
  // smallest and largest new value per channel: rounding to a code is
  // monotonic, so their codes are the bounds of the codes
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    lo[e] = BF16 ? 0x7F807F80u : 0x7C007C00u;  // infinities
    hi[e] = lo[e] | 0x80008000u;
  }
  auto look = [&](const uint4 &v, bool live) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) am2 = max16<BF16, true>(am2, u[e] & 0x7FFF7FFFu);
    if (bounds && live) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = min16<BF16>(lo[e], u[e]);
        hi[e] = max16<BF16, false>(hi[e], u[e]);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kHold; ++k) look(held[k], a + g + k * RG < z);
  for (int r = a + g + kHold * RG; r < z; r += RG) look(load(r), true);
  auto block_max = [&](uint32_t v) -> uint32_t {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((tid & 31) == 0) red[tid >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kAppendThreads / 32; ++k) v = max(v, red[k]);
    return v;
  };
  uint32_t am = block_max(max(am2 & 0xFFFFu, am2 >> 16));
  bool odd = false;  // a NaN, an infinity or a value beyond the largest scale
  if (am >= (BF16 ? 0x7F80u : 0x7C00u)) {  // rare, the same for every thread: the finite values'
    odd = true;
    am = 0u;
    for (int r = a + g; r < z; r += RG) {
      const uint4 v = load(r);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t l = u[e] & 0x7FFFu, m = (u[e] >> 16) & 0x7FFFu;
        if (l < (BF16 ? 0x7F80u : 0x7C00u)) am = max(am, l);
        if (m < (BF16 ? 0x7F80u : 0x7C00u)) am = max(am, m);
        if (bounds) {  // a NaN is stored as zero
          const uint32_t f = nan_to_zero<BF16>(u[e]);
          lo[e] = min16<BF16>(lo[e], f);
          hi[e] = max16<BF16, false>(hi[e], f);
        }
      }
    }
    __syncthreads();
    am = block_max(am);
  }
  if constexpr (BF16)
    am <<= 16;
  else
    am = __float_as_uint(__half2float(__ushort_as_half((unsigned short)am)));
  // ---- the scale
  const int e_need = (int)(am >> 23) - 127 - LEAD + ((am & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  odd |= e_need > 30;
  const float need = __uint_as_float((uint32_t)(min(max(e_need, -30), 30) + 127) << 23);
  const float s = a > 0 ? fmaxf(s_old, need) : need;
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0u;
  const float inv = 1.f / s;  // exact for a power of two
  if (odd && tid == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_VALUE);
  auto encode = [&](uint4 v, auto exact) -> uint2 {
    float f[8];
    unpack8<BF16>(v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = decltype(exact)::value ? f[e] * inv : __fdiv_rn(f[e], s);
    return make_uint2(fp8x2<E5M2>(f[0], f[1]) | fp8x2<E5M2>(f[2], f[3]) << 16,
                      fp8x2<E5M2>(f[4], f[5]) | fp8x2<E5M2>(f[6], f[7]) << 16);
  };
  // ---- new rows
  const int64_t row = p.c_ts[w];
  auto store = [&](auto exact) {
    uint8_t *d = dst + (a + g) * row;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      if (a + g + k * RG < z) *reinterpret_cast<uint2 *>(d) = encode(held[k], exact);
      d += RG * row;
    }
    for (int r = a + g + kHold * RG; r < z; r += RG, d += RG * row)
      *reinterpret_cast<uint2 *>(d) = encode(load(r), exact);
  };
  if (odd) {  // rare
    uint8_t *d = dst + (a + g) * row;
    for (int r = a + g; r < z; r += RG, d += RG * row) {
      uint4 v = load(r);
      v = make_uint4(nan_to_zero<BF16>(v.x), nan_to_zero<BF16>(v.y), nan_to_zero<BF16>(v.z),
                     nan_to_zero<BF16>(v.w));
      *reinterpret_cast<uint2 *>(d) = encode(v, std::false_type{});
    }
  } else if (pow2) {
    store(std::true_type{});
  } else {
    store(std::false_type{});
  }
  // the bounds of the new rows, as the values of their codes
  __half2 lo2[4], hi2[4];
  if (bounds) {
    if (a + g < z) {
      const uint4 vl = make_uint4(lo[0], lo[1], lo[2], lo[3]), vh = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      const uint2 cl = pow2 ? encode(vl, std::true_type{}) : encode(vl, std::false_type{});
      const uint2 ch = pow2 ? encode(vh, std::true_type{}) : encode(vh, std::false_type{});
      values8<E5M2>(cl, lo2);
      values8<E5M2>(ch, hi2);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo2[e] = __halves2half2(__ushort_as_half(0x7C00), __ushort_as_half(0x7C00));
        hi2[e] = __halves2half2(__ushort_as_half(0xFC00), __ushort_as_half(0xFC00));
      }
    }
  }
  // ---- rows the block holds already: under a larger scale, and in the bounds
  const bool grow = a > 0 && s > s_old;
  if (grow || bounds) {
    const float f = s_old / s;
    for (int r = g; r < a; r += RG) {
      uint2 codes = *reinterpret_cast<const uint2 *>(dst + r * p.c_ts[w]);
      if (grow) {
        const uint32_t in[4] = {codes.x, codes.x >> 16, codes.y, codes.y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t hh = fp8x2_to_f16x2<E5M2>(in[e]);
          const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&hh));
          o[e] = fp8x2<E5M2>(v.x * f, v.y * f);
        }
        codes = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        *reinterpret_cast<uint2 *>(dst + r * p.c_ts[w]) = codes;
      }
      if (bounds) {
        __half2 v[4];
        values8<E5M2>(codes, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo2[e] = __hmin2(lo2[e], v[e]);
          hi2[e] = __hmax2(hi2[e], v[e]);
        }
      }
    }
  }
  if (tid == 0) *sp = s;
  // ---- bounds: over the row groups, first those of a warp
  if (bounds) {
#pragma unroll
    for (int o = 16; o >= CH; o >>= 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo2[e] = __hmin2(lo2[e], __shfl_xor_sync(0xffffffffu, lo2[e], o));
        hi2[e] = __hmax2(hi2[e], __shfl_xor_sync(0xffffffffu, hi2[e], o));
      }
    }
    constexpr int WG = CH < 32 ? kAppendThreads / 32 : RG;  // what is left, CH chunks each
    if (CH >= 32 || (tid & 31) < CH) {
      const int x = CH < 32 ? (tid >> 5) * CH + c : tid;
      lohi[0][x] = *reinterpret_cast<const uint4 *>(lo2);
      lohi[1][x] = *reinterpret_cast<const uint4 *>(hi2);
    }
    __syncthreads();
    if (tid < 2 * CH) {
      const int mm = tid / CH, cc = tid % CH;
      const __half2 *v = reinterpret_cast<const __half2 *>(&lohi[mm][cc]);
      __half2 t[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int k = 1; k < WG; ++k) {
        const uint4 q = lohi[mm][cc + k * CH];
        const __half2 *u = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = mm ? __hmax2(t[e], u[e]) : __hmin2(t[e], u[e]);
      }
      const uint32_t *u = reinterpret_cast<const uint32_t *>(t);
      *reinterpret_cast<uint2 *>(p.bounds + (int64_t)phys * p.b_page + (int64_t)h * p.b_head +
                                 (int64_t)(slot / p.blk) * p.b_blk + mm * p.b_mm + 8 * cc) =
          make_uint2(fp8x2_of_f16x2<E5M2>(u[0]) | fp8x2_of_f16x2<E5M2>(u[1]) << 16,
                     fp8x2_of_f16x2<E5M2>(u[2]) | fp8x2_of_f16x2<E5M2>(u[3]) << 16);
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendParams &p, bool bf16, bool e5m2, dim3 grid, cudaStream_t st) {
  if (bf16) {
    if (e5m2) append_kernel<D, true, true><<<grid, kAppendThreads, 0, st>>>(p);
    else append_kernel<D, true, false><<<grid, kAppendThreads, 0, st>>>(p);
  } else {
    if (e5m2) append_kernel<D, false, true><<<grid, kAppendThreads, 0, st>>>(p);
    else append_kernel<D, false, false><<<grid, kAppendThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, bool bf16, bool e5m2, cudaStream_t stream) {
  const dim3 grid((unsigned)p.touched, 2u * p.Hkv, (unsigned)p.B);
  switch (p.D) {
    case 64: return launch_d<64>(p, bf16, e5m2, grid, stream);
    case 128: return launch_d<128>(p, bf16, e5m2, grid, stream);
    case 256: return launch_d<256>(p, bf16, e5m2, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace vae4
