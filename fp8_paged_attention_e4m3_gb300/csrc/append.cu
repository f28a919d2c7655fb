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
// One CTA per (block, head and K | V, sequence).  A thread asks for its rows
// before it knows the page and keeps up to eight of them in registers between the
// maximum and the rounding, so that the rows of a block of up to 64 tokens at
// D = 128 (128 at 64, 32 at 256) and their codes cross memory once each (a row's
// 16 bits in, 8 out); it tracks the bounds as 16-bit values, since rounding to a
// code is monotonic.  2 x 16384 new tokens, 8 heads of 128, blocks of 64: 202 MB
// in 33.8 us, 6.0 TB/s, 0.88 of the copy peak.  What had kept it from that were
// instructions, not bytes: 256 threads of four rows each took 43.6 us with 69
// percent of the issue slots in use, since what a warp does once per block
// (lengths, page, scale, bounds) then costs as much as its rows; and 48 us before
// products with the inverse scale stayed in 16 bits and divisions by the page and
// the block became products.  Rows past the eighth of a thread are loaded again
// for the rounding: blocks of 128 tokens 48.6 us, of 256 59.9; of 64 at D = 256
// 47.2 (of 32: 32.7), of 128 58.1, of 256 63.1, for as many bytes.  A step of few
// rows is the launch and the chain lengths -> rows -> maximum -> store: 2.1 to
// 3.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kAppendThreads = 128;

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
// two FP16 values -> two E4M3 codes, to nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(d) : "r"(h));
  return d;
}
// f16x2 that holds two FP8 values -> their codes (exact)
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2_of_f16x2(uint32_t h) {
  if constexpr (E5M2) return __byte_perm(h, 0u, 0x4431) & 0xFFFFu;
  return e4m3x2_of_f16x2(h);
}

// 8 codes -> their values
template <bool E5M2>
__device__ __forceinline__ void values8(uint2 codes, __half2 (&v)[4]) {
  const uint32_t h[4] = {fp8x2_to_f16x2<E5M2>(codes.x), fp8x2_to_f16x2<E5M2>(codes.x >> 16),
                         fp8x2_to_f16x2<E5M2>(codes.y), fp8x2_to_f16x2<E5M2>(codes.y >> 16)};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const __half2 *>(&h[e]);
}

// maximum and minimum of two pairs of 16-bit values (not a NaN if one is a number)
template <bool BF16>
__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("max.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
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
// the larger magnitude of two pairs, of either sign; a NaN stays
template <bool BF16>
__device__ __forceinline__ uint32_t maxabs16(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t mul16(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF16)
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
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

// kHold: rows a thread keeps
template <int D, bool BF16, bool E5M2, int kHold>
__global__ void __launch_bounds__(kAppendThreads, kHold > 4 ? 7 : 8) append_kernel(const AppendParams p) {
  constexpr int CH = D / 8;                    // 8-element chunks per row
  constexpr int RG = kAppendThreads / CH;      // rows per pass
  constexpr int LEAD = E5M2 ? 15 : 8;          // FPMAX = 1.75 * 2^LEAD
  __shared__ uint32_t red[kAppendThreads / 32];
  __shared__ uint4 lohi[2][kAppendThreads];
  const int tid = threadIdx.x, c = tid % CH, g = tid / CH;
  const int b = blockIdx.z, h = blockIdx.y >> 1, w = blockIdx.y & 1;
  await_previous();
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
  const int64_t blk0 = div16(new0, p.blk_m) + (int64_t)blockIdx.x;  // the CTA's block
  if (blk0 * p.blk >= L) return;
  const int t0 = (int)blk0 * p.blk;
  const int a = max(new0 - t0, 0);                     // rows the block holds already
  const int z = min(p.blk, L - t0);                    // rows it holds afterwards
  // the first kHold rows of a thread are requested before the page is known;
  // they stay in registers for both passes
  const int64_t x_row = p.x_si[w];
  const uint16_t *x = static_cast<const uint16_t *>(p.x[w]) + (int64_t)b * p.x_sb[w] +
                      (int64_t)h * p.x_sh[w] + (int64_t)(t0 - new0) * x_row + 8 * c;
  const uint16_t *xk = x + (a + g) * x_row;
  auto load = [&](int r) { return __ldcs(reinterpret_cast<const uint4 *>(x + r * x_row)); };
  uint4 held[kHold];
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    held[k] = a + g + k * RG < z ? __ldcs(reinterpret_cast<const uint4 *>(xk)) : make_uint4(0u, 0u, 0u, 0u);
    xk += RG * x_row;
  }
  const int lp = div16(t0, p.page_m), slot = t0 - lp * p.page;
  const int sub = (int)blk0 - lp * p.nb;  // the block in its page
  const int phys = p.bt[(int64_t)b * p.bt_sb + lp];
  if (phys < 0 || phys >= p.n_pages) {
    if (tid == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    return;
  }
  float *sp = p.scales + (int64_t)phys * p.s_page + w * p.s_kv + (int64_t)h * p.s_head + sub;
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
    for (int e = 0; e < 4; ++e) am2 = maxabs16<BF16>(am2, u[e]);
    if (bounds && live) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = min16<BF16>(lo[e], u[e]);
        hi[e] = max16<BF16>(hi[e], u[e]);
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
  uint32_t am = block_max(max(am2 & 0x7FFFu, am2 >> 16 & 0x7FFFu));
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
          hi[e] = max16<BF16>(hi[e], f);
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
  // s a power of two: x / s is a product with its inverse, in FP32 exact, in
  // BF16 too, and in FP16 (if it holds the inverse) but for quotients below
  // 2^-14, which round to an E4M3 zero like their exact values
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0u;
  const bool direct = pow2 && (BF16 || E5M2 || (s >= 0x1p-15f && s <= 0x1p14f));
  // (s lies within 2^-40 .. 2^40: the inverse of a power of two by its exponent)
  const float inv = pow2 ? __uint_as_float(0x7F000000u - __float_as_uint(s)) : 0.f;
  const uint32_t inv16 = BF16 ? (__float_as_uint(inv) >> 16) * 0x10001u
                              : __half_as_ushort(__float2half_rn(inv)) * 0x10001u;
  if (odd && tid == 0 && p.status) atomicOr(p.status, VAE4_STATUS_BAD_VALUE);
  auto encode = [&](uint4 v, auto exact) -> uint2 {
    constexpr bool EX = decltype(exact)::value;
    if constexpr (EX && (BF16 || !E5M2)) {
      uint32_t u[4] = {v.x, v.y, v.z, v.w}, d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = mul16<BF16>(u[e], inv16);
        if constexpr (BF16)
          d[e] = fp8x2<E5M2>(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
        else
          d[e] = e4m3x2_of_f16x2(u[e]);
      }
      return make_uint2(d[0] | d[1] << 16, d[2] | d[3] << 16);
    } else {
      float f[8];
      unpack8<BF16>(v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = EX ? f[e] * inv : __fdiv_rn(f[e], s);
      return make_uint2(fp8x2<E5M2>(f[0], f[1]) | fp8x2<E5M2>(f[2], f[3]) << 16,
                        fp8x2<E5M2>(f[4], f[5]) | fp8x2<E5M2>(f[6], f[7]) << 16);
    }
  };
  // minimum and maximum over the threads of a channel chunk, first those of a
  // warp; valid in the first 2 CH threads: thread (mm, c) has chunk c's
  auto over_rows = [&](uint4 l4, uint4 h4, auto mn, auto mx) -> uint4 {
    uint32_t l[4] = {l4.x, l4.y, l4.z, l4.w}, u[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
    for (int o = 16; o >= CH; o >>= 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[e] = mn(l[e], __shfl_xor_sync(0xffffffffu, l[e], o));
        u[e] = mx(u[e], __shfl_xor_sync(0xffffffffu, u[e], o));
      }
    }
    constexpr int WG = CH < 32 ? kAppendThreads / 32 : RG;  // what is left, CH chunks each
    if (CH >= 32 || (tid & 31) < CH) {
      const int x = CH < 32 ? (tid >> 5) * CH + c : tid;
      lohi[0][x] = make_uint4(l[0], l[1], l[2], l[3]);
      lohi[1][x] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __syncthreads();
    if (tid >= 2 * CH) return make_uint4(0u, 0u, 0u, 0u);
    const int mm = tid / CH, cc = tid % CH;
    uint4 t = lohi[mm][cc];
#pragma unroll
    for (int k = 1; k < WG; ++k) {
      const uint4 q = lohi[mm][cc + k * CH];
      t = mm ? make_uint4(mx(t.x, q.x), mx(t.y, q.y), mx(t.z, q.z), mx(t.w, q.w))
             : make_uint4(mn(t.x, q.x), mn(t.y, q.y), mn(t.z, q.z), mn(t.w, q.w));
    }
    return t;
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
  } else if (direct) {
    store(std::true_type{});
  } else {
    store(std::false_type{});
  }
  // ---- rows the block holds already: under a larger scale, and in the bounds
  const bool grow = a > 0 && s > s_old;
  alignas(16) __half2 lo2[4], hi2[4];  // bounds of their codes' values
  if (grow || (bounds && a > 0)) {
    const float f = s_old / s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo2[e] = __halves2half2(__ushort_as_half(0x7C00), __ushort_as_half(0x7C00));
      hi2[e] = __halves2half2(__ushort_as_half(0xFC00), __ushort_as_half(0xFC00));
    }
    for (int r = g; r < a; r += RG) {
      uint2 codes = *reinterpret_cast<const uint2 *>(dst + r * row);
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
        *reinterpret_cast<uint2 *>(dst + r * row) = codes;
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
  // ---- bounds, over the row groups: of the new values, rounded at the end
  // (rounding is monotonic), or, with earlier rows, of the codes' values
  if (bounds) {
    auto rounded = [&](uint4 v) {
      return direct ? encode(v, std::true_type{}) : encode(v, std::false_type{});
    };
    const uint4 ln = make_uint4(lo[0], lo[1], lo[2], lo[3]), hn = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    uint2 d;
    if (a == 0) {
      d = rounded(over_rows(ln, hn, [](uint32_t x, uint32_t y) { return min16<BF16>(x, y); },
                            [](uint32_t x, uint32_t y) { return max16<BF16>(x, y); }));
    } else {  // (a thread without new rows: the infinities round to the largest codes)
      __half2 v[4];
      values8<E5M2>(rounded(ln), v);
#pragma unroll
      for (int e = 0; e < 4; ++e) lo2[e] = __hmin2(lo2[e], v[e]);
      values8<E5M2>(rounded(hn), v);
#pragma unroll
      for (int e = 0; e < 4; ++e) hi2[e] = __hmax2(hi2[e], v[e]);
      const uint4 m = over_rows(*reinterpret_cast<const uint4 *>(lo2), *reinterpret_cast<const uint4 *>(hi2),
                                [](uint32_t x, uint32_t y) { return min16<false>(x, y); },
                                [](uint32_t x, uint32_t y) { return max16<false>(x, y); });
      d = make_uint2(fp8x2_of_f16x2<E5M2>(m.x) | fp8x2_of_f16x2<E5M2>(m.y) << 16,
                     fp8x2_of_f16x2<E5M2>(m.z) | fp8x2_of_f16x2<E5M2>(m.w) << 16);
    }
    if (tid < 2 * CH) {
      const int mm = tid / CH, cc = tid % CH;
      *reinterpret_cast<uint2 *>(p.bounds + (int64_t)phys * p.b_page + (int64_t)h * p.b_head +
                                 (int64_t)sub * p.b_blk + mm * p.b_mm + 8 * cc) = d;
    }
  }
}

template <int D, int kHold>
cudaError_t launch_h(const AppendParams &p, bool bf16, bool e5m2, dim3 grid, cudaStream_t st) {
  auto *kernel = bf16 ? (e5m2 ? append_kernel<D, true, true, kHold> : append_kernel<D, true, false, kHold>)
                      : (e5m2 ? append_kernel<D, false, true, kHold> : append_kernel<D, false, false, kHold>);
  return launch_dependent(kernel, grid, kAppendThreads, 0, st, p);
}

template <int D>
cudaError_t launch_d(const AppendParams &p, bool bf16, bool e5m2, dim3 grid, cudaStream_t st) {
  // Four rows per thread where they hold a block's new rows, else eight (a block
  // of 64 tokens at D = 128 is then read once): 33.9 us for the prompts above,
  // 45.5 with four; eight cost a step of few rows 0.2 to 0.3 us more
  constexpr int rows = kAppendThreads / (D / 8);  // per pass
  return std::min(p.blk, p.Qmax) <= 4 * rows ? launch_h<D, 4>(p, bf16, e5m2, grid, st)
                                             : launch_h<D, 8>(p, bf16, e5m2, grid, st);
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
