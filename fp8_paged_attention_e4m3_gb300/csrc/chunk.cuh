// Attention of chunks of new tokens over the paged FP8 cache, on the 5th-generation
// tensor cores: one persistent CTA per SM that walks an equal share of the batch.
//
// Of a row (one query of one head) with z_t = scale s_K q.dec(K_t) over the keys that it
// sees, kept in log2 units:
//     w_t = 2^(z_t + log2 s_V - m),  l = sum w_t / s_V,  out = sum w_t dec(V_t) / l
// for any reference m near the maximum; m is raised, and what was summed rescaled, only
// when a weight would pass 2^15.9.  The block's s_V is in the exponent, so that V enters its
// product as it is decoded.
//
// Both products are FP16: FP8 becomes FP16 exactly, in one conversion, and the tensor cores
// add in FP32.  4 D operations per score against one exp2 and some four other instructions:
// the tensor cores bound the kernel (D = 256: 0.87 of the measured dense rate), below that
// the softmax's chain: its warps wait for the fetch of instructions and for tensor memory,
// and no unit is full (D = 128: 0.66, tensor cores at work in 54 % of the cycles, instructions
// issued in 46 %; D = 64: 0.38).
//
// A unit is R = 512 (D = 64 and 256: 256) rows of a KV head's queries: K and V are read and
// decoded once for all of them, and where a tile of 128 keys would not leave room for two
// tiles of rows (D >= 128), a pair of CTAs shares it, each decoding half.
//
// Measured: 8192 tokens of 64 heads on 8 of 128, FP16 869 us (1266 TFLOP/s), BF16 944; 2048
// behind 65536 of 6 heads on 1 of 256, 482 to 488 us (1670); 4096 behind 12288 of 32 on 8 of
// 64, 656 us (733), of 256 behind 4096, 576 to 585 us (1420); 64 tokens of 8 on 8 of 128
// behind 131072, 125 us (2.1 TB/s of keys: a row tile a quarter full, one pass of decoding per
// 64 rows).  Scores that keep growing cost rescaled accumulators: the first with a standard
// deviation of 4 in the place of 1 863 us, of 8 1078.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "block_common.cuh"
#include "chunk_params.h"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {
namespace chunk {

constexpr int kTile = 128;     // keys per tile
// Key tiles of time that a unit's set-up and end take.  (64 single tokens behind 500 to 2831,
// 32 heads on 8 of 128: 171 us with 1, 160 with 2, 149 with 3, 140 with 5, 146 with 8; a batch of
// chunks and single tokens, 24 heads on 8: 1446, 1441, 1435, 1436 and 1443, of 64 channels 592,
// 587, 587, 590 and 597.)
constexpr int kUnitCost = 3;
// A CTA's share is at least this many tiles.  (32 of 1024 tokens of 2 heads on 1 of 64: 12.8 us
// with 1, 12.2 with 2, 14.0 with 3, 15.8 with 5; larger calls do not tell.)
constexpr int kMinTiles = 3;

template <int D>
struct Cfg {
  static constexpr int CG = chunk_group(D);    // CTAs that share a unit
  static constexpr int MT = D <= 128 ? 2 : 1;  // row tiles per CTA
  static constexpr int R = chunk_rows(D);      // rows of a unit
  static_assert(R == MT * 128 * CG, "rows");
  // K and V are decoded in pieces of 128 rows of 64 channels; of a tile a CTA has the
  // keys (K) or the channels (V) of its half, or all
  static constexpr int PIECE = 16384, RING = 4;  // bytes; pieces held, of K and of V
  static constexpr int NC = D / 64 / CG;       // pieces of a K or V tile
  static constexpr int KR = 128 / CG;          // keys of K that a CTA has
  static constexpr int QT = 128 * D * 2;       // one tile of queries
  static constexpr int NSW = 4 * MT;           // softmax warps
  // warps: softmax, decoders, MMA (one per accumulator), plan; up to 16 in all leave each
  // 128 registers
  // (MT = 2: 3 decoders decode 64 queries' 131072 keys in 137 us, 4 in 125, 5 in 130)
  static constexpr int ND = MT == 2 ? 4 : 8;
  static constexpr int W_DEC = NSW, W_MMA = NSW + ND, W_PLAN = W_MMA + MT;
  static constexpr int NTHREADS = 32 * (W_PLAN + 1);
  // A decoder that waits for a place has passed the one before it of any other warp's
  // (no more pieces are under way than the rings hold), so parities are unambiguous.
  static_assert(ND <= 2 * RING, "decoders");
  // Scores are made KW keys at a time, into one of two buffers of the row tile, so that
  // the next ones are there when the softmax is through with these.
  static constexpr int KW = MT == 2 ? 64 : 128, SPT = 128 / KW;  // steps per key tile
  static constexpr int BPS = KW / CG / 16;     // boxes of 16 keys of a step that a CTA has of K
  // TMEM columns: scores (and weights in their place), accumulators
  static constexpr int SCOL = 0, OCOL = 256;
  static constexpr int NSEG = 4, NGRP = 4;     // segments, groups of four tiles held
  static constexpr int OFF_Q = 0, OFF_K = MT * QT, OFF_V = OFF_K + RING * PIECE,
                       OFF_SMALL = OFF_V + RING * PIECE;
  static constexpr int B_SEGF = 0, B_SEGE = B_SEGF + NSEG, B_INFOF = B_SEGE + NSEG,
                       B_INFOE = B_INFOF + NGRP, B_KF = B_INFOE + NGRP, B_KE = B_KF + RING,
                       B_VF = B_KE + RING, B_VE = B_VF + RING, B_QF = B_VE + RING, B_SF = B_QF + 2,
                       B_PF = B_SF + 2 * MT, B_PV = B_PF + 2 * MT, B_OE = B_PV + 2 * MT,
                       B_DRAIN = B_OE + 2,
                       NBARS = B_DRAIN + MT;
  static constexpr int S_SCAL = 512, S_SEG = 576, S_INFO = S_SEG + NSEG * 64,
                       S_ROW = S_INFO + NGRP * 4 * 256, S_END = S_ROW + MT * 128 * 8,
                       SMALL = S_END + 128 * 8;
  static constexpr int SMEM = OFF_SMALL + SMALL + 1024;
  static_assert(NBARS * 8 <= S_SCAL && SMEM <= 232448, "shared memory");
};

struct Segment {
  int b, h, row0, j0, j1;  // sequence, KV head, first row, key tiles; j1 = j0: the end
  int L, q, kend;          // length, queries, end of the keys
  int slot;                // of the partial state; -1: the whole unit
  int rows;                // live rows of the unit
  int pad[6];
};
static_assert(sizeof(Segment) == 64, "layout");

// What the roles have to know of a tile, for each of its boxes of 16 keys.
struct alignas(16) Tile {
  long long k[8], v[8];  // where the rows start, from the caches' bases; -1: no keys, or invalid
  float a[8], g[8];      // s_K, log2 s_V
  float inv[8];          // 1 / s_V
  int bad[8];
};
static_assert(sizeof(Tile) == 256, "layout");

// ---------------------------------------------------------------------------
// The plan.  Units are (sequence, KV head, R rows of the chunk's q G rows, query by
// query), laid end to end on a line whose places are G-ths of a key: a unit takes
// G (128 kUnitCost + L - q) + min((u + 1) R, q G) of them, about its visible keys, so
// that places before a unit have a closed form.
struct Lens {
  int L, q;
};
__device__ __forceinline__ Lens lens_of(const ChunkParams &p, int b) {
  const int32_t *s = p.seq + (int64_t)b * p.seq_sb;
  const int L = load_dep(s), q = p.seq_has_qlen ? load_dep(s + 1) : p.Qmax;
  const bool live = L > 0 && L <= p.capacity && q > 0 && q <= p.Qmax && q <= L;
  return live ? Lens{L, q} : Lens{0, 0};
}
__device__ __forceinline__ long long base_cost(const ChunkParams &p, Lens v) {
  return (long long)p.G * (kTile * kUnitCost + v.L - v.q);
}
__device__ __forceinline__ int units_of(const ChunkParams &p, Lens v, int R) {
  return (v.q * p.G + R - 1) / R;
}
// places of the first u units of a head (u < its units)
__device__ __forceinline__ long long places(const ChunkParams &p, Lens v, int R, int u) {
  return u * base_cost(p, v) + (long long)R * u * (u + 1) / 2;
}
__device__ __forceinline__ long long head_places(const ChunkParams &p, Lens v, int R) {
  if (v.q == 0) return 0;
  return places(p, v, R, units_of(p, v, R) - 1) + base_cost(p, v) + (long long)v.q * p.G;
}

struct Plan {
  long long pos, end, share;  // place to go on from, the CTA's end, places per CTA
  long long start;            // of sequence b
  int b;
  Lens v;
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One warp: the CTA's share, and the sequence where it starts.
static __device__ __noinline__ void plan_begin(const ChunkParams &p, int R, int cta, Plan &o, int lane) {
  long long sum = 0;
  for (int b = lane; b < p.B; b += 32) sum += p.Hkv * head_places(p, lens_of(p, b), R);
  const long long total = warp_sum(sum);
  const long long least = (long long)(kMinTiles * kTile + 2) * p.G;
  o.share = max((total + p.ctas - 1) / p.ctas, least);
  o.pos = min(total, cta * o.share);
  o.end = min(total, o.pos + o.share);
  o.b = 0;
  o.start = 0;
  o.v = Lens{0, 0};
  if (o.pos >= o.end) return;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const Lens v = b0 + lane < p.B ? lens_of(p, b0 + lane) : Lens{0, 0};
    const long long mine = p.Hkv * head_places(p, v, R);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, o.start + incl > o.pos);
    if (hit) {
      const int src = __ffs(hit) - 1;
      o.b = b0 + src;
      o.v = Lens{__shfl_sync(0xffffffffu, v.L, src), __shfl_sync(0xffffffffu, v.q, src)};
      o.start += __shfl_sync(0xffffffffu, incl - mine, src);
      return;
    }
    o.start += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The next segment with keys (j1 > j0), or the end (j1 = j0).  The whole warp calls
// it with the same state.
static __device__ __noinline__ Segment plan_next(const ChunkParams &p, int R, int cta, bool write, Plan &o) {
  Segment s;
  s.j0 = s.j1 = 0;
  while (o.pos < o.end) {
    long long head = head_places(p, o.v, R);
    while (o.pos >= o.start + p.Hkv * head) {
      o.start += p.Hkv * head;
      o.v = lens_of(p, ++o.b);
      head = head_places(p, o.v, R);
    }
    const long long in = o.pos - o.start;
    const int h = (int)(in / head);
    const long long off = in - h * head;
    const int units = units_of(p, o.v, R);
    int u = 0;
    for (int lo = 0, hi = units; hi - lo > 1;) {  // the unit that holds the place
      const int mid = (lo + hi) / 2;
      (places(p, o.v, R, mid) <= off ? lo : hi) = mid;
      u = lo;
    }
    const int last = min((u + 1) * R, o.v.q * p.G);  // rows up to its end
    const long long at = o.start + h * head + places(p, o.v, R, u);
    const long long cost = base_cost(p, o.v) + last, setup = (long long)p.G * kTile * kUnitCost;
    const int keys = o.v.L - o.v.q + (last - 1) / p.G + 1;
    const int nt = (keys + kTile - 1) / kTile;
    // tiles before a place of the unit: the same for both CTAs that a place divides
    auto tiles = [&](long long x) -> int {
      return x <= setup ? 0 : x >= cost ? nt : (int)((x - setup) * nt / (cost - setup));
    };
    const long long to = min(o.end, at + cost);
    s.j0 = tiles(o.pos - at);
    s.j1 = tiles(to - at);
    o.pos = to;
    if (s.j1 <= s.j0) continue;
    s.b = o.b;
    s.h = h;
    s.row0 = u * R;
    s.L = o.v.L;
    s.q = o.v.q;
    s.kend = min(s.j1 * kTile, keys);
    s.rows = last - u * R;
    const bool ends = s.j1 == nt;
    s.slot = s.j0 > 0 ? p.ctas + cta : ends ? -1 : cta;
    if (s.j0 == 0 && !ends && write && (threadIdx.x & 31) == 0) {
      // the CTAs after this one that hold more of it: up to the one of its last place
      const int c1 = (int)((at + cost + o.share - 1) / o.share) - 1;
      ChunkSplit x;
      x.b = s.b;
      x.h = h;
      x.row0 = s.row0;
      x.parts = c1 - cta + 1;
      x.rows = s.rows;
      p.split[cta] = x;
    }
    return s;
  }
  return s;
}

// ---------------------------------------------------------------------------
template <bool WIDE>
__device__ __forceinline__ uint4 load_raw(const uint8_t *p) {
  uint4 v;
  if constexpr (WIDE) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  } else {
    const uint2 a = load_dep(reinterpret_cast<const uint2 *>(p));
    const uint2 b = load_dep(reinterpret_cast<const uint2 *>(p + 8));
    v = make_uint4(a.x, a.y, b.x, b.y);
  }
  return v;
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// A row of BF16 queries in shared memory (a thread's row r of a tile) becomes FP16: the
// products' operands are of one type, and FP8 becomes FP16 in one conversion (as BF16, in
// five operations, 8192 tokens of 64 heads of 128 took 1485 us).  The row is multiplied
// with the power of two that brings its largest magnitude to 2^14 .. 2^15: BF16's 8 bits
// then are FP16's down to 2^-28 of that, and what is smaller is off by at most 2^-39 of it,
// far less than the FP32 sum of the products is off by.  Returns the exponent of the power's
// inverse (0 for a row of zeros; infinities and NaN stay what they are).
template <int D>
__device__ __forceinline__ int row_to_f16(uint8_t *q, int r) {
  auto at = [&](int c) -> uint4 * {
    return reinterpret_cast<uint4 *>(q + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
  uint32_t top = 0;  // the largest finite magnitude
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = *at(c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
      if (lo < 0x7F80u) top = max(top, lo);
      if (hi < 0x7F80u) top = max(top, hi);
    }
  }
  const int e = top == 0 ? 141 : max((int)(top >> 7), 20);  // the biased exponent
  const float f = __int_as_float((268 - e) << 23);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint4 v = *at(c);
    v.x = pack_half2(__uint_as_float(v.x << 16) * f, __uint_as_float(v.x & 0xFFFF0000u) * f);
    v.y = pack_half2(__uint_as_float(v.y << 16) * f, __uint_as_float(v.y & 0xFFFF0000u) * f);
    v.z = pack_half2(__uint_as_float(v.z << 16) * f, __uint_as_float(v.z & 0xFFFF0000u) * f);
    v.w = pack_half2(__uint_as_float(v.w << 16) * f, __uint_as_float(v.w & 0xFFFF0000u) * f);
    *at(c) = v;
  }
  return e - 141;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::NTHREADS, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const float kInf = __int_as_float(0x7f800000);
  // The reference is set kBelow under the row's largest score and stays until a weight would
  // pass 2^kTau, inside FP16: so what FP16's subnormals leave of small weights is off by
  // 2^-27 of the largest.  (Lower still, and scores of a standard deviation of 4 raise it:
  // 8192 tokens of 64 heads of 128 take 864 us with 0, 863 with 2, 870 with 3, 891 with 4,
  // 1070 with 8.)  Where the row's second step has nothing within 2^-kFar of its first, as
  // behind a first token that takes most of the weight, often with values near zero, the
  // reference goes down by 8 once: the output is what the small ones leave.  (Takes
  // 0 to 1 % of the time, 1.6 % with a kFar of 10.)
  constexpr float kTau = 15.9f, kBelow = 2.0f, kFar = 14.0f;
  constexpr float kLarge = 0x1p12f;  // references from here on take rounded scores

  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (sbase - raw_addr);
  const uint32_t sQ = sbase + C::OFF_Q, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V,
                 sSm = sbase + C::OFF_SMALL;
  uint8_t *gSm = gbase + C::OFF_SMALL;
  auto bar = [&](int i) -> uint32_t { return sSm + 8u * (uint32_t)i; };
  volatile int *abort_f = reinterpret_cast<volatile int *>(gSm + C::S_SCAL);
  Segment *seg_s = reinterpret_cast<Segment *>(gSm + C::S_SEG);
  Tile *tile_s = reinterpret_cast<Tile *>(gSm + C::S_INFO);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x / C::CG, rank = blockIdx.x % C::CG;  // group of CTAs, and place in it

  if (tid < C::NBARS) {
    uint32_t cnt = 1;
    if (tid >= C::B_SEGE && tid < C::B_SEGE + C::NSEG) cnt = C::NSW + C::ND + (rank == 0 ? C::MT : 0);
    if (tid >= C::B_INFOF && tid < C::B_INFOF + C::NGRP) cnt = 32;
    if (tid >= C::B_INFOE && tid < C::B_INFOE + C::NGRP) cnt = C::NSW + C::ND;
    // (those below are the first CTA's, whose thread issues for the group)
    if ((tid >= C::B_KF && tid < C::B_KF + C::RING) || (tid >= C::B_VF && tid < C::B_VF + C::RING))
      cnt = C::NC * C::CG;
    if ((tid >= C::B_KE && tid < C::B_KE + C::RING) || (tid >= C::B_VE && tid < C::B_VE + C::RING)) cnt = C::MT;
    if ((tid >= C::B_QF && tid < C::B_QF + 2) || (tid >= C::B_PF && tid < C::B_PF + 2 * C::MT) ||
        (tid >= C::B_OE && tid < C::B_OE + 2))
      cnt = 4 * C::CG;
    tc::mbar_init(bar(tid), cnt);
  }
  if (tid == 0) *abort_f = 0;
  if (warp == C::W_MMA) {
    if constexpr (C::CG == 2) {
      tc::tmem_alloc_pair(sSm + C::S_SCAL + 4, 512);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(sSm + C::S_SCAL + 4, 512);
      tc::tmem_relinquish();
    }
  }
  tc::mbar_fence_init();
  tc::tc_fence_before();
  __syncthreads();
  if constexpr (C::CG == 2) tc::cluster_sync();  // the barriers of both are there
  tc::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t *>(gSm + C::S_SCAL + 4);
  if (tbase != 0u) *abort_f = 1;  // never: all 512 columns are the CTA's, from column 0
  await_previous();

  const long long LIM = p.wait_limit;
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {  // one answer for the warp
    return __all_sync(0xffffffffu, tc::mbar_wait_brief(b, parity, abort_f, LIM));
  };
  // a warp's arrival on a barrier of the CTA that issues; its earlier writes are visible
  // there to who waits for it
  auto arrive_first = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) {
      if constexpr (C::CG == 2)
        tc::mbar_arrive_at(b, 0);
      else
        tc::mbar_arrive(b);
    }
  };
  bool mma_issued = false;

  if (warp == C::W_PLAN) {
    // =============================== plan, pages and scales
    Plan plan;
    if (lane == 0 && rank == 0) p.split[cta].parts = 0;
    plan_begin(p, C::R, cta, plan, lane);
    int ns = 0, ng = 0;
    bool ok = true;
    while (ok) {
      const Segment s = plan_next(p, C::R, cta, rank == 0, plan);
      if (ns >= C::NSEG && !(ok = warp_wait(bar(C::B_SEGE + ns % C::NSEG), (ns / C::NSEG - 1) & 1))) break;
      if (lane == 0) {
        seg_s[ns % C::NSEG] = s;
        tc::mbar_arrive(bar(C::B_SEGF + ns % C::NSEG));
      }
      ++ns;
      if (s.j1 <= s.j0) break;
      const int32_t *row = p.bt + (int64_t)s.b * p.bt_sb;
      for (int key0 = s.j0 * kTile; key0 < s.j1 * kTile; key0 += 4 * kTile, ++ng) {
        const int key = key0 + 16 * lane;
        long long xk = -1, xv = -1;
        float xa = 1.f, xg = 0.f, xi = 1.f;
        int bad = 0;
        if (key < s.kend) {
          const int lp = div16(key, p.page_m), slot = key - lp * p.page;
          const int page = load_dep(row + lp);
          unsigned bits = VAE4_STATUS_BAD_BLOCK;
          if (page >= 0 && page < p.n_pages) {
            const float *sp = p.scales + (int64_t)page * p.s_page + (int64_t)s.h * p.s_head +
                              (div16(key, p.blk_m) - lp * p.page_blocks);
            const float sk = load_dep(sp), sv = load_dep(sp + p.s_kv);
            bits = VAE4_STATUS_BAD_SCALE;
            if (sk >= kMinScale && sk <= kMaxScale && sv >= kMinScale && sv <= kMaxScale) {
              xk = (long long)page * p.k_ps + slot * p.k_ts + s.h * p.k_hs;
              xv = (long long)page * p.v_ps + slot * p.v_ts + s.h * p.v_hs;
              xa = sk;
              xg = __log2f(sv);
              xi = __fdividef(1.f, sv);
              bits = 0;
            }
          }
          if (bits) {
            bad = 1;
            atomicOr(p.status, bits);
          }
        }
        if (ng >= C::NGRP && !(ok = warp_wait(bar(C::B_INFOE + ng % C::NGRP), (ng / C::NGRP - 1) & 1))) break;
        Tile &x = tile_s[(ng % C::NGRP) * 4 + (lane >> 3)];
        x.k[lane & 7] = xk;
        x.v[lane & 7] = xv;
        x.a[lane & 7] = xa;
        x.g[lane & 7] = xg;
        x.inv[lane & 7] = xi;
        x.bad[lane & 7] = bad;
        tc::mbar_arrive(bar(C::B_INFOF + ng % C::NGRP));
      }
    }
  } else if (warp >= C::W_MMA) {
    // =============================== the products, issued by one elected lane
    // A warp per accumulator, as the issue is a warp's serial code: one warp for both bound
    // the kernel (8192 tokens of 64 heads of 128: 1121 us instead of 863).  Both run the
    // same code (two copies of it: 879, and 708 instead of 656 for 4096 behind 12288 of 32
    // heads of 64: the fetch of instructions is what the roles share).  What the issue
    // depends on stays the same for the warp, in uniform registers, and ring slots follow
    // from a tile's number.  The first CTA of a pair issues for both; the other's warps have
    // nothing to do, and do not wait for segments, which may take longer than any wait.
    constexpr uint32_t id_qk = tc::idesc_f16(128 * C::CG, C::KW, 0, 0);
    constexpr uint32_t id_pv = tc::idesc_f16(128 * C::CG, D, 0, 1);
    const uint64_t dq = tc::smem_desc(sQ, 16, 1024), dk = tc::smem_desc(sK, 16, 1024),
                   dv = tc::smem_desc(sV, C::PIECE, 1024);
    constexpr uint32_t TPR = C::RING / C::NC;  // tiles that a ring holds
    constexpr uint32_t TILE16 = C::NC * C::PIECE / 16;
    const int t = __shfl_sync(0xffffffffu, warp - C::W_MMA, 0);
    int ns = 0;
    uint32_t tiles0 = 0;       // key tiles of earlier segments
    uint32_t done = 0;         // key tiles that the accumulator has taken in them
    uint32_t no = 0;           // parity of the segments with tiles for the accumulator
    bool had = false;          // has it had one?
    bool ok = rank == 0;
    auto wait_all = [&](uint32_t b, uint32_t parity) {  // arrivals of the whole group
      if (C::CG == 2 && LIM >= tc::kMinWaitLimit && __all_sync(0xffffffffu, tc::mbar_try_wait_cluster(b, parity)))
        return;
      ok = ok && warp_wait(b, parity);
      if constexpr (C::CG == 2) ok = ok && __all_sync(0xffffffffu, tc::mbar_try_wait_cluster(b, parity));
    };
    auto commit = [&](uint32_t b) {
      if constexpr (C::CG == 2)
        tc::mma_commit_pair(b);
      else
        tc::mma_commit(b);
    };
    // A step's buffer, and the parity of its use: step h of the accumulator's tile n.
    auto buffer = [&](uint32_t n, int h) -> uint32_t { return 2 * t + (C::SPT == 2 ? h : n & 1); };
    auto parity = [&](uint32_t n) -> uint32_t { return (C::SPT == 2 ? n : n >> 1) & 1; };
    while (ok) {
      if (!(ok = warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1))) break;
      const Segment &sg = seg_s[ns % C::NSEG];
      const int tiles = __shfl_sync(0xffffffffu, sg.j1 - sg.j0, 0);
      const bool solo = C::MT == 2 && __shfl_sync(0xffffffffu, sg.rows, 0) <= 128 * C::CG;
      __syncwarp();
      if (tc::elect_one()) tc::mbar_arrive(bar(C::B_SEGE + ns % C::NSEG));
      ++ns;
      if (tiles <= 0) break;
      // One tile of rows: the key tiles go to the two accumulators in turn.  Each gives
      // back the other's tile beside its own, so that neither is a ring ahead.
      const int qt = solo ? 0 : t, step = solo ? 2 : 1, n = solo ? (tiles + 1 - t) / 2 : tiles;
      const uint32_t first = tiles0 + (solo ? t : 0);
      auto other = [&](int i) -> int { return 2 * i + 1 - t; };
      // scores of step h of the accumulator's tile i
      auto scores = [&](int i, int h) {
        const uint32_t kt = first + i * step, x = kt % TPR, buf = buffer(done + i, h);
        if (h == 0) wait_all(bar(C::B_KF + x), (kt / TPR) & 1);
        tc::tc_fence_after();
        if (ok && tc::elect_one()) {
          const uint64_t b = dk + x * TILE16 + h * (C::KR * 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            // (64 channels of 128 rows of Q, of KR rows of K)
            const uint64_t ak = dq + qt * (C::QT / 16) + (k >> 2) * 1024 + 2 * (k & 3),
                           bk = b + (k >> 2) * (C::KR * 8) + 2 * (k & 3);
            if constexpr (C::CG == 2)
              tc::mma_ss_pair(C::SCOL + buf * C::KW, ak, bk, id_qk, k > 0);
            else
              tc::mma_ss(C::SCOL + buf * C::KW, ak, bk, id_qk, k > 0);
          }
          commit(bar(C::B_SF + buf));
          if (h == C::SPT - 1) {
            commit(bar(C::B_KE + x));
            if (solo && other(i) < tiles) commit(bar(C::B_KE + (tiles0 + other(i)) % TPR));
          }
        }
        __syncwarp();
      };
      // the accumulator takes the step's weights
      auto values = [&](int i, int h) {
        const uint32_t vt = first + i * step, x = vt % TPR, buf = buffer(done + i, h);
        wait_all(bar(C::B_PF + buf), parity(done + i));
        if (h == 0) {
          if (i == 0 && had) wait_all(bar(C::B_OE + t), no ^ 1);
          wait_all(bar(C::B_VF + x), (vt / TPR) & 1);
        }
        tc::tc_fence_after();
        if (ok && tc::elect_one()) {
          const uint64_t b = dv + x * TILE16 + h * (C::KW * 8);
#pragma unroll
          for (int k = 0; k < C::KW / 16; ++k) {
            const uint32_t ak = C::SCOL + buf * C::KW + k * 8;
            if constexpr (C::CG == 2)
              tc::mma_ts_pair(C::OCOL + t * D, ak, b + 128 * k, id_pv, i > 0 || h > 0 || k > 0);
            else
              tc::mma_ts(C::OCOL + t * D, ak, b + 128 * k, id_pv, i > 0 || h > 0 || k > 0);
          }
          if (h == C::SPT - 1) {
            commit(bar(C::B_VE + x));
            if (solo && other(i) < tiles) commit(bar(C::B_VE + (tiles0 + other(i)) % TPR));
          }
          commit(bar(C::B_PV + buf));
        }
        __syncwarp();
      };
      if (n > 0) wait_all(bar(C::B_QF + t), no);
      mma_issued = true;
      // The scores two steps on follow the value product that frees their buffer.
      if (n > 0) {
        scores(0, 0);
        if (C::SPT == 2) scores(0, 1);
        if (C::SPT == 1 && n > 1) scores(1, 0);
      }
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int to = i + 2 / C::SPT;
#pragma unroll
        for (int h = 0; h < C::SPT; ++h) {
          values(i, h);
          if (to < n) scores(to, h);
        }
      }
      if (t == 1 && solo && (tiles & 1)) {  // the last tile has no other
        const uint32_t kt = tiles0 + tiles - 1, x = kt % TPR;
        wait_all(bar(C::B_KF + x), (kt / TPR) & 1);  // (the one before it in its place is done with)
        wait_all(bar(C::B_VF + x), (kt / TPR) & 1);
        if (ok && tc::elect_one()) {
          commit(bar(C::B_KE + x));
          commit(bar(C::B_VE + x));
        }
        __syncwarp();
      }
      tiles0 += tiles;
      done += n;
      if (n > 0) {
        no ^= 1;
        had = true;
      }
    }
  } else if (warp >= C::W_DEC) {
    // =============================== decoders: a warp per piece
    // Pieces of K and V in the order K, V of tile 0, K, V of tile 1, ... go round the
    // warps.  A piece's 128 rows of 64 bytes are requested at once, 4 lanes per row, and
    // decoded when they are there and their place is free: the other warps' pieces are
    // under way meanwhile.
    const int r8 = lane >> 2, u = lane & 3;
    const uint32_t dst = (uint32_t)r8 * 128;
    const uint32_t x0 = (uint32_t)((2 * u) ^ r8) << 4, x1 = (uint32_t)((2 * u + 1) ^ r8) << 4;
    const uint8_t *kb = p.k_base + 16 * u + r8 * p.k_ts, *vb = p.v_base + 16 * u + r8 * p.v_ts;
    const int64_t k8 = 8 * p.k_ts, v8 = 8 * p.v_ts;
    constexpr int PPT = 2 * C::NC;  // pieces per tile
    int ns = 0, ng = 0;
    uint32_t tiles = 0;             // before the segment
    int turn = warp - C::W_DEC;     // pieces until the warp's next one
    bool ok = true;
    while (ok) {
      if (!(ok = warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1))) break;
      const Segment &sg = seg_s[ns % C::NSEG];
      const int j0 = sg.j0, n = sg.j1 - sg.j0, kend = sg.kend;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(C::B_SEGE + ns % C::NSEG));
      ++ns;
      if (n <= 0) break;
      for (int g0 = 0; g0 < n && ok; g0 += 4, ++ng) {
        const int pieces = min(4, n - g0) * PPT;
        if (!(ok = warp_wait(bar(C::B_INFOF + ng % C::NGRP), (ng / C::NGRP) & 1))) break;
#pragma unroll 1
        for (; turn < pieces; turn += C::ND) {
          const int jl = turn / PPT, pc = turn % PPT, c = pc % C::NC;
          const bool isv = pc >= C::NC;
          const uint32_t x = (tiles + g0 + jl) * C::NC + c;  // the piece's number among K's or V's
          // the rows of a piece: the CTA's keys (its part of each step's) of 64 channels, or
          // of 64 after another (K); 128 keys of 64 of the CTA's channels (V)
          const Tile &tl = tile_s[(ng % C::NGRP) * 4 + jl];
          const long long *bx = isv ? tl.v : tl.k + rank * C::BPS;
          const int left = kend - (j0 + g0 + jl) * kTile - (isv ? 0 : rank * C::BPS * 16) - r8;  // keys from row r8 on
          const uint8_t *base = isv ? vb + rank * (D / C::CG) + 64 * c : kb + 64 * C::CG * c;
          const int64_t s8 = isv ? v8 : k8;
          uint4 raw[16];
          auto request = [&](auto wide_) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int ik = i % (C::KR / 8), dk0 = 64 * (i / (C::KR / 8));  // K: row in the channels' group
              const int kb16 = (ik >> 1) / C::BPS * (C::KW / 16) + (ik >> 1) % C::BPS;
              const int b16 = isv ? i >> 1 : kb16;
              const long long at = bx[b16];
              const bool live = at >= 0 && 16 * b16 + 8 * (i & 1) < left;
              raw[i] = make_uint4(0u, 0u, 0u, 0u);
              if (live) raw[i] = load_raw<decltype(wide_)::value>(base + at + (i & 1 ? s8 : 0) + (isv ? 0 : dk0));
            }
          };
          if (p.wide)
            request(std::true_type{});
          else
            request(std::false_type{});
          const uint32_t slot = x % C::RING, use = x / C::RING, grp = slot / C::NC;
          if (use > 0 && !(ok = warp_wait(bar((isv ? C::B_VE : C::B_KE) + grp), (use - 1) & 1))) break;
          const uint32_t to = (isv ? sV : sK) + slot * C::PIECE + dst;
          auto decode = [&](auto e5m2) {
            constexpr bool E5 = decltype(e5m2)::value;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * e] = fp8x2_to_f16x2<E5>(v[e]);
                o[2 * e + 1] = fp8x2_to_f16x2<E5>(v[e] >> 16);
              }
              st_shared16(to + i * 1024 + x0, o[0], o[1], o[2], o[3]);
              st_shared16(to + i * 1024 + x1, o[4], o[5], o[6], o[7]);
            }
          };
          if (p.e5m2)
            decode(std::true_type{});
          else
            decode(std::false_type{});
          tc::fence_proxy_async_smem();
          arrive_first(bar((isv ? C::B_VF : C::B_KF) + grp));
        }
        turn -= pieces;
        __syncwarp();
        if (ok && lane == 0) tc::mbar_arrive(bar(C::B_INFOE + ng % C::NGRP));
      }
      tiles += n;
    }
  } else {
    // =============================== softmax: thread = row of tile t
    const int t = warp >> 2, tr = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    long long *row_s = reinterpret_cast<long long *>(gSm + C::S_ROW) + t * 128;
    float2 *end_s = reinterpret_cast<float2 *>(gSm + C::S_END);
    int ns = 0, ng = 0, count = 0;
    bool alive = true;
    // The value product of the row tile's step x of all segments.
    auto values_done = [&](int x) -> bool { return warp_wait(bar(C::B_PV + 2 * t + (x & 1)), (x >> 1) & 1); };
    for (;;) {
      alive = alive && warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1);
      // One answer for all softmax warps: they enter a segment, with its barriers that have no
      // time limit, all or none.
      if (tc::named_bar_or(1, 32 * C::NSW, !alive)) break;
      // (the segment's place is given back at its end: what is needed once is read there)
      const Segment &s = seg_s[ns % C::NSEG];
      const uint32_t seg_free = bar(C::B_SEGE + ns % C::NSEG);
      ++ns;
      const int j0 = s.j0, j1 = s.j1;
      if (j1 <= j0) break;
      // One tile of rows: both groups of warps have its rows, and every other key tile each
      // (a chain of scores, softmax and value product would leave the tensor cores idle).
      const bool solo = C::MT == 2 && s.rows <= 128 * C::CG;
      const int rt = solo ? 0 : t;  // row tile
      // the row's query and head, and whether it is one of the unit's
      auto row_of = [&](int &i, long long &head) -> bool {
        const int r = (rt * C::CG + rank) * 128 + tr, rr = s.row0 + r;
        i = rr / p.G;
        head = s.h * p.G + rr - i * p.G;
        return r < s.rows;
      };
      int lim;  // the last key that the row sees (rows past the unit's: all, of zeros)
      {
        int i;
        long long head;
        const bool live = row_of(i, head);
        row_s[tr] = live ? s.b * p.q_sb + i * p.q_si + head * p.q_sh : -1;
        lim = live ? s.L - s.q + i : s.kend - 1;
      }
      const int min_lim = __reduce_min_sync(0xffffffffu, lim);
      tc::named_bar(2 + t, 128);
      const bool has_q = !solo || t == 0;  // the group stages the queries
      int qe = 0;  // the row's queries have to be multiplied with 2^qe
      if (has_q) {
        constexpr int QCH = D / 8;  // 16-byte pieces per row
        const __half *qb = static_cast<const __half *>(p.q);  // (or BF16)
#pragma unroll 4
        for (int x = tr; x < 128 * QCH; x += 128) {
          const int r = x / QCH, cc = x - r * QCH;
          const long long at = row_s[r];
          cp_async16(sQ + t * C::QT + (cc >> 3) * 16384 + r * 128 + (((cc & 7) ^ (r & 7)) << 4),
                     qb + (at >= 0 ? at + cc * 8 : 0), at >= 0);
        }
        tc::cp_async_wait_all();
        if (p.bf16) {
          tc::named_bar(2 + t, 128);
          qe = row_to_f16<D>(gbase + C::OFF_Q + t * C::QT, tr);
          if (solo) end_s[tr].x = __int_as_float(qe);
        }
        tc::fence_proxy_async_smem();
        arrive_first(bar(C::B_QF + t));
        if (solo && j1 - j0 > 1) arrive_first(bar(C::B_QF + 1));  // (the other has tiles too)
      }
      if (solo && p.bf16) {  // the second group needs the rows' factors too
        tc::named_bar(4, 256);
        qe = __float_as_int(end_s[tr].x);
      }
      // A raw score times s_K of 2^-40 .. 2^40 and `qs` is one in log2 units.  Where that
      // factor would leave FP32's normal range, so that a zero could become NaN, and the
      // -infinity of a hidden key too, raw scores are first multiplied with `pre`.  (A power
      // past FP32's own range takes every score to zero or infinity, as the true one would.)
      qe += p.alpha_e;
      const int ce = min(max(qe, -86), 86);
      const float qs = p.alpha * __int_as_float((127 + ce) << 23);
      const float pre = __int_as_float((127 + min(max(qe - ce, -126), 127)) << 23);
      // Are the row's scores rounded to log2 units, in place, before anything else?  As a
      // rule one operation makes the exponent of a weight from a raw score and log2 s_V - m,
      // two roundings off by 2^-24 |m| each: below kLarge 2^-12 in all, but past 2^24 the
      // weight of the largest key itself would be past FP16, or nothing.
      bool rounded = qe != ce, any_rounded = __any_sync(0xffffffffu, rounded);
      float m = -kInf, l = 0.f;
      bool bad = false;
      int seen = 0;  // steps of the segment
      for (int j = j0; j < j1; ++j) {
        const int jl = j - j0, g = ng % C::NGRP;
        if ((jl & 3) == 0) alive = alive && warp_wait(bar(C::B_INFOF + g), (ng / C::NGRP) & 1);
        auto group_end = [&]() {
          if ((jl & 3) == 3 || j == j1 - 1) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(C::B_INFOE + g));
            ++ng;
          }
        };
        if (solo && (jl & 1) != t) {
          if (alive) group_end();
          continue;
        }
        const Tile &tl = tile_s[g * 4 + (jl & 3)];
#pragma unroll 1
        for (int half = 0; half < C::SPT; ++half) {
          constexpr int NK = C::KW / 16;  // boxes of 16 keys
          float a8[NK], g8[NK];
#pragma unroll
          for (int k = 0; k < NK; k += 4) {
            *reinterpret_cast<float4 *>(&a8[k]) = *reinterpret_cast<const float4 *>(&tl.a[half * NK + k]);
            *reinterpret_cast<float4 *>(&g8[k]) = *reinterpret_cast<const float4 *>(&tl.g[half * NK + k]);
          }
#pragma unroll
          for (int k = 0; k < NK; ++k) a8[k] *= qs;
          const int sb = 2 * t + (count & 1);  // score buffer
          alive = alive && warp_wait(bar(C::B_SF + sb), (count >> 1) & 1);
          if (!alive) break;
          tc::tc_fence_after();
          const int k0 = j * kTile + half * C::KW;
          const bool masked = k0 + C::KW - 1 > min_lim;
          const uint32_t sc = tbase + lane_off + C::SCOL + sb * C::KW;
          // The row's scores, 16 at a time, the next requested before these are looked at.
          // (64 of them held in registers, or one pass whose sums tell whether the weights
          // fit, took as long; rolled into loops that wait for each request, 8 % longer.)
          uint32_t y[2][16];
          float mx;
          bool raise, lower, some, round = rounded;
#pragma unroll 1
          for (;;) {
            if (masked || any_rounded) {  // in place: what the row does not see becomes -infinity
              int see = lim - k0;
#pragma unroll 1
              for (int c = 0; c < C::KW / 32; ++c, see -= 32) {
                uint32_t x[32];
                tc::tmem_ld32(sc + 32 * c, x);
                tc::tmem_wait_ld();
                if (round) {
#pragma unroll
                  for (int b = 0; b < 2; ++b) {
                    const int k = half * NK + 2 * c + b;
                    const float f = tl.a[k] * qs, g2 = tl.g[k];
#pragma unroll
                    for (int e = 16 * b; e < 16 * b + 16; ++e)
                      x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]) * pre, f, g2));
                  }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e > see) x[e] = 0xff800000u;
                tc::tmem_st32(sc + 32 * c, x);
              }
              tc::tmem_wait_st();
            }
            if (round) {
#pragma unroll
              for (int k = 0; k < NK; ++k) {
                a8[k] = 1.f;
                g8[k] = 0.f;
              }
            }
            mx = -kInf;
            tc::tmem_ld16(sc, y[0]);
#pragma unroll
            for (int k = 0; k < NK; ++k) {
              uint32_t(&x)[16] = y[k & 1];
              tc::tmem_wait_ld();
              tc::tmem_ld16(sc + 16 * ((k + 1) % NK), y[(k + 1) & 1]);  // (from the first again)
              auto score = [&](int e) -> float { return __uint_as_float(x[e]); };
              float m0 = max3(score(0), score(1), score(2)), m1 = max3(score(8), score(9), score(10));
#pragma unroll
              for (int e = 3; e < 7; e += 2) {
                m0 = max3(m0, score(e), score(e + 1));
                m1 = max3(m1, score(e + 8), score(e + 9));
              }
              mx = fmaxf(mx, fmaf(max3(m0, m1, fmaxf(score(7), score(15))), a8[k], g8[k]));
            }
            raise = mx > m + kTau;
            lower = seen == 1 && mx < m + (kBelow - kFar);
            some = __any_sync(0xffffffffu, raise || lower);
            if (!some) break;
            round = raise && !rounded && fabsf(mx) >= kLarge;  // from this step on
            if (!__any_sync(0xffffffffu, round)) break;
            rounded |= round;
            any_rounded = true;
          }
          if (some) {
            // (a reference past 2^22 would lose kBelow)
            const float mn = raise ? (fabsf(mx) < 0x1p22f ? mx - kBelow : mx) : lower ? m - 8.f : m;
            const float f = raise && m == -kInf ? 0.f : mn != m ? fast_exp2(m - mn) : 1.f;
            l *= f;
            m = mn;
            if (seen > 0) {
              alive = values_done(count - 1);
              if (!alive) break;
              tc::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t r[16];
                tc::tmem_ld16(tbase + lane_off + C::OCOL + t * D + c, r);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                tc::tmem_st16(tbase + lane_off + C::OCOL + t * D + c, r);
              }
            }
          }
          const float base = m == -kInf ? 0.f : m;
          // weights of 16 keys at a time into the place of scores that have been read
          float inv = tl.inv[half * NK];
          int badb = tl.bad[half * NK];
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            uint32_t(&x)[16] = y[k & 1];
            tc::tmem_wait_ld();
            if (k < NK - 1) tc::tmem_ld16(sc + 16 * (k + 1), y[(k + 1) & 1]);
            const float2 A = make_float2(a8[k], a8[k]), B = make_float2(g8[k] - base, g8[k] - base);
            float2 sum = make_float2(0.f, 0.f);
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float2 w = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), A, B);
              w.x = fast_exp2(w.x);
              w.y = fast_exp2(w.y);
              sum = add2(sum, w);
              h[e] = pack_half2(w.x, w.y);
            }
            l = fmaf(sum.x + sum.y, inv, l);
            if (badb && k0 + 16 * k <= lim) bad = true;
            if (k < NK - 1) {
              inv = tl.inv[half * NK + k + 1];
              badb = tl.bad[half * NK + k + 1];
            }
            tc::tmem_st8(sc + 8 * k, h);
          }
          tc::tmem_wait_st();
          tc::tc_fence_before();
          arrive_first(bar(C::B_PF + sb));
          ++count;
          ++seen;
        }
        if (alive) group_end();
      }
      // ---- the rows out of TMEM
      if (seen > 0) alive = alive && values_done(count - 1);
      tc::tc_fence_after();
      if (bad) l = -1.f;
      float f0 = 1.f, f1 = 0.f;  // of the accumulators
      if (solo) {  // the first group joins both and writes
        if (t == 1) end_s[tr] = make_float2(m, l);
        tc::tc_fence_before();
        alive = !tc::named_bar_or(4, 256, !alive);
        tc::tc_fence_after();
        if (t == 0) {
          const float2 o = end_s[tr];
          const float M = fmaxf(l > 0.f ? m : -kInf, o.y > 0.f ? o.x : -kInf);
          f0 = l <= 0.f ? 0.f : fast_exp2(m - M);
          f1 = o.y <= 0.f ? 0.f : fast_exp2(o.x - M);
          l = l < 0.f || o.y < 0.f ? -1.f : f0 * l + f1 * o.y;  // (NaN if one is)
          m = M;
        }
      }
      if (alive && !(solo && t == 1)) {
        const bool both = solo && j1 - j0 > 1;
        int i;
        long long head;
        const bool live = row_of(i, head);
        const uint32_t oc = tbase + lane_off + C::OCOL + t * D;
        const int64_t at = (int64_t)s.slot * C::R + (t * C::CG + rank) * 128 + tr;
        const float inv = l <= 0.f ? 0.f : __fdiv_rn(1.f, l);  // (NaN if l is)
        __half *o = static_cast<__half *>(p.out) + (live ? s.b * p.o_sb + i * p.o_si + head * p.o_sh : 0);
        if (s.slot >= 0) *reinterpret_cast<float2 *>(p.ws_ml + at * 2) = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t r[16];
          tc::tmem_ld16(oc + c, r);
          tc::tmem_wait_ld();
          if (both) {
            uint32_t q[16];
            tc::tmem_ld16(oc + D + c, q);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              r[e] = __float_as_uint(fmaf(f1, __uint_as_float(q[e]), f0 * __uint_as_float(r[e])));
          }
          if (s.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4 *>(p.ws_o + at * D + c + 4 * e) =
                  make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          } else {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = __uint_as_float(r[2 * e]), y = __uint_as_float(r[2 * e + 1]);
              h[e] = l <= 0.f ? 0u : pack16(x * inv, y * inv, p.bf16);
            }
            if (live) {
              *reinterpret_cast<uint4 *>(o + c) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4 *>(o + c + 8) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
        }
        tc::tc_fence_before();
      }
      // (what the first group has read of the second's may go)
      if (solo && tc::named_bar_or(5, 256, !alive)) alive = false;
      if (!alive) continue;
      if (seen > 0) arrive_first(bar(C::B_OE + t));
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(seg_free);
    }
  }

  // ---- wind-down; after a wait that ran out, in either CTA: mark everything of the group
  // invalid, once both have stopped
  tc::cp_async_wait_all();
  __syncthreads();
  bool aborted = *abort_f != 0;
  if (aborted && mma_issued && tc::elect_one()) {  // (of an issuing warp, its products)
    const uint32_t drain = bar(C::B_DRAIN + warp - C::W_MMA);
    if constexpr (C::CG == 2)
      tc::mma_commit_pair(drain);
    else
      tc::mma_commit(drain);
    volatile int no_abort = 0;
    tc::mbar_wait_brief(drain, 0, &no_abort, p.drain_limit);
  }
  __syncwarp();
  if constexpr (C::CG == 2) {
    tc::cluster_sync();  // nothing of the other CTA's reaches this one's memory any more
    aborted = aborted || tc::ld_shared_at(sSm + C::S_SCAL, rank ^ 1) != 0;
    tc::cluster_sync();
  }
  if (aborted) {
    Plan plan;
    if (warp == C::W_PLAN) plan_begin(p, C::R, cta, plan, lane);
    for (;;) {
      if (warp == C::W_PLAN) {
        const Segment s = plan_next(p, C::R, cta, rank == 0, plan);
        if (lane == 0) seg_s[0] = s;
      }
      __syncthreads();
      const Segment s = seg_s[0];
      if (s.j1 <= s.j0) break;
      if (tid == 0) atomicOr(p.status, VAE4_STATUS_TIMEOUT);
      if (s.slot >= 0) {
        for (int x = tid; x < C::R; x += C::NTHREADS) p.ws_ml[((int64_t)s.slot * C::R + x) * 2 + 1] = -1.f;
      } else {
        for (int x = tid; x < s.rows * (D / 8); x += C::NTHREADS) {
          const int rr = s.row0 + x / (D / 8), i = rr / p.G;
          *reinterpret_cast<uint4 *>(static_cast<__half *>(p.out) + s.b * p.o_sb + i * p.o_si +
                                     (long long)(s.h * p.G + rr - i * p.G) * p.o_sh + x % (D / 8) * 8) =
              make_uint4(0u, 0u, 0u, 0u);
        }
      }
      __syncthreads();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == C::W_MMA) {
    if constexpr (C::CG == 2)
      tc::tmem_dealloc_pair(tbase, 512);
    else
      tc::tmem_dealloc(tbase, 512);
  }
}

template <int D>
cudaError_t launch_d(const ChunkParams &p, cudaStream_t stream) {
  using C = Cfg<D>;
  // the shared-memory opt-in is set once per context
  constexpr int kDevs = 64;
  static std::atomic<unsigned long long> configured[kDevs] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const unsigned long long ctx = current_context_id();
  if (dev < 0 || dev >= kDevs || ctx == 0 ||
      configured[dev].load(std::memory_order_acquire) != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kDevs)
      configured[dev].store(current_context_id(), std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.ctas * C::CG));
  cfg.blockDim = dim3(C::NTHREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C::CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, chunk_kernel<D>, p);
}

// one head dim each, compiled in a translation unit of its own
cudaError_t launch_64(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_128(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_256(const ChunkParams &p, cudaStream_t s);

}  // namespace chunk
}  // namespace vae4
