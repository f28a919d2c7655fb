// Attention of chunks of new tokens over the paged FP8 cache, on the 5th-generation
// tensor cores: one persistent CTA per SM that walks an equal share of the batch.
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
constexpr int kUnitCost = 3;   // key tiles of time that a unit's set-up and end take
constexpr int kMinTiles = 3;   // a CTA's share is at least this many tiles

template <int D>
struct Cfg {
  static constexpr int MT = D <= 128 ? 2 : 1;  // row tiles
  static constexpr int R = MT * 128;           // rows of a unit
  static constexpr int NC = D / 64;            // 16 KB pieces of a K or V tile
  static constexpr int KPC = 128 / NC;         // keys per piece of V
  static constexpr int RING = 4;               // pieces held, of K and of V
  static constexpr int PIECE = 16384;
  static constexpr int QT = 128 * D * 2;       // one tile of queries
  static constexpr int NSW = 4 * MT;           // softmax warps
  // warps: softmax, K decoders (4), V decoders (4), MMA, plan
  static constexpr int W_K = NSW, W_V = NSW + 4, W_MMA = NSW + 8, W_PLAN = NSW + 9;
  static constexpr int NTHREADS = 32 * (NSW + 10);
  // TMEM columns: scores (and weights in their place), accumulators
  static constexpr int SCOL = 0, OCOL = 256;
  static constexpr int NSEG = 4, NGRP = 4;     // segments, groups of four tiles held
  static constexpr int OFF_Q = 0, OFF_K = MT * QT, OFF_V = OFF_K + RING * PIECE,
                       OFF_SMALL = OFF_V + RING * PIECE;
  static constexpr int B_SEGF = 0, B_SEGE = B_SEGF + NSEG, B_INFOF = B_SEGE + NSEG,
                       B_INFOE = B_INFOF + NGRP, B_KF = B_INFOE + NGRP, B_KE = B_KF + RING,
                       B_VF = B_KE + RING, B_VE = B_VF + RING, B_QF = B_VE + RING, B_SF = B_QF + 2,
                       B_PF = B_SF + 2, B_PV = B_PF + 2, B_OE = B_PV + 2, B_DRAIN = B_OE + 2,
                       NBARS = B_DRAIN + 1;
  static constexpr int S_SCAL = 512, S_SEG = 576, S_INFO = S_SEG + NSEG * 64,
                       S_ROW = S_INFO + NGRP * 32 * 32, SMALL = S_ROW + R * 8;
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

// 16 keys: where their rows start, their scales
struct alignas(16) Box {
  long long k, v;  // offsets from the caches' bases; -1: no keys, or invalid
  float a, g, inv; // a score in log2 units per raw product, log2 s_V, 1 / s_V
  int bad;
};
static_assert(sizeof(Box) == 32, "layout");

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
static __device__ __noinline__ Segment plan_next(const ChunkParams &p, int R, int cta, Plan &o) {
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
    if (s.j0 == 0 && !ends && (threadIdx.x & 31) == 0) {
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
__device__ __forceinline__ uint4 load_raw(const uint8_t *p, int wide) {
  uint4 v;
  if (wide) {
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

enum class Decode { E4M3_F16, E5M2_F16, E4M3_BF16, E5M2_BF16 };
template <Decode M>
__device__ __forceinline__ uint32_t decode2(uint32_t two) {
  if constexpr (M == Decode::E4M3_F16) return fp8x2_to_f16x2<false>(two);
  if constexpr (M == Decode::E5M2_F16) return fp8x2_to_f16x2<true>(two);
  if constexpr (M == Decode::E4M3_BF16) return fp8x2_to_bf16x2<false>(two);
  return fp8x2_to_bf16x2<true>(two);
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  return pack_half2(a, b);
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::NTHREADS, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const float kInf = __int_as_float(0x7f800000);
  constexpr float kTau = 15.0f;  // weights up to 2^15, inside FP16

  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (sbase - raw_addr);
  const uint32_t sQ = sbase + C::OFF_Q, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V,
                 sSm = sbase + C::OFF_SMALL;
  uint8_t *gSm = gbase + C::OFF_SMALL;
  auto bar = [&](int i) -> uint32_t { return sSm + 8u * (uint32_t)i; };
  volatile int *abort_f = reinterpret_cast<volatile int *>(gSm + C::S_SCAL);
  Segment *seg_s = reinterpret_cast<Segment *>(gSm + C::S_SEG);
  Box *box_s = reinterpret_cast<Box *>(gSm + C::S_INFO);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  if (tid < C::NBARS) {
    uint32_t cnt = 1;
    if (tid >= C::B_SEGE && tid < C::B_SEGE + C::NSEG) cnt = C::NSW + 9;
    if (tid >= C::B_INFOF && tid < C::B_INFOF + C::NGRP) cnt = 32;
    if (tid >= C::B_INFOE && tid < C::B_INFOE + C::NGRP) cnt = C::NSW + 8;
    if ((tid >= C::B_KF && tid < C::B_KF + C::RING) || (tid >= C::B_VF && tid < C::B_VF + C::RING)) cnt = 4;
    if ((tid >= C::B_QF && tid < C::B_QF + 2) || (tid >= C::B_PF && tid < C::B_PF + 2) ||
        (tid >= C::B_OE && tid < C::B_OE + 2))
      cnt = 128;
    tc::mbar_init(bar(tid), cnt);
  }
  if (tid == 0) *abort_f = 0;
  if (warp == C::W_MMA) {
    tc::tmem_alloc(sSm + C::S_SCAL + 4, 512);
    tc::tmem_relinquish();
  }
  tc::mbar_fence_init();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t *>(gSm + C::S_SCAL + 4);
  if (tbase != 0u) *abort_f = 1;  // never: all 512 columns are the CTA's, from column 0
  await_previous();

  const long long LIM = p.wait_limit;
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {  // one answer for the warp
    return __all_sync(0xffffffffu, tc::mbar_wait_brief(b, parity, abort_f, LIM));
  };
  bool mma_issued = false;

  if (warp == C::W_PLAN) {
    // =============================== plan, pages and scales
    Plan plan;
    if (lane == 0) p.split[cta].parts = 0;
    plan_begin(p, C::R, cta, plan, lane);
    int ns = 0, ng = 0;
    bool ok = true;
    while (ok) {
      const Segment s = plan_next(p, C::R, cta, plan);
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
        Box x;
        x.k = x.v = -1;
        x.a = x.inv = 1.f;
        x.g = 0.f;
        x.bad = 0;
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
              x.k = (long long)page * p.k_ps + slot * p.k_ts + s.h * p.k_hs;
              x.v = (long long)page * p.v_ps + slot * p.v_ts + s.h * p.v_hs;
              x.a = p.alpha * sk;
              x.g = __log2f(sv);
              x.inv = __fdividef(1.f, sv);
              bits = 0;
            }
          }
          if (bits) {
            x.bad = 1;
            atomicOr(p.status, bits);
          }
        }
        if (ng >= C::NGRP && !(ok = warp_wait(bar(C::B_INFOE + ng % C::NGRP), (ng / C::NGRP - 1) & 1))) break;
        box_s[(ng % C::NGRP) * 32 + lane] = x;
        tc::mbar_arrive(bar(C::B_INFOF + ng % C::NGRP));
      }
    }
  } else if (warp == C::W_MMA) {
    // =============================== the products, issued by one elected lane
    const uint32_t id_qk = tc::idesc_f16(128, 128, 0, 0) | (p.bf16 ? (1u << 7 | 1u << 10) : 0u);
    constexpr uint32_t id_pv = tc::idesc_f16(128, D, 0, 1);
    int ns = 0, nk = 0, nv = 0;  // segments, pieces of K and V
    int nt[2] = {0, 0};          // score tiles issued (MT = 2: per row tile; else per buffer)
    int np[2] = {0, 0};          // weight tiles consumed
    int nq[2] = {0, 0};          // segments of each row tile
    bool ok = true;
    while (ok) {
      if (!(ok = warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1))) break;
      const int j0 = seg_s[ns % C::NSEG].j0, j1 = seg_s[ns % C::NSEG].j1;
      const int live = C::MT == 2 && seg_s[ns % C::NSEG].rows > 128 ? 2 : 1;
      __syncwarp();
      if (tc::elect_one()) tc::mbar_arrive(bar(C::B_SEGE + ns % C::NSEG));
      ++ns;
      if (j1 <= j0) break;
      // scores of row tile t into buffer s from the next tile of K
      auto scores = [&](int t, int s, bool last) -> bool {
  #pragma unroll
        for (int c = 0; c < C::NC; ++c) {
          const int x = nk + c;
          if (t == 0 && !warp_wait(bar(C::B_KF + x % C::RING), (x / C::RING) & 1)) return false;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint64_t a = tc::smem_desc(sQ + t * C::QT + c * 16384, 16, 1024);
            const uint64_t b = tc::smem_desc(sK + (x % C::RING) * C::PIECE, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_ss(C::SCOL + s * 128, a + 2 * k, b + 2 * k, id_qk, c > 0 || k > 0);
            if (last) tc::mma_commit(bar(C::B_KE + x % C::RING));
            if (c == C::NC - 1) tc::mma_commit(bar(C::B_SF + s));
          }
          __syncwarp();
        }
        mma_issued = true;
        ++nt[s];
        if (last) nk += C::NC;
        return true;
      };
      // the accumulator of row tile t takes the weights in buffer s
      auto values = [&](int t, int s, bool first, bool last) -> bool {
        if (!warp_wait(bar(C::B_PF + s), np[s] & 1)) return false;
        ++np[s];
        if (first && nq[t] > 0 && !warp_wait(bar(C::B_OE + t), (nq[t] - 1) & 1)) return false;
#pragma unroll
        for (int c = 0; c < C::NC; ++c) {
          const int x = nv + c;
          if (t == 0 && !warp_wait(bar(C::B_VF + x % C::RING), (x / C::RING) & 1)) return false;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint64_t b = tc::smem_desc(sV + (x % C::RING) * C::PIECE, C::KPC * 128, 1024);
#pragma unroll
            for (int k = 0; k < C::KPC / 16; ++k)
              tc::mma_ts(C::OCOL + t * D, C::SCOL + s * 128 + (c * (C::KPC / 16) + k) * 8, b + 128 * k,
                         id_pv, !first || c > 0 || k > 0);
            if (last) tc::mma_commit(bar(C::B_VE + x % C::RING));
            if (c == C::NC - 1) tc::mma_commit(bar(C::B_PV + s));
          }
          __syncwarp();
        }
        if (last) nv += C::NC;
        return true;
      };
      for (int t = 0; t < live && ok; ++t) ok = warp_wait(bar(C::B_QF + t), nq[t] & 1);
      if constexpr (C::MT == 2) {
        for (int t = 0; t < live && ok; ++t) ok = scores(t, t, t == live - 1);
        for (int j = j0; j < j1 && ok; ++j)
          for (int t = 0; t < live && ok; ++t) {
            ok = values(t, t, j == j0, t == live - 1);
            if (ok && j + 1 < j1) ok = scores(t, t, t == live - 1);
          }
      } else {
        int s = nt[0] == nt[1] ? 0 : 1;  // buffers alternate through all segments
        ok = ok && scores(0, s, true);
        for (int j = j0; j < j1 && ok; ++j, s ^= 1) {
          if (j + 1 < j1) ok = scores(0, s ^ 1, true);
          ok = ok && values(0, s, j == j0, true);
        }
      }
      for (int t = 0; t < live; ++t) ++nq[t];
    }
  } else if (warp >= C::W_K) {
    // =============================== decoders: 4 lanes per 64-wide row piece
    const bool isv = warp >= C::W_V;
    const int w = (warp - C::W_K) & 3, r8 = lane >> 2, u = lane & 3;
    const uint8_t *base = (isv ? p.v_base : p.k_base) + 16 * u;
    const int64_t ts = isv ? p.v_ts : p.k_ts;
    const int64_t off0 = r8 * ts, off1 = (8 + r8) * ts;
    const uint32_t ring = isv ? sV : sK;
    const int fullb = isv ? C::B_VF : C::B_KF, emptyb = isv ? C::B_VE : C::B_KE;
    const uint32_t dst = (uint32_t)(32 * w + r8) * 128 + 0u;
    const uint32_t x0 = (uint32_t)((2 * u) ^ r8) << 4, x1 = (uint32_t)((2 * u + 1) ^ r8) << 4;
    const int wide = p.wide;
    auto decode = [&](auto mode) {
      constexpr Decode M = decltype(mode)::value;
      constexpr int AHEAD = 3;  // pieces requested before the one that is decoded
      uint4 raw[AHEAD][4];
      bool have[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) have[a] = false;
      int ns = 0, ng = 0;            // segments and groups begun
      int j = 0, j0 = 0, j1 = 0, kend = 0, c = 0;
      bool open = false, more = true, ok = true;
      // request the next piece
      auto request = [&](uint4 (&r)[4]) -> bool {
        if (!more) return false;
        if (!open) {
          if (!(ok = warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1))) return more = false;
          const Segment &s = seg_s[ns % C::NSEG];
          j = j0 = s.j0;
          j1 = s.j1;
          kend = s.kend;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(C::B_SEGE + ns % C::NSEG));
          ++ns;
          if (j1 <= j0) return more = false;
          open = true;
          c = 0;
        }
        const int jl = j - j0, g = ng % C::NGRP;
        if (c == 0 && (jl & 3) == 0 && !(ok = warp_wait(bar(C::B_INFOF + g), (ng / C::NGRP) & 1)))
          return more = false;
        // the warp's 32 rows of the piece: 16-key boxes 2w, 2w + 1 of K; of V rows
        // run over the piece's keys, then over groups of 64 channels
        const int key_w = isv ? c * C::KPC + (32 * w) % C::KPC : 32 * w;
        const int d0 = isv ? 64 * ((32 * w) / C::KPC) : 64 * c;
        const Box *bx = box_s + g * 32 + (jl & 3) * 8 + (key_w >> 4);
        const int key = j * kTile + key_w + r8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long at = isv ? bx[i >> 1].v : bx[i >> 1].k;
          r[i] = make_uint4(0u, 0u, 0u, 0u);
          if (at >= 0 && key + 8 * i < kend) r[i] = load_raw(base + at + (i & 1 ? off1 : off0) + d0, wide);
        }
        if (++c == C::NC) {
          c = 0;
          ++j;
          if (j == j1 || ((j - j0) & 3) == 0) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(C::B_INFOE + g));
            ++ng;
          }
          open = j < j1;
        }
        return true;
      };
      int n = 0;  // pieces decoded
      for (bool any = true; any;) {
        any = false;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          if (have[a]) {
            const int slot = n % C::RING;
            if (n >= C::RING && !(ok = warp_wait(bar(emptyb + slot), (n / C::RING - 1) & 1))) {
              any = false;
              more = false;
              break;
            }
            const uint32_t to = ring + slot * C::PIECE + dst;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v[4] = {raw[a][i].x, raw[a][i].y, raw[a][i].z, raw[a][i].w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * e] = decode2<M>(v[e]);
                o[2 * e + 1] = decode2<M>(v[e] >> 16);
              }
              st_shared16(to + i * 1024 + x0, o[0], o[1], o[2], o[3]);
              st_shared16(to + i * 1024 + x1, o[4], o[5], o[6], o[7]);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(fullb + slot));
            ++n;
          }
          have[a] = request(raw[a]);
          any |= have[a];
        }
      }
    };
    if (!isv && p.bf16) {
      if (p.e5m2)
        decode(std::integral_constant<Decode, Decode::E5M2_BF16>{});
      else
        decode(std::integral_constant<Decode, Decode::E4M3_BF16>{});
    } else if (p.e5m2) {
      decode(std::integral_constant<Decode, Decode::E5M2_F16>{});
    } else {
      decode(std::integral_constant<Decode, Decode::E4M3_F16>{});
    }
  } else {
    // =============================== softmax: thread = row of tile t
    const int t = warp >> 2, tr = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    long long *row_s = reinterpret_cast<long long *>(gSm + C::S_ROW) + t * 128;
    int ns = 0, ng = 0, count = 0;
    bool alive = true;
    // the value product of tile x (of all segments) is done; with two score buffers up
    // to two of them are under way, so each buffer has a barrier of its own
    auto values_done = [&](int x) -> bool {
      return C::MT == 2 ? warp_wait(bar(C::B_PV + t), x & 1)
                        : warp_wait(bar(C::B_PV + (x & 1)), (x >> 1) & 1);
    };
    for (;;) {
      alive = alive && warp_wait(bar(C::B_SEGF + ns % C::NSEG), (ns / C::NSEG) & 1);
      if (tc::named_bar_or(1 + t, 128, !alive)) break;  // one answer for the four warps
      const Segment s = seg_s[ns % C::NSEG];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(C::B_SEGE + ns % C::NSEG));
      ++ns;
      if (s.j1 <= s.j0) break;
      if (t * 128 >= s.rows) {  // no row of this tile: only the groups go by
        for (int j = s.j0; j < s.j1; j += 4, ++ng) {
          alive = alive && warp_wait(bar(C::B_INFOF + ng % C::NGRP), (ng / C::NGRP) & 1);
          if (alive && lane == 0) tc::mbar_arrive(bar(C::B_INFOE + ng % C::NGRP));
        }
        continue;
      }
      const int rr = s.row0 + t * 128 + tr, i = rr / p.G;
      const bool live = t * 128 + tr < s.rows;
      const long long head = (long long)(s.h * p.G + rr - i * p.G);
      row_s[tr] = live ? s.b * p.q_sb + i * p.q_si + head * p.q_sh : -1;
      tc::named_bar(1 + t, 128);
      {
        constexpr int QCH = D / 8;  // 16-byte pieces per row
        const __half *qb = static_cast<const __half *>(p.q);
#pragma unroll 4
        for (int x = tr; x < 128 * QCH; x += 128) {
          const int r = x / QCH, cc = x - r * QCH;
          const long long at = row_s[r];
          cp_async16(sQ + t * C::QT + (cc >> 3) * 16384 + r * 128 + (((cc & 7) ^ (r & 7)) << 4),
                     qb + (at >= 0 ? at + cc * 8 : 0), at >= 0);
        }
        tc::cp_async_wait_all();
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(bar(C::B_QF + t));
      }
      // the last key that the row sees (rows past the unit's: all, of zeros)
      const int lim = live ? s.L - s.q + i : s.kend - 1;
      const int min_lim = __reduce_min_sync(0xffffffffu, lim);
      float m = -kInf, l = 0.f;
      bool bad = false;
      for (int j = s.j0; j < s.j1; ++j, ++count) {
        const int jl = j - s.j0, g = ng % C::NGRP;
        if ((jl & 3) == 0) alive = alive && warp_wait(bar(C::B_INFOF + g), (ng / C::NGRP) & 1);
        const int sb = C::MT == 2 ? t : count & 1;                 // score buffer
        const int sn = C::MT == 2 ? count : count >> 1;            // its use
        alive = alive && warp_wait(bar(C::B_SF + sb), sn & 1);
        if (!alive) continue;
        tc::tc_fence_after();
        const Box *bx = box_s + g * 32 + (jl & 3) * 8;
        const int k0 = j * kTile;
        const bool masked = k0 + kTile - 1 > min_lim;
        const uint32_t sc = tbase + lane_off + C::SCOL + sb * 128;
        float mx = -kInf;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tc::tmem_ld32(sc + 32 * c, r);
          tc::tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k0 + 32 * c + e > lim) r[e] = 0xff800000u;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mb = __uint_as_float(r[16 * k]);
#pragma unroll
            for (int e = 1; e < 16; ++e) mb = fmaxf(mb, __uint_as_float(r[16 * k + e]));
            mx = fmaxf(mx, fmaf(mb, bx[2 * c + k].a, bx[2 * c + k].g));
          }
        }
        const bool raise = mx > m + kTau;
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? mx : m;
          const float f = raise ? (m == -kInf ? 0.f : fast_exp2(m - mn)) : 1.f;
          l *= f;
          m = mn;
          if (j > s.j0) {
            alive = values_done(count - 1);
            if (!alive) continue;
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
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32], h[16];
          tc::tmem_ld32(sc + 32 * c, r);
          tc::tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k0 + 32 * c + e > lim) r[e] = 0xff800000u;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const Box &x = bx[2 * c + k];
            const float A = x.a, B = x.g - base;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float e0 = fast_exp2(fmaf(__uint_as_float(r[16 * k + 2 * e]), A, B));
              const float e1 = fast_exp2(fmaf(__uint_as_float(r[16 * k + 2 * e + 1]), A, B));
              sum += e0 + e1;
              h[8 * k + e] = pack_half2(e0, e1);
            }
            l = fmaf(sum, x.inv, l);
            if (x.bad && k0 + 16 * (2 * c + k) <= lim) bad = true;
          }
          tc::tmem_st16(sc + 16 * c, h);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(bar(C::B_PF + sb));
        if ((jl & 3) == 3 || j == s.j1 - 1) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(C::B_INFOE + g));
          ++ng;
        }
      }
      // ---- the rows out of TMEM
      alive = alive && values_done(count - 1);
      if (!alive) continue;
      tc::tc_fence_after();
      if (bad) l = -1.f;
      if (s.slot >= 0) {
        const int64_t at = (int64_t)s.slot * C::R + t * 128 + tr;
        *reinterpret_cast<float2 *>(p.ws_ml + at * 2) = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tc::tmem_ld32(tbase + lane_off + C::OCOL + t * D + c, r);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4 *>(p.ws_o + at * D + c + 4 * e) =
                make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
        }
      } else {
        const float inv = l <= 0.f ? 0.f : __fdiv_rn(1.f, l);  // (NaN if l is)
        __half *o = static_cast<__half *>(p.out) + (live ? s.b * p.o_sb + i * p.o_si + head * p.o_sh : 0);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32], h[16];
          tc::tmem_ld32(tbase + lane_off + C::OCOL + t * D + c, r);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = __uint_as_float(r[2 * e]), y = __uint_as_float(r[2 * e + 1]);
            h[e] = l <= 0.f ? 0u : pack16(x * inv, y * inv, p.bf16);
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4 *>(o + c + 8 * e) =
                  make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
          }
        }
      }
      tc::tc_fence_before();
      tc::mbar_arrive(bar(C::B_OE + t));
    }
  }

  // ---- wind-down; after a wait that ran out: mark everything of the CTA invalid
  tc::cp_async_wait_all();
  __syncthreads();
  const bool aborted = *abort_f != 0;
  if (aborted) {
    if (warp == C::W_MMA && mma_issued && tc::elect_one()) {
      tc::mma_commit(bar(C::B_DRAIN));
      volatile int no_abort = 0;
      tc::mbar_wait_brief(bar(C::B_DRAIN), 0, &no_abort, p.drain_limit);
    }
    Plan plan;
    if (warp == C::W_PLAN) plan_begin(p, C::R, cta, plan, lane);
    for (;;) {
      if (warp == C::W_PLAN) {
        const Segment s = plan_next(p, C::R, cta, plan);
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
  if (warp == C::W_MMA) tc::tmem_dealloc(tbase, 512);
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
  return launch_dependent(chunk_kernel<D>, dim3((unsigned)p.ctas), C::NTHREADS, C::SMEM, stream, p);
}

// one head dim each, compiled in a translation unit of its own
cudaError_t launch_64(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_128(const ChunkParams &p, cudaStream_t s);
cudaError_t launch_256(const ChunkParams &p, cudaStream_t s);

}  // namespace chunk
}  // namespace vae4
