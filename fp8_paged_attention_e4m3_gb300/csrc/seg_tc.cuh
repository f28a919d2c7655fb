// Split kernel of attention over a block-scaled cache, dense or over sparse
// attention's visit lists, on the 5th-generation tensor cores (tcgen05, TMEM
// accumulators, TMA tensor loads): one persistent CTA per SM that walks an
// equal share of the whole batch's keys.
//
// Work.  A unit is (sequence, KV head, row group of N rows) with its keys in
// half-tiles of 64; units are laid end to end, each preceded by kUnitCost
// half-tiles' worth of set-up, and CTA c takes places [c q, (c + 1) q) of that
// line, q = ceil(total / CTAs): segments of consecutive units, so that every
// SM is busy to the end whatever the mix of lengths and heads.  (A grid with
// one partition per CTA ran 256 streams of 10 .. 33 thousand tokens, D = 128,
// in two waves of unequal CTAs: 478 us.)  A unit that lies in one CTA is
// finished there; the others leave FP32 (max, sum, unnormalised P.V) per CTA
// for the combine: the CTA where a unit starts writes slot c, the later ones
// slot CTAs + c, so a unit that starts in CTA c has its parts in slots c,
// CTAs + c + 1, CTAs + c + 2, ...
//
// What bounds it.  The keys' bytes, read once: 32 sequences of up to 32749
// tokens, 8 heads of 128 (1.42 GB), take 234 us with the combine, 0.90 of the
// copy peak (245 on some GPUs), with the softmax and the decoders beside the
// copies.  One sequence of 262144 tokens, 48 rows of 256 (134 MB), takes 35.0 us
// (0.57): 3 us to the first copy (lengths, plan, page), 3 to the first scores, 20
// at the memory's rate, up to 4 for the SMs whose rows are raised most often, 4
// for the combine.  Two row groups (more than 64 rows a KV head) each read the
// keys: 96 rows over the same sequence take 52.9 us.  Strides that no tensor map
// takes (8-byte copies): 68 and 752 us.
//
// Mathematics.  With t = softmax_scale log2(e) s_K (q . dec(K)) the score of a
// key in log2 units and g = log2 s_V of its block, its weight is
// w = 2^(t + g - m), m a running reference of t + g per row: O accumulates
// w dec(V) (FP16 weights, FP32 sums) and l accumulates w / s_V in FP32 from
// the unrounded weight, so O / l = sum e^z s_V dec(V) / sum e^z for any m.
// Within 2^-40 .. 2^40 no scale makes a weight or a sum overflow.
// w is FP16 as in the head-scaled kernels (the tensor product takes one type for
// both operands, and BF16 would leave it 8 bits): with m the largest t + g of the
// tile that set it, a weight below 2^-14 of the row's largest is off by up to
// 2^-25 of that, and l, which has it unrounded, counts it all the same.  Putting
// m 7 below the largest instead (weights from 2^7, the next raise after a growth
// of 2^8 instead of 2^15) would make that 2^-32, for more raises: 262144 tokens
// of 48 rows of 256 took 39.1 us instead of 35.0, 16 sequences over 64 blocks of
// 64 42.2 instead of 41.6.
//
// Warp roles (20 warps; a 21st would leave a sixth warp on one scheduler and 80
// instead of 96 registers per thread: 1.2 times as long), each running through
// all segments so that the copies and decodes of a segment overlap the end of
// the previous one:
//   K / V producer  : walk the block table (or the visit list) and issue TMA
//                     loads (128-byte swizzle) of 16, 32 or 64 keys, whatever
//                     the page (block) is a multiple of, into rings of raw
//                     half-tiles.  (Boxes of 16 keys of 128 bytes held the
//                     copies to 0.71 of the copy peak with all other work
//                     taken out, boxes of 64 to 0.88.)  Their loops are one
//                     warp's serial code and bound the copies of small keys:
//                     with the scales passed by one of them the batch above
//                     took 266 us.  The K producer also plans the segments.
//   K decoders (4)  : thread = key; exact FP8 -> FP16 into tensor memory, the
//                     A operand of S^T = K . Q^T.
//   V decoders (4)  : transposing 8-bit ldmatrix, the same conversion, into
//                     tensor memory, the A operand of O^T = V^T . P^T.
//   score MMA, value MMA: one thread each issues the products of a tile.  The
//                     score warp also passes on the scales (positions, masks)
//                     of 512 keys at a time, one 16-key box per lane, requested
//                     512 keys ahead.
//   softmax (8)     : thread = key, half of the N rows each.  The reference m
//                     of a row is raised only when a weight would pass 2^15
//                     (one vote per tile); then only the rows concerned, and
//                     only the groups of 8 accumulator columns that hold them,
//                     are rescaled.  (The first tile raises every row: its
//                     maxima by one warp reduction per row instead of shuffles
//                     took 262144 tokens of 48 rows of 256 from 43.0 to 37.3
//                     us.)  At a segment's end they load the next
//                     segment's queries while the value product runs, then
//                     write the rows out.
//
// Every mbarrier wait is bounded; on expiry the CTA raises an abort flag,
// every role winds down, outstanding copies and MMAs are drained, TMEM is
// freed and the CTA's segments are marked invalid (status TIMEOUT).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {
namespace seg {

constexpr int kUnitCost = 3;   // half-tiles of time that a segment's set-up and end take
constexpr int kMaxSeg = 64;    // segments a CTA plans at a time

struct Segment {
  int b;        // sequence (kListed: stream)
  int h_rg;     // KV head | row group << 16
  int k0, k1;   // keys (kListed: along the visit list)
  int L, ql;    // length and queries of the sequence
  int slot;     // of the partial state; -1: the whole unit, finished here
  int pad;
};

template <int D, int N>
struct Cfg {
  static_assert(N % 16 == 0 && N >= 16 && N <= 64, "rows per CTA");
  static constexpr int NSW = 8;                 // softmax warps
  static constexpr int NC = N / 2;              // rows per softmax thread
  static constexpr int IB = D < 128 ? D : 128;  // bytes of a swizzled row
  static constexpr int SMASK = IB == 128 ? 7 : 3;     // 128B / 64B swizzle
  static constexpr int DB = D / 64 < 2 ? 2 : D / 64;  // 64-d blocks of V^T (D=64 padded)
  static constexpr int MH = DB / 2;             // 128-row M halves of V^T.P^T
  static constexpr int SC = (N + 31) / 32 * 32; // TMEM columns per accumulator
  // K tiles in TMEM and P^T tiles in shared memory: two where a key is at most
  // 128 bytes; else one K tile, released in two halves for N = 16
  static constexpr int NKB = D <= 128 ? 2 : 1;
  static constexpr int NPT = D <= 128 ? 2 : 1;
  static constexpr int KFG = (N <= 16 && D > 128) ? 2 : 1;
  static constexpr int KCOL = 0, SCOL = 128, OCOL = 128 + 2 * SC;
  static constexpr int VCOL = OCOL + MH * SC;
  static constexpr int VTC = MH * 32;           // columns per V^T half-tile
  static constexpr int NVF = (512 - VCOL) / VTC < 4 ? (512 - VCOL) / VTC : 4;
  static constexpr int QB = (D / 64) * N * 128; // Q, K-major SW128
  static constexpr int PB = 128 * 128;          // P^T, MN-major SW128 (N <= 64)
  static constexpr int RSLOT = 64 * D;          // one raw K or V half-tile
  static constexpr int LIMIT = 232448 - 1024;   // opt-in maximum minus alignment slack
  // groups of 512 keys whose scales are held: the score warp runs two tiles
  // ahead of the softmax and must not wait for it here
  static constexpr int NSG = 4;
  // small region: barriers, scalars, row state, scale boxes, segments
  static constexpr int S_SCAL = 640, S_M = 704, S_BASE = S_M + 512, S_THR = S_BASE + 512,
                       S_POS = S_THR + 512, S_ROW = S_POS + 256, S_RED = S_ROW + 1024,
                       S_LINV = S_RED + 1024, S_BOX = S_LINV + 256, S_MASK = S_BOX + NSG * 512,
                       S_SEG = S_MASK + NSG * 128, S_BAD = S_SEG + kMaxSeg * 32,
                       SMALL = S_BAD + kMaxSeg * 4;
  static constexpr int NRAW = (LIMIT - QB - NPT * PB - SMALL) / RSLOT;
  static constexpr int NVM = D <= 128 ? 8 : 4;
  static constexpr int NKR = NRAW / 2 < 8 ? NRAW / 2 : 8;
  static constexpr int NVR = NRAW - NKR < NVM ? NRAW - NKR : NVM;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + QB;
  static constexpr int OFF_KR = OFF_P + NPT * PB;
  static constexpr int OFF_VR = OFF_KR + NKR * RSLOT;
  static constexpr int OFF_SMALL = OFF_VR + NVR * RSLOT;
  static constexpr int SMEM = OFF_SMALL + SMALL + 1024;
  static constexpr int NTHREADS = 32 * 20;
  static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + NKR, B_VFULL = B_KEMPTY + NKR,
                       B_VEMPTY = B_VFULL + NVR, B_KREADY = B_VEMPTY + NVR,
                       B_KFREE = B_KREADY + NKB, B_VREADY = B_KFREE + NKB * KFG,
                       B_VFREE = B_VREADY + NVF, B_SFULL = B_VFREE + NVF, B_SFREE = B_SFULL + 2,
                       B_PREADY = B_SFREE + 2, B_PVDONE = B_PREADY + NPT,
                       B_SCFULL = B_PVDONE + NPT, B_SCEMPTY = B_SCFULL + NSG,
                       B_QREADY = B_SCEMPTY + NSG, B_DRAINQK = B_QREADY + 1,
                       B_DRAINPV = B_DRAINQK + 1, NBARS = B_DRAINPV + 1;
  static_assert(NBARS * 8 <= S_SCAL, "barriers");
  static_assert(NKB == 1 || (NKR >= 4 && KFG == 1 && D / 2 * NKB <= 128), "K tiles in TMEM");
  static_assert(NKR >= 2 && NVF >= 2 && NVR >= NVF, "slot reuse order (see the decoders)");
  static_assert(VCOL + NVF * VTC <= 512, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(NC % 8 == 0 && sizeof(Segment) == 32, "layout");
};

enum : int { kWSoftmax = 0, kWKDec = 8, kWVDec = 12, kWKProd = 16, kWVProd = 17, kWQk = 18,
             kWPv = 19 };

__device__ __forceinline__ uint32_t sw128(uint32_t off) { return off ^ (((off >> 7) & 7u) << 4); }

// maximum over the warp (a NaN does not count)
__device__ __forceinline__ float warp_max(float x) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(d) : "f"(x));
  return d;
}

// ---------------------------------------------------------------------------
// The plan: which segments a CTA walks.

// (tokens, queries) of group x: a sequence, or a stream of the visit lists;
// tokens = 0 if it has nothing to walk.
__device__ __forceinline__ int2 group_len(const SegParams &p, int x) {
  const int L = p.pairs[(int64_t)x * p.pair_sb];
  const int ql = p.has_qlen ? p.pairs[(int64_t)x * p.pair_sb + 1] : p.Qmax;
  const bool live = L > 0 && L <= p.capacity && ql > 0 && ql <= p.Qmax && ql <= L;
  return make_int2(live ? L : 0, ql);
}

// Where the plan's lengths come from: staged in shared memory, read as they
// are (st = null), or, for a dry run, one invented group.
struct Lengths {
  const int2 *st;
  int groups;
  bool dry;
  __device__ __forceinline__ int2 of(const SegParams &p, int x) const {
    if (x >= groups) return make_int2(0, 0);
    if (dry) return make_int2(640, 1);
    return st ? st[x] : group_len(p, x);
  }
};

// A group's row groups with a live query (its units are heads x row groups,
// at most two: 96 rows in groups of 48) and a unit's places.
__device__ __forceinline__ int row_groups(const SegParams &p, int2 v, int N) {
  return v.x <= 0 ? 0 : v.y * p.G > N ? 2 : 1;
}
__device__ __forceinline__ int unit_places(int2 v) { return kUnitCost + (v.x + 63) / 64; }

// One warp: the segments of CTA `cta` into seg[], at most kMaxSeg, from place
// state[2] on (first: from the CTA's first, after the line's length has been
// counted); leaves the line and the place to go on from (its end: the CTA's
// last place) in state[0 .. 2] and (segments, 1 if more follow) in state[-2],
// state[-1].  The CTA where a unit starts records its first CTA and its parts
// for the combine (parts = -1: finished in one CTA).
// A batch of up to 32 groups is read by the warp itself and scanned once.
template <bool LISTED>
static __device__ __noinline__ void plan_segments(const SegParams &p, Lengths len, int N, int cta,
                                                  bool first, volatile int *state, Segment *seg,
                                                  int *bad, int lane) {
  int2 v = make_int2(0, 0);
  int2 vis = make_int2(0, 0);  // LISTED: tokens to walk and length of the stream
  const bool known = LISTED && len.groups <= 32 && !len.dry;
  if (known) {
    if (lane < len.groups) {
      const BlockStream r = p.streams[lane];
      v = make_int2(r.ql > 0 ? r.n16 : 0, r.ql);  // (the list's writer has checked them)
      vis = make_int2(r.n, r.L);
    }
  } else {
    v = len.of(p, lane);
  }
  int rgs, pl, cost, incl;
  auto scan = [&]() {  // the lane's places, and those up to its end in the chunk
    rgs = row_groups(p, v, N);
    pl = unit_places(v);
    cost = p.unit_heads * rgs * pl;
    incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
  };
  scan();
  int total, q, from;
  if (first) {
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (len.groups > 32) {
      int sum = 0;
      for (int x0 = 32; x0 < len.groups; x0 += 128) {
        int2 w[4];  // four groups per lane in flight
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = len.of(p, x0 + 32 * e + lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum += p.unit_heads * row_groups(p, w[e], N) * unit_places(w[e]);
      }
      total += (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
    }
    q = total > 0 ? (total + p.ctas - 1) / p.ctas : 1;
    from = cta * q;
  } else {
    total = state[0];
    q = state[1];
    from = state[2];
  }
  const int end = min((cta + 1) * q, total);
  int n = 0, next = end;
  int base = 0;  // place where group x0 starts
  for (int x0 = 0; x0 < len.groups && base < end; x0 += 32) {
    if (x0 > 0) {
      v = len.of(p, x0 + lane);
      scan();
    }
    const int start = base + incl - cost;
    const bool is_hit = cost > 0 && start < end && start + cost > from;
    if (LISTED && is_hit && !known && !len.dry) {
      const BlockStream rec = p.streams[x0 + lane];
      vis = make_int2(rec.n, rec.L);
    }
    unsigned hit = __ballot_sync(0xffffffffu, is_hit);
    base += __shfl_sync(0xffffffffu, incl, 31);
    while (hit) {
      const int src = __ffs(hit) - 1;
      hit &= hit - 1;
      const int gs = __shfl_sync(0xffffffffu, start, src);
      const int n_rg = __shfl_sync(0xffffffffu, rgs, src), gp = __shfl_sync(0xffffffffu, pl, src);
      const int gl = __shfl_sync(0xffffffffu, v.x, src), gq = __shfl_sync(0xffffffffu, v.y, src);
      const int vn = __shfl_sync(0xffffffffu, vis.x, src), vl = __shfl_sync(0xffffffffu, vis.y, src);
      const int gu = p.unit_heads * n_rg, nh = gp - kUnitCost;
      const int u0 = from > gs + gp ? (from - gs) / gp : 0;
      for (int ub = u0; ub < gu && gs + ub * gp < end; ub += 32) {
        const int u = min(ub + lane, gu);
        const int us = gs + u * gp + kUnitCost;  // place of its first half-tile
        // half-tiles in this CTA (at most once per CTA: `from` is a unit's start later on)
        const int a = max(us, cta * q), z = min(us + nh, end);
        const bool mine = u < gu && z > a && us - kUnitCost + gp > from;
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        const int at = n + __popc(m & ((1u << lane) - 1u));
        if (mine && at < kMaxSeg) {
          const int h = u >> (n_rg - 1), rg = u - h * n_rg;
          Segment s;
          s.b = x0 + src;
          s.h_rg = h | rg << 16;
          s.k0 = (a - us) * 64;
          s.k1 = min((z - us) * 64, gl);
          s.L = gl;
          s.ql = gq;
          const bool starts = a == us, ends = z == us + nh;
          s.slot = !starts ? p.ctas + cta : ends ? -1 : cta;
          s.pad = 0;
          if (LISTED && !len.dry) {
            s.h_rg = s.b % p.Hkv | rg << 16;
            s.k1 = min(s.k1, vn);
            s.L = vl;
          }
          seg[at] = s;
          bad[at] = 0;
          if (starts && !len.dry) {
            const int str = LISTED ? s.b : s.b * p.Hkv + h;
            const int parts = ends ? -1 : (us + nh - 1) / q - cta + 1;
            p.tab[(int64_t)str * p.n_rg + rg] = make_int2(cta, parts);
          }
        }
        n += __popc(m);
        if (n > kMaxSeg) {  // full: go on from the first unit that did not fit
          const int left = __popc(m) - (n - kMaxSeg);  // of this round's that fit
          unsigned mm = m;
          for (int k = 0; k < left; ++k) mm &= mm - 1;
          next = gs + (ub + __ffs(mm) - 1) * gp;
          n = kMaxSeg;
          goto done;
        }
      }
    }
  }
done:
  __syncwarp();
  if (lane == 0) {
    state[0] = total;
    state[1] = q;
    state[2] = next;
    state[-2] = n;
    state[-1] = n > 0 && next < end;
  }
}

// The same for a batch of one unit: no scan (0.7 to 1.2 us less to the first copy).
template <bool LISTED>
static __device__ __noinline__ void plan_one(const SegParams &p, Lengths len, int cta,
                                             volatile int *state, Segment *seg, int *bad, int lane) {
  int2 v, vis = make_int2(0, 0);
  if (LISTED && !len.dry) {
    const BlockStream r = p.streams[0];
    v = make_int2(r.ql > 0 ? r.n16 : 0, r.ql);
    vis = make_int2(r.n, r.L);
  } else {
    v = len.of(p, 0);
  }
  const int total = v.x > 0 ? unit_places(v) : 0;
  const int q = total > 0 ? (total + p.ctas - 1) / p.ctas : 1;
  const int a = max(kUnitCost, cta * q), end = min((cta + 1) * q, total);
  if (lane == 0) {
    if (end > a) {
      const bool starts = a == kUnitCost, ends = end == total;
      Segment s;
      s.b = 0;
      s.h_rg = 0;
      s.k0 = (a - kUnitCost) * 64;
      s.k1 = min((end - kUnitCost) * 64, LISTED && !len.dry ? vis.x : v.x);
      s.L = LISTED && !len.dry ? vis.y : v.x;
      s.ql = v.y;
      s.slot = !starts ? p.ctas + cta : ends ? -1 : cta;
      s.pad = 0;
      seg[0] = s;
      bad[0] = 0;
      if (starts && !len.dry) p.tab[0] = make_int2(cta, ends ? -1 : (total - 1) / q - cta + 1);
    }
    state[-2] = end > a;
    state[-1] = 0;
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Zero the raw V bytes of keys kz .. 63 of a half-tile slot in the columns
// V decoder warp dq reads (d = 128 mh + 32 dq + 0..31).  The slot was written
// by the tensor copy (async proxy) and will be again after the decoders
// release it, hence the proxy fence after the generic stores.  lb: log2 of
// the keys per box.
template <int D, int IB, int SMASK, int MH>
static __device__ __noinline__ void zero_v_tail(uint8_t *raw, int kz, int lb, int dq, int lane) {
  constexpr int NG = 2 * MH;  // 16-byte column granules of the warp per key
  for (int i = lane; i < (64 - kz) * NG; i += 32) {
    const int k = kz + i / NG, g = i % NG;
    const int dch = 128 * (g >> 1) + 32 * dq + 16 * (g & 1);
    if (dch < D) {
      const int dh = dch / IB, cc = (dch % IB) >> 4;
      const uint32_t off = (uint32_t)((k & ((1 << lb) - 1)) * IB + cc * 16);
      *reinterpret_cast<uint4 *>(raw + ((k >> lb) << lb) * D + dh * (IB << lb) +
                                 (off ^ (((off >> 7) & SMASK) << 4))) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}

// Copies of one half-tile for caches whose strides are multiples of 8 bytes
// but not all of 16, which no tensor map can describe: 8-byte asynchronous
// copies into the layout of 16-key boxes; each lane's completion arrives on
// the slot's "full" barrier (32 arrivals per phase).  Keys at or past `keys`
// and pages below zero are zero-filled.  phys, box: lanes 0-3, their box.
template <int D>
static __device__ __noinline__ void copy_half(const uint8_t *hbase, int64_t ps, int64_t ts, int keys,
                                              int phys, int box, uint32_t slot, uint32_t full,
                                              int lane) {
  constexpr int IB = D < 128 ? D : 128, SMASK = IB == 128 ? 7 : 3;
  constexpr int CPK = D / 8, KPI = 32 / CPK;  // 8-byte chunks per key, keys per instruction
  const uint64_t pol = tc::l2_evict_first_policy();
  const int c = lane % CPK, kk = lane / CPK;
  const int dh = (8 * c) / IB, cb = (8 * c) % IB;  // this lane's chunk: IB block, byte in it
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const int pg = __shfl_sync(0xffffffffu, phys, g);
    const int sb = __shfl_sync(0xffffffffu, box, g);
    const uint8_t *src = hbase + (int64_t)max(pg, 0) * ps + (int64_t)(16 * sb + kk) * ts + 8 * c;
#pragma unroll
    for (int r = kk; r < 16; r += KPI) {
      const bool ok = pg >= 0 && 16 * g + r < keys;
      const uint32_t off = (uint32_t)(r * IB + cb);
      tc::cp_async8_hint(slot + g * (16 * D) + dh * (16 * IB) + (off ^ (((off >> 7) & SMASK) << 4)),
                         ok ? src : hbase, ok ? 8 : 0, pol);
      src += KPI * ts;
    }
  }
  tc::cp_async_mbar_arrive_noinc(full);
}

// ---------------------------------------------------------------------------
template <int D, int N, bool LISTED>
__global__ void __launch_bounds__(Cfg<D, N>::NTHREADS, 1)
    seg_kernel(const SegParams p, const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v) {
  using C = Cfg<D, N>;
  constexpr int kKFull = C::B_KFULL, kKEmpty = C::B_KEMPTY, kVFull = C::B_VFULL,
                kVEmpty = C::B_VEMPTY, kKReady = C::B_KREADY, kKFree = C::B_KFREE,
                kVReady = C::B_VREADY, kVFree = C::B_VFREE, kSFull = C::B_SFULL,
                kSFree = C::B_SFREE, kPReady = C::B_PREADY, kPvDone = C::B_PVDONE,
                kScFull = C::B_SCFULL, kScEmpty = C::B_SCEMPTY, kQReady = C::B_QREADY,
                kDrainQk = C::B_DRAINQK, kDrainPv = C::B_DRAINPV;
  extern __shared__ uint8_t smem_raw[];
  const float kInf = __int_as_float(0x7f800000);
  constexpr float kLog2e = 1.4426950408889634f;
  // lazy-rescale threshold (log2 units): P <= 2^15, inside FP16
  constexpr float kTau = 15.0f;

  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (sbase - raw_addr);
  const uint32_t sQ = sbase + C::OFF_Q, sP = sbase + C::OFF_P, sKR = sbase + C::OFF_KR,
                 sVR = sbase + C::OFF_VR, sSm = sbase + C::OFF_SMALL;
  uint8_t *gP = gbase + C::OFF_P, *gKR = gbase + C::OFF_KR, *gSm = gbase + C::OFF_SMALL;
  auto bar = [&](int i) -> uint32_t { return sSm + 8u * (uint32_t)i; };
  volatile int *abort_f = reinterpret_cast<volatile int *>(gSm + C::S_SCAL);
  // segments, 1 if more follow; the line's places, those per CTA, the next place
  int *nseg_s = reinterpret_cast<int *>(gSm + C::S_SCAL + 8);
  Segment *seg_s = reinterpret_cast<Segment *>(gSm + C::S_SEG);
  int *bad_s = reinterpret_cast<int *>(gSm + C::S_BAD);         // per segment

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool producer = warp == kWKProd || warp == kWVProd;
  const int cta = blockIdx.x;
  const bool one_unit = p.groups == 1 && p.unit_heads * p.n_rg == 1;

  // ---- set-up that touches only this CTA's shared memory and TMEM, done
  // before the grid dependency wait so it overlaps the previous kernel's tail
  static_assert(C::NBARS <= 96, "one thread per barrier");
  if (tid < 96) {
    if (const int i = tid; i < C::NBARS) {
      uint32_t cnt = 1;
      if (i >= kKEmpty && i < kKEmpty + C::NKR)
        cnt = 64;
      else if ((i >= kKReady && i < kKReady + C::NKB) || (i >= kVEmpty && i < kVEmpty + C::NVR) ||
               (i >= kVReady && i < kVReady + C::NVF))
        cnt = 128;
      else if ((i >= kSFree && i < kSFree + 2) || (i >= kPReady && i < kPReady + C::NPT) ||
               (i >= kScEmpty && i < kScEmpty + C::NSG) || i == kQReady)
        cnt = 32 * C::NSW;
      else if (i >= kScFull && i < kScFull + C::NSG)
        cnt = 32;
      else if (p.cpasync && ((i >= kKFull && i < kKFull + C::NKR) ||
                             (i >= kVFull && i < kVFull + C::NVR)))
        cnt = 32;  // one arrival per producer lane (8-byte copies)
      tc::mbar_init(bar(i), cnt);
    }
    if (tid == 0) *abort_f = 0;
  }
  if (producer && lane == 0 && !p.cpasync)  // kernel parameters
    tc::prefetch_tensormap(warp == kWVProd ? &tmap_v : &tmap_k);
  if (warp == kWKProd) {
    // The plan's code runs once on an invented batch, while the previous kernel
    // ends and the barriers and TMEM are set up: its instructions are then at
    // hand when the lengths arrive (its first run took 6000 cycles).
    const Lengths dry{nullptr, 1, true};
    if (one_unit)
      plan_one<LISTED>(p, dry, 0, nseg_s + 2, seg_s, bad_s, lane);
    else
      plan_segments<LISTED>(p, dry, N, 0, true, nseg_s + 2, seg_s, bad_s, lane);
  }
  if (warp == kWQk) {
    tc::tmem_alloc(sSm + C::S_SCAL + 4, 512);
    tc::tmem_relinquish();
  }
  tc::mbar_fence_init();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t *>(gSm + C::S_SCAL + 4);
  if (tbase != 0u) *abort_f = 1;  // never: all 512 columns are the CTA's, from column 0
  // launched as a programmatic dependent: everything below may read what the
  // previous kernel on the stream wrote or overwrite what it reads
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  // the combine may be placed as SMs free up; it waits for this grid
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  const long long LIM = p.wait_limit;
  const int lb = p.box_log2;  // keys per tensor copy
  // counters of the role that run through all segments: half-tiles or tiles,
  // and segments (score MMA) or groups of scales (softmax)
  int count = 0, count2 = 0;
  int groups = 0;  // of scales passed (score MMA)
  bool mma_issued = false;
  bool first = true;

  for (;;) {  // up to kMaxSeg segments at a time
    // Whether the roles run is one answer for the CTA, read here, where no role
    // runs that could raise the flag: the softmax warps meet at barriers that
    // have no time limit, so they enter all or none.
    const bool wound_down = *abort_f != 0;
    // ---- the plan, by the K producer; the lengths of more than 32 groups are
    // staged by all threads in the K ring (idle here), but read as they are if
    // they do not fit, or if copies that a timed-out batch of segments left in
    // flight may still write the ring
    const bool staged = !wound_down && p.groups > 32 && p.groups <= C::NKR * C::RSLOT / 8;
    int2 *st_len = reinterpret_cast<int2 *>(gKR);
    if (staged) {
      for (int x = tid; x < p.groups; x += C::NTHREADS) st_len[x] = group_len(p, x);
      __syncthreads();
    }
    if (warp == kWKProd) {
      const Lengths len{staged ? st_len : nullptr, p.groups, false};
      if (one_unit)
        plan_one<LISTED>(p, len, cta, nseg_s + 2, seg_s, bad_s, lane);
      else
        plan_segments<LISTED>(p, len, N, cta, first, nseg_s + 2, seg_s, bad_s, lane);
    }
    if (staged) tc::fence_proxy_async_smem();  // the ring is next written by tensor copies
    __syncthreads();
    const int nseg = nseg_s[0];
    const bool more = nseg_s[1] != 0;
    auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {  // one answer for the warp
      return __all_sync(0xffffffffu, tc::mbar_wait_brief(b, parity, abort_f, LIM));
    };
    auto tiles_of = [&](int s) -> int { return (seg_s[s].k1 - seg_s[s].k0 + 127) >> 7; };

    if (wound_down) {
      // (the segments are only marked below)
    } else if (producer) {
      // =============================== producers (K ring, V ring)
      const bool isv = warp == kWVProd;
      const int nslot = isv ? C::NVR : C::NKR;
      const int fullb = isv ? kVFull : kKFull, emptyb = isv ? kVEmpty : kKEmpty;
      const uint32_t ring = isv ? sVR : sKR;
      const uint64_t pol = tc::l2_evict_first_policy();
      const CUtensorMap *map = isv ? &tmap_v : &tmap_k;
      const int unit = LISTED ? p.blk : p.page;  // tokens per table (list) entry
      const int nbox = 64 >> lb;                 // copies per half-tile
      const unsigned long long unit_m = LISTED ? p.blk_m : p.page_m;
      int st = 0, u = 0;  // ring slot and its pass
      if (count > 0) {
        u = count / nslot;
        st = count - u * nslot;
      }
      // Copies are prepared 32 at a time, one per lane (its page, and its
      // token in the page), from table entries requested a group ahead: the
      // loop over half-tiles is one warp's serial code and its length is what
      // bounds the copies of small keys.
      auto next_group = [&](int2 it) -> int2 {  // (segment, group of 32 copies) after it
        if (it.x >= nseg) return it;
        return seg_s[it.x].k0 + ((it.y + 1) << (5 + lb)) < seg_s[it.x].k1 ? make_int2(it.x, it.y + 1)
                                                                        : make_int2(it.x + 1, 0);
      };
      auto copy_key = [&](int2 it) -> int {  // the lane's key in the group, -1: past the segment
        if (it.x >= nseg) return -1;
        const int key = seg_s[it.x].k0 + (it.y << (5 + lb)) + (lane << lb);
        return key < seg_s[it.x].k1 ? key : -1;
      };
      int2 raw = make_int2(-1, 0);  // the entry's page and first 16-token box in the page
      auto request = [&](int2 it) {
        const int key = copy_key(it);
        raw = make_int2(-1, 0);
        if (key >= 0) {
          if constexpr (LISTED)
            raw = load_dep(reinterpret_cast<const int2 *>(
                p.list + (int64_t)seg_s[it.x].b * p.list_cap + div16(key, unit_m)));
          else
            raw.x = load_dep(p.bt + (int64_t)seg_s[it.x].b * p.bt_sb + div16(key, unit_m));
        }
      };
      int page = 0, tok = 0;  // of the lane's copy; the page past the last one reads as zeros
      auto prepare = [&](int2 it) {
        const int key = copy_key(it);
        tok = key >= 0 ? key - div16(key, unit_m) * unit + 16 * raw.y : 0;
        page = raw.x;
        if (key >= 0 && (page < 0 || page >= p.n_pages)) atomicOr(&bad_s[it.x], 1);
        if (page < 0 || page >= p.n_pages) page = (int)p.n_pages;
      };
      int2 itc = make_int2(0, 0);
      request(itc);
      bool ok = true;
      auto produce = [&](auto nb_tag) {
        constexpr int NB = decltype(nb_tag)::value;  // copies per half-tile
        for (int s = 0; s < nseg && ok; ++s) {
          const int h = seg_s[s].h_rg & 0xFFFF;
          const int nhalf = 2 * tiles_of(s);
          for (int t = 0; t < nhalf; ++t) {
            if (t % (32 / NB) == 0) {  // (a half-tile past the segment's end may start a group)
              if (itc.x == s) {
                prepare(itc);
                itc = next_group(itc);
                request(itc);
              } else {
                page = (int)p.n_pages;
              }
            }
            if (u > 0 && !(ok = warp_wait(bar(emptyb + st), (u - 1) & 1))) break;
            const uint32_t slot = ring + st * C::RSLOT, full = bar(fullb + st);
            if (!p.cpasync) {
              int pg[NB], tk[NB];
#pragma unroll
              for (int g = 0; g < NB; ++g) {
                pg[g] = __shfl_sync(0xffffffffu, page, (t * NB + g) & 31);
                tk[g] = __shfl_sync(0xffffffffu, tok, (t * NB + g) & 31);
              }
              if (tc::elect_one()) {
                tc::mbar_arrive_expect_tx(full, C::RSLOT);
                // one copy: 64 / NB keys x D bytes of head h, as blocks of rows
                // of IB bytes (swizzled); coordinates (byte, token in page,
                // block, head, page)
#pragma unroll
                for (int g = 0; g < NB; ++g)
                  tc::tma_load_5d_hint(slot + g * (64 / NB) * D, map, 0, tk[g], 0, h, pg[g], full, pol);
              }
              __syncwarp();
            } else {
              const int mine = __shfl_sync(0xffffffffu, page, (t * 4 + lane) & 31);
              const int box = __shfl_sync(0xffffffffu, tok, (t * 4 + lane) & 31) >> 4;
              const uint8_t *hb = (isv ? p.v_base : p.k_base) + (int64_t)h * (isv ? p.v_hs : p.k_hs);
              copy_half<D>(hb, isv ? p.v_ps : p.k_ps, isv ? p.v_ts : p.k_ts,
                           seg_s[s].k1 - seg_s[s].k0 - 64 * t, mine < p.n_pages ? mine : -1, box, slot,
                           full, lane);
            }
            ++count;
            if (++st == nslot) {
              st = 0;
              ++u;
            }
          }
        }
      };
      if (nbox == 1)
        produce(std::integral_constant<int, 1>{});
      else if (nbox == 2)
        produce(std::integral_constant<int, 2>{});
      else
        produce(std::integral_constant<int, 4>{});
    } else if (warp == kWQk) {
      // =============================== score MMA issuer: S^T = K . Q^T
      // The whole warp runs the loop and one elected lane issues, so that the
      // operands stay in uniform registers (TMEM addresses are constants: the
      // CTA holds all 512 columns).
      // ---- scales, four tiles at a time: lane = one 16-key box of a group of
      // 512 keys (a box lies in one block).  A group is requested a group ahead
      // of its use, the page ids that lead to it two.
      float4 *box_s = reinterpret_cast<float4 *>(gSm + C::S_BOX);
      uint32_t *mask_s = reinterpret_cast<uint32_t *>(gSm + C::S_MASK);
      auto step = [&](int2 it) -> int2 {  // (segment, group) after it
        if (it.x >= nseg) return it;
        return 4 * (it.y + 1) < tiles_of(it.x) ? make_int2(it.x, it.y + 1) : make_int2(it.x + 1, 0);
      };
      auto key_of = [&](int2 it) -> int {  // -1: past the segment
        if (it.x >= nseg) return -1;
        const int key = seg_s[it.x].k0 + 512 * it.y + 16 * lane;
        return key < seg_s[it.x].k1 ? key : -1;
      };
      auto load_page = [&](int2 it) -> int {
        if constexpr (LISTED) return 0;
        const int key = key_of(it);
        return key >= 0 ? load_dep(p.bt + (int64_t)seg_s[it.x].b * p.bt_sb + div16(key, p.page_m)) : -1;
      };
      float4 f = make_float4(0.f, 0.f, 1.f, 0.f);  // (s_K, s_V); listed: the entry's
      int2 e = make_int2(0, 0);                    // listed: first token, mask
      bool live = false;
      auto load_scales = [&](int2 it, int page) {
        const int key = key_of(it);
        live = key >= 0;
        if constexpr (LISTED) {
          if (live) {
            const int x = div16(key, p.blk_m);
            const BlockEntry *en = p.list + (int64_t)seg_s[it.x].b * p.list_cap + x;
            e = load_dep(reinterpret_cast<const int2 *>(&en->tok0));
            e.x += key - x * p.blk;
            f = load_dep(reinterpret_cast<const float4 *>(&en->alpha));
          }
        } else {
          live = live && page >= 0 && page < p.n_pages;
          if (live) {
            const float *sp = p.scales + (int64_t)page * p.s_page +
                              (int64_t)(seg_s[it.x].h_rg & 0xFFFF) * p.s_head +
                              (div16(key, p.blk_m) - div16(key, p.page_m) * p.page_blocks);
            f.x = load_dep(sp);
            f.y = load_dep(sp + p.s_kv);
          }
        }
      };
      int2 it0 = make_int2(0, 0), it1 = step(it0);
      int page1 = -1;
      load_scales(it0, load_page(it0));
      page1 = load_page(it1);
      auto pass_scales = [&]() -> bool {  // group it0; then request the next
        const int sl = groups % C::NSG;
        if (groups >= C::NSG && !warp_wait(bar(kScEmpty + sl), (groups / C::NSG - 1) & 1))
          return false;
        float4 o = make_float4(0.f, 0.f, 1.f, 0.f);  // past the segment, or invalid
        if (live) {
          if constexpr (LISTED) {
            o = make_float4(f.x, f.y, f.z, __int_as_float(e.x));
            mask_s[sl * 32 + lane] = (uint32_t)e.y;
          } else {
            const float sk = f.x, sv = f.y;
            if (sk >= kMinScale && sk <= kMaxScale && sv >= kMinScale && sv <= kMaxScale)
              o = make_float4(p.sm_scale * kLog2e * sk, __log2f(sv), __fdividef(1.f, sv), 0.f);
            else
              atomicOr(&bad_s[it0.x], 2);
          }
        }
        box_s[sl * 32 + lane] = o;
        tc::mbar_arrive(bar(kScFull + sl));
        ++groups;
        load_scales(it1, page1);
        it0 = it1;
        it1 = step(it1);
        page1 = load_page(it1);
        return true;
      };
      constexpr uint32_t id_qk = tc::idesc_f16(128, N, 0, 0);
      const uint64_t dq0 = tc::smem_desc(sQ, 16, 1024);
      bool ok = true;
      for (int s = 0; s < nseg && ok; ++s, ++count2) {
        const int ntiles = tiles_of(s);
        if (!(ok = warp_wait(bar(kQReady), count2 & 1))) break;
        for (int jl = 0; jl < ntiles; ++jl, ++count) {
          const int j = count, kb = j % C::NKB;
          if ((jl & 3) == 0 && !(ok = pass_scales())) break;
          if (!(ok = warp_wait(bar(kKReady + kb), (j / C::NKB) & 1))) break;
          if (j >= 2 && !(ok = warp_wait(bar(kSFree + (j & 1)), ((j >> 1) - 1) & 1))) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint32_t d = C::SCOL + (j & 1) * C::SC;
            constexpr int MPG = D / 16 / C::KFG;  // MMAs per released group
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              tc::mma_ts(d, C::KCOL + kb * 64 + ks * 8,
                         dq0 + (((ks >> 2) * (N * 128) + (ks & 3) * 32) >> 4), id_qk, ks > 0);
              if constexpr (C::KFG > 1)
                if ((ks + 1) % MPG == 0) tc::mma_commit(bar(kKFree + ks / MPG));
            }
            tc::mma_commit(bar(kSFull + (j & 1)));
            if constexpr (C::KFG == 1) tc::mma_commit(bar(kKFree + kb));
          }
          __syncwarp();
          mma_issued = true;
        }
      }
    } else if (warp == kWPv) {
      // =============================== value MMA issuer: O^T += V^T . P^T
      constexpr uint32_t id_pv = tc::idesc_f16(128, N, 0, 1);
      const uint64_t dp0 = tc::smem_desc(sP, 16384, 1024);
      bool ok = true;
      for (int s = 0; s < nseg && ok; ++s) {
        const int ntiles = tiles_of(s);
        for (int jl = 0; ok && jl < ntiles; ++jl, ++count) {
          const int pb = count % C::NPT;
          if (!(ok = warp_wait(bar(kPReady + pb), (count / C::NPT) & 1))) break;
#pragma unroll
          for (int kh = 0; kh < 2; ++kh) {
            const int t = 2 * count + kh, vs = t % C::NVF;
            if (!(ok = warp_wait(bar(kVReady + vs), (t / C::NVF) & 1))) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int mh = 0; mh < C::MH; ++mh) {
#pragma unroll
                for (int k4 = 0; k4 < 4; ++k4) {
                  const int ks = kh * 4 + k4;
                  tc::mma_ts(C::OCOL + mh * C::SC, C::VCOL + vs * C::VTC + mh * 32 + k4 * 8,
                             dp0 + ((pb * C::PB + ks * 2048) >> 4), id_pv,
                             (jl > 0 || ks > 0) ? 1u : 0u);
                }
              }
              tc::mma_commit(bar(kVFree + vs));
              if (kh == 1) tc::mma_commit(bar(kPvDone + pb));
            }
            __syncwarp();
            mma_issued = true;
          }
        }
      }
    } else if (warp >= kWKDec && warp < kWVDec) {
      // =============================== K decoders (thread = key)
      const int dq = warp & 3;              // TMEM lane quadrant = keys 32*dq.. of a tile
      const int kh = dq >> 1;               // half-tile of the 128-key tile
      const int kk = 32 * (dq & 1) + lane;  // key within the half-tile
      const uint32_t lane_off = (uint32_t)(32 * dq) << 16;
      const int row = kk & ((1 << lb) - 1);
      const uint32_t key_off = (uint32_t)(((kk >> lb) << lb) * D + row * C::IB);
      const uint32_t swz = ((uint32_t)(row * C::IB) >> 7) & C::SMASK;  // (16-byte chunks of a row)
      int ntl = 0;
      for (int s = 0; s < nseg; ++s) ntl += tiles_of(s);
      auto decode_k = [&](auto e5m2) {
        constexpr bool E5 = decltype(e5m2)::value;
        for (int jl = 0; jl < ntl; ++jl, ++count) {
          // K -> TMEM: column c holds d = 2c (low half), 2c+1 (high half).
          // Wait for the score MMAs that last read this K tile first: they
          // prove every decoder warp finished that tile, hence waited for
          // every earlier use of this raw slot, so the parity wait on the
          // slot below cannot match an older phase.
          const int j = count, t = 2 * j + kh;
          const int st = t % C::NKR, kb = j % C::NKB;
          if (j >= C::NKB && !tc::mbar_wait_brief(bar(kKFree + kb), (j / C::NKB - 1) & 1, abort_f, LIM))
            break;
          if (!tc::mbar_wait_brief(bar(kKFull + st), (t / C::NKR) & 1, abort_f, LIM)) break;
          tc::tc_fence_after();
          const uint8_t *rawK = gKR + st * C::RSLOT + key_off;
          bool ok = true;
#pragma unroll
          for (int grp = 0; grp < D / 64; ++grp) {
            if constexpr (C::KFG > 1) {
              if (grp > 0 && j > 0) {
                if (!(ok = tc::mbar_wait_brief(bar(kKFree + grp * C::KFG / (D / 64)), (j - 1) & 1,
                                         abort_f, LIM)))
                  break;
                tc::tc_fence_after();
              }
            }
            uint32_t r[32];
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const int c = grp * 4 + q4;  // 16-byte chunk of the key row
              const int dh = (c * 16) / C::IB, cc = ((c * 16) % C::IB) >> 4;
              // (rows of 64 bytes share a swizzle line: bit 2 of the chunk
              // is the row's low bit, which key_off carries)
              const uint4 w = *reinterpret_cast<const uint4 *>(rawK + dh * (C::IB << lb) +
                                                               ((cc ^ swz) << 4));
              const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                r[q4 * 8 + 2 * e] = fp8x2_to_f16x2<E5>(wv[e]);
                r[q4 * 8 + 2 * e + 1] = fp8x2_to_f16x2<E5>(wv[e] >> 16);
              }
            }
            const uint32_t (&r0)[16] = *reinterpret_cast<const uint32_t(*)[16]>(&r[0]);
            const uint32_t (&r1)[16] = *reinterpret_cast<const uint32_t(*)[16]>(&r[16]);
            tc::tmem_st16(tbase + lane_off + C::KCOL + kb * 64 + grp * 32, r0);
            tc::tmem_st16(tbase + lane_off + C::KCOL + kb * 64 + grp * 32 + 16, r1);
          }
          if (!ok) break;
          tc::tmem_wait_st();
          tc::tc_fence_before();
          tc::mbar_arrive(bar(kKReady + kb));
          tc::mbar_arrive(bar(kKEmpty + st));
        }
      };
      if (p.e5m2)
        decode_k(std::true_type{});
      else
        decode_k(std::false_type{});
    } else if (warp >= kWVDec && warp < kWKProd) {
      // =============================== V decoders (warp = 32 d per 128-d block)
      const int dq = warp & 3;  // TMEM lane quadrant = d 32*dq.. of each 128-d block
      // ldmatrix rows: threads 0-15 give keys 0-15 of a 16-key group, 16-31
      // the same rows of the next group
      const int pr = lane & 15, pg = lane >> 4;
      uint32_t grp_off[2];  // byte offset of the thread's row in groups 2 kp + pg
      uint32_t swz[2];
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {
        const int key = 16 * (2 * kp + pg) + pr, row = key & ((1 << lb) - 1);
        grp_off[kp] = (uint32_t)(((key >> lb) << lb) * D + row * C::IB);
        swz[kp] = ((uint32_t)(row * C::IB) >> 7) & C::SMASK;
      }
      auto decode_v = [&](auto e5m2) {
        constexpr bool E5 = decltype(e5m2)::value;
        bool ok = true;
        for (int s = 0; s < nseg && ok; ++s) {
          const int keys = seg_s[s].k1 - seg_s[s].k0, nhalf = 2 * tiles_of(s);
          for (int tl = 0; tl < nhalf; ++tl, ++count) {
            // V -> V^T in TMEM (lane = d, column c = keys 2c, 2c+1).  Wait
            // for the value MMA that last read the V^T slot first: it proves
            // half-tiles up to t - NVF >= t - NVR were decoded, i.e. this raw
            // slot's previous use is complete, so the parity wait below is
            // unambiguous.
            const int t = count, st = t % C::NVR, vs = t % C::NVF;
            if (t >= C::NVF &&
                !(ok = tc::mbar_wait_brief(bar(kVFree + vs), ((t / C::NVF) - 1) & 1, abort_f, LIM)))
              break;
            if (!(ok = tc::mbar_wait_brief(bar(kVFull + st), (t / C::NVR) & 1, abort_f, LIM))) break;
            tc::tc_fence_after();
            const uint32_t rawV = sVR + st * C::RSLOT;
            // The box holding the segment's last key is loaded whole; what
            // lies past it may never have been written (a NaN code there would
            // turn the masked key's P = 0 into a NaN product), so this warp
            // zeroes its columns of those keys.
            const int kz = keys - 64 * tl;
            if (kz > 0 && kz < 64 && (kz & ((1 << lb) - 1)) != 0)
              zero_v_tail<D, C::IB, C::SMASK, C::MH>(gbase + C::OFF_VR + st * C::RSLOT, kz, lb, dq,
                                                     lane);
#pragma unroll
            for (int mh = 0; mh < C::MH; ++mh) {
#pragma unroll
              for (int dc = 0; dc < 2; ++dc) {
                const int dch = 128 * mh + 32 * dq + 16 * dc;  // first d of the 16-d chunk
                if (dch < D) {
                  const int dh = dch / C::IB, cc = (dch % C::IB) >> 4;
#pragma unroll
                  for (int kp = 0; kp < 2; ++kp) {  // keys 32 kp .. 32 kp + 31
                    uint32_t m4[4];
                    ldsm_b8_trans_x2(m4, rawV + dh * (C::IB << lb) + grp_off[kp] + ((cc ^ swz[kp]) << 4));
                    // m4[0]: keys 4(l%4) + 0..3 of d = l/4, m4[1]: of d + 8;
                    // m4[2], m4[3]: the same for the keys 16 later
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      v[2 * e] = fp8x2_to_f16x2<E5>(m4[e]);
                      v[2 * e + 1] = fp8x2_to_f16x2<E5>(m4[e] >> 16);
                    }
                    tc::tmem_st_16x256b_x2(tbase + ((uint32_t)(32 * dq + 16 * dc) << 16) + C::VCOL +
                                               vs * C::VTC + mh * 32 + kp * 16,
                                           v);
                  }
                }
              }
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(bar(kVReady + vs));
            tc::mbar_arrive(bar(kVEmpty + st));
          }
        }
      };
      if (p.e5m2)
        decode_v(std::true_type{});
      else
        decode_v(std::false_type{});
    } else {
      // =============================== softmax (thread = key, NC rows)
      const int q = warp & 3, cg = warp >> 2;
      const int col0 = cg * C::NC;
      const uint32_t lane_off = (uint32_t)(32 * q) << 16;
      constexpr int nsm = 32 * C::NSW;
      float *m_s = reinterpret_cast<float *>(gSm + C::S_M);        // [2][64] reference (log2 units)
      float *base_s = reinterpret_cast<float *>(gSm + C::S_BASE);  // [2][64] m, or 0 while m = -inf
      float *thr_s = reinterpret_cast<float *>(gSm + C::S_THR);    // [2][64] m + tau
      int *pos_s = reinterpret_cast<int *>(gSm + C::S_POS);        // last visible key per row
      // output offset per row; two copies, for this segment and the next
      long long *rows_s = reinterpret_cast<long long *>(gSm + C::S_ROW);
      float *red = reinterpret_cast<float *>(gSm + C::S_RED);
      float *linv_s = reinterpret_cast<float *>(gSm + C::S_LINV);  // row sums of the segment
      volatile int *mb_s = reinterpret_cast<volatile int *>(gSm + C::S_SCAL + 32);  // per column group
      const float4 *box_s = reinterpret_cast<const float4 *>(gSm + C::S_BOX);
      const uint32_t *mask_s = reinterpret_cast<const uint32_t *>(gSm + C::S_MASK);
      // queries of segment s into shared memory (rows past the unit's: zeros)
      auto load_q = [&](int s) {
        const Segment &sg = seg_s[s];
        const int bq = LISTED ? sg.b / p.Hkv : sg.b, h = sg.h_rg & 0xFFFF, row0 = (sg.h_rg >> 16) * N;
        const __half *qb = static_cast<const __half *>(p.q) + (int64_t)bq * p.q_sb;
        constexpr int QCH = D / 8;  // 16-byte chunks per query row
#pragma unroll
        for (int c = tid; c < N * QCH; c += nsm) {
          const int r = c / QCH, cc = c - r * QCH;
          const int rr = row0 + r, i = rr / p.G, g = rr - i * p.G;
          const bool live = i < sg.ql;
          const __half *src = qb + (live ? (int64_t)i * p.q_si + (int64_t)(h * p.G + g) * p.q_sh + cc * 8 : 0);
          cp_async16(sQ + (cc >> 3) * (N * 128) + sw128(r * 128 + (cc & 7) * 16), src, live);
        }
      };
      auto q_ready = [&]() {  // this thread's part of the queries is in place
        tc::cp_async_wait_all();
        tc::fence_proxy_async_smem();  // Q is read by the tensor core
        tc::mbar_arrive(bar(kQReady));
      };
      bool alive = true;
      if (nseg > 0) {
        load_q(0);
        q_ready();
      }
      for (int s = 0; s < nseg; ++s) {
        const int k0 = seg_s[s].k0, k1 = seg_s[s].k1, ql = seg_s[s].ql;
        const int ntiles = (k1 - k0 + 127) >> 7;
        const int min_pos = seg_s[s].L - ql;  // every live row sees keys up to here
        const int row0 = (seg_s[s].h_rg >> 16) * N, h = seg_s[s].h_rg & 0xFFFF;
        const int slot = seg_s[s].slot;
        // ---- row state (the previous segment's was last read before the
        // second barrier of its end, but for the output offsets)
        long long *row_s = rows_s + (s & 1) * 64;
        if (tid < N) {
          const int rr = row0 + tid, i = rr / p.G;
          const int bq = LISTED ? seg_s[s].b / p.Hkv : seg_s[s].b;
          const bool live = i < ql;
          pos_s[tid] = live ? min_pos + i : -1;
          row_s[tid] = live ? (int64_t)bq * p.o_sb + (int64_t)i * p.o_si +
                                  (int64_t)(h * p.G + rr - i * p.G) * p.o_sh
                            : -1;
          m_s[tid] = -kInf;
          base_s[tid] = 0.f;
          thr_s[tid] = -kInf;
        }
        tc::named_bar(1, nsm);
        int mb = 0;  // which copy of the row references is current
        const uint32_t all_queries = (1u << ql) - 1u;
        float lpart[C::NC];
#pragma unroll
        for (int c = 0; c < C::NC; ++c) lpart[c] = 0.f;
        for (int jl = 0; jl < ntiles; ++jl, ++count) {
          const int j = count, buf = j & 1;
          // ---- the key's scales, position and mask
          const int sl = count2 % C::NSG;
          if ((jl & 3) == 0)
            alive = alive &&
                    tc::mbar_wait_brief(bar(kScFull + sl), (count2 / C::NSG) & 1, abort_f, LIM);
          const int x = sl * 32 + (jl & 3) * 8 + 2 * q + (lane >> 4);
          const float4 ks = box_s[x];  // alpha, log2 s_V, 1 / s_V, first token
          const int key = k0 + 128 * jl + 32 * q + lane;
          const int pos = LISTED ? __float_as_int(ks.w) + (lane & 15) : key;
          const uint32_t mask = LISTED ? mask_s[x] : 0u;
          if ((jl & 3) == 3 || jl == ntiles - 1) {
            tc::mbar_arrive(bar(kScEmpty + sl));
            ++count2;
          }
          // ---- scores
          float t[C::NC];
          alive = alive && tc::mbar_wait_brief(bar(kSFull + buf), (j >> 1) & 1, abort_f, LIM);
          if (alive) {
            tc::tc_fence_after();
#pragma unroll
            for (int c8 = 0; c8 < C::NC / 8; ++c8) {
              uint32_t r[8];
              tc::tmem_ld8(tbase + lane_off + C::SCOL + buf * C::SC + col0 + c8 * 8, r);
#pragma unroll
              for (int e = 0; e < 8; ++e) t[c8 * 8 + e] = __uint_as_float(r[e]);
            }
            tc::tmem_wait_ld();
            tc::tc_fence_before();
          } else {
#pragma unroll
            for (int c = 0; c < C::NC; ++c) t[c] = 0.f;
          }
          tc::mbar_arrive(bar(kSFree + buf));
          // the segment's score products are done: the queries may be replaced
          if (jl == ntiles - 1 && s + 1 < nseg && alive) load_q(s + 1);

          const float *thr = thr_s + mb * 64 + col0;
          bool exceed = false;
          if (key < k1 && pos <= min_pos && (!LISTED || (mask & all_queries) == all_queries)) {
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
              t[c] = fmaf(t[c], ks.x, ks.y);
              exceed |= t[c] > thr[c];
            }
          } else {
            const bool kvalid = key < k1;
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
              const int ps = pos_s[col0 + c];  // of query ps - min_pos (-1: no query)
              bool see = kvalid && pos <= ps;
              if constexpr (LISTED) see = see && ((mask >> ((ps - min_pos) & 31)) & 1u);
              t[c] = see ? fmaf(t[c], ks.x, ks.y) : -kInf;
              exceed |= t[c] > thr[c];
            }
          }
          // did any score of the tile exceed its row's threshold (the four warps
          // of the column group; the other group's rows are its own affair)
          if (tc::named_bar_or(2 + cg, 128, exceed)) {
            // maxima over the tile's 128 keys; a row is raised if its own passes
            // its threshold
            float mine = -kInf;
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
              const float mx = warp_max(t[c]);
              if (lane == c) mine = mx;
            }
            if (lane < C::NC) red[warp * 32 + lane] = mine;
            tc::named_bar(2 + cg, 128);
            if (q == 0 && lane < C::NC) {  // one warp per column group combines the quadrants
              float mt = red[(cg * 4) * 32 + lane];
#pragma unroll
              for (int qq = 1; qq < 4; ++qq) mt = fmaxf(mt, red[(cg * 4 + qq) * 32 + lane]);
              const float mn = mt > thr[lane] ? mt : m_s[mb * 64 + col0 + lane];
              const int o = (mb ^ 1) * 64 + col0 + lane;
              m_s[o] = mn;
              base_s[o] = mn == -kInf ? 0.f : mn;
              thr_s[o] = mn + kTau;
            }
            tc::named_bar(2 + cg, 128);
            const float *mo = m_s + mb * 64 + col0, *mn = m_s + (mb ^ 1) * 64 + col0;
            if (jl > 0) {
              // factors 2^(m_old - m_new) for the running sums ...
#pragma unroll
              for (int c = 0; c < C::NC; ++c)
                lpart[c] *= mn[c] == mo[c] ? 1.f : fast_exp2(mo[c] - mn[c]);
              // ... and for the O^T columns, once P.V of the previous tile is done
              alive = alive && tc::mbar_wait_brief(bar(kPvDone + (j - 1) % C::NPT),
                                             ((j - 1) / C::NPT) & 1, abort_f, LIM);
              if (alive) {
                tc::tc_fence_after();
#pragma unroll 1
                for (int c8 = 0; c8 < C::NC / 8; ++c8) {
                  float f[8];
                  bool change = false;  // the same for the whole warp
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float a = mo[c8 * 8 + e], b2 = mn[c8 * 8 + e];
                    change |= a != b2;
                    f[e] = a == b2 ? 1.f : fast_exp2(a - b2);
                  }
                  if (change) {
#pragma unroll
                    for (int mh = 0; mh < C::MH; ++mh) {
                      const uint32_t ta = tbase + lane_off + C::OCOL + mh * C::SC + col0 + c8 * 8;
                      uint32_t r[8];
                      tc::tmem_ld8(ta, r);
                      tc::tmem_wait_ld();
#pragma unroll
                      for (int e = 0; e < 8; ++e)
                        r[e] = __float_as_uint(__uint_as_float(r[e]) * f[e]);
                      tc::tmem_st8(ta, r);
                    }
                  }
                }
                tc::tmem_wait_st();
              }
            }
            mb ^= 1;
          }
          // the P buffer is free once P.V of the tile that last used it is done
          const int pb = j % C::NPT;
          uint8_t *gPj = gP + pb * C::PB;
          if (j >= C::NPT)
            alive = alive && tc::mbar_wait_brief(bar(kPvDone + pb), (j / C::NPT - 1) & 1, abort_f, LIM);
          // w = 2^(t - m): FP16 into P^T (MN-major, 128-byte swizzle); the row
          // sums add w / s_V
          const float *bs = base_s + mb * 64 + col0;
          const int kt = 32 * q + lane;  // key within the tile
#pragma unroll
          for (int c8 = 0; c8 < C::NC / 8; ++c8) {
            uint32_t hw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = c8 * 8 + 2 * e;
              const float e0 = fast_exp2(t[c] - bs[c]);
              const float e1 = fast_exp2(t[c + 1] - bs[c + 1]);
              lpart[c] = fmaf(e0, ks.z, lpart[c]);
              lpart[c + 1] = fmaf(e1, ks.z, lpart[c + 1]);
              hw[e] = pack_half2(e0, e1);
            }
            const int r0 = col0 + c8 * 8;
            const uint32_t po = sw128((uint32_t)(kt * 128 + (r0 >> 3) * 16));
            *reinterpret_cast<uint4 *>(gPj + po) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          }
          tc::fence_proxy_async_smem();
          tc::tc_fence_before();
          tc::mbar_arrive(bar(kPReady + pb));
        }
        if (s + 1 < nseg) q_ready();

        // ---- the segment's end: row sums, then the rows out of TMEM
#pragma unroll
        for (int c8 = 0; c8 < C::NC; c8 += 8) {  // eight rows at a time, halved at each exchange
          float v8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v8[e] = lpart[c8 + e];
#pragma unroll
          for (int o = 16, k = 4; k > 0; o >>= 1, k >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int e = 0; e < k; ++e)
              v8[e] = (up ? v8[e + k] : v8[e]) +
                      __shfl_xor_sync(0xffffffffu, up ? v8[e] : v8[e + k], o);
          }
          float sm = v8[0];
          sm += __shfl_xor_sync(0xffffffffu, sm, 2);
          sm += __shfl_xor_sync(0xffffffffu, sm, 1);
          if ((lane & 3) == 0) red[warp * 32 + c8 + (lane >> 2)] = sm;
        }
        if (q == 0 && lane == 0) mb_s[cg] = mb;
        const int jz = count - 1;  // the segment's last tile
        alive = alive && tc::mbar_wait_brief(bar(kPvDone + jz % C::NPT), (jz / C::NPT) & 1, abort_f, LIM);
        tc::tc_fence_after();
        tc::named_bar(1, nsm);
        if (tid < N) {
          const int r = tid, g2 = r / C::NC, c = r - g2 * C::NC;
          float l = 0.f;
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) l += red[(g2 * 4 + qq) * 32 + c];
          const bool ok = *reinterpret_cast<volatile int *>(bad_s + s) == 0;
          linv_s[r] = ok ? l : -1.f;
          if (slot >= 0 && alive) {
            p.ws_ml[((int64_t)slot * N + r) * 2 + 0] = m_s[mb_s[g2] * 64 + r];
            p.ws_ml[((int64_t)slot * N + r) * 2 + 1] = ok ? l : -1.f;
          }
        }
        tc::named_bar(1, nsm);
        if (alive) {
          constexpr int NG = C::MH * (N / 8);  // 8-column groups per lane quadrant, two warps each
#pragma unroll 1
          for (int g = cg; g < NG; g += 2) {
            const int mh = g / (N / 8), c8 = g % (N / 8);
            uint32_t r[8];
            tc::tmem_ld8(tbase + lane_off + C::OCOL + mh * C::SC + c8 * 8, r);
            tc::tmem_wait_ld();
            const int d = 128 * mh + 32 * q + lane;
            if (d < D) {
              if (slot >= 0) {
                float *o = p.ws_o + ((int64_t)slot * N + c8 * 8) * D + d;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[(int64_t)e * D] = __uint_as_float(r[e]);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int row = c8 * 8 + e;
                  const long long at = row_s[row];
                  const float l = linv_s[row];
                  if (at >= 0)
                    static_cast<__half *>(p.out)[at + d] =
                        __float2half_rn(l <= 0.f ? 0.f : __fdividef(__uint_as_float(r[e]), l));  // (NaN if l is)
                }
              }
            }
          }
          tc::tc_fence_before();
        }
      }
    }

    // ---- end of this batch of segments
    __syncthreads();
    const bool aborted = *abort_f != 0;
    for (int s = 0; s < nseg; ++s) {
      if (aborted) {  // mark every segment of the CTA invalid
        const Segment sg = seg_s[s];
        if (sg.slot >= 0) {
          if (tid < N) p.ws_ml[((int64_t)sg.slot * N + tid) * 2 + 1] = -1.f;
        } else {
          const int bq = LISTED ? sg.b / p.Hkv : sg.b, h = sg.h_rg & 0xFFFF;
          for (int x = tid; x < N * D; x += C::NTHREADS) {
            const int rr = (sg.h_rg >> 16) * N + x / D, i = rr / p.G;
            if (i < sg.ql)
              static_cast<__half *>(p.out)[(int64_t)bq * p.o_sb + (int64_t)i * p.o_si +
                                           (int64_t)(h * p.G + rr - i * p.G) * p.o_sh + x % D] =
                  __ushort_as_half(0);
          }
        }
      }
      if (!LISTED && tid == 0 && bad_s[s] != 0)  // (the list's writer has reported its own)
        atomicOr(p.status, ((bad_s[s] & 1) ? VAE4_STATUS_BAD_BLOCK : 0u) |
                               ((bad_s[s] & 2) ? VAE4_STATUS_BAD_SCALE : 0u));
    }
    if (aborted && tid == 0 && nseg > 0) atomicOr(p.status, VAE4_STATUS_TIMEOUT);
    if (!more) break;
    first = false;
    __syncthreads();
  }

  // ---- wind-down: drain copies and MMAs, free TMEM.  A run without an abort
  // has waited for every load and MMA it issued; after an abort some may
  // still be in flight.
  const bool drain = *abort_f != 0;
  if (drain && producer && lane == 0 && !p.cpasync) {
    const int fullb = warp == kWVProd ? kVFull : kKFull;
    const int nslot = warp == kWVProd ? C::NVR : C::NKR;
    volatile int no_abort = 0;
    for (int s = 0; s < nslot && s < count; ++s) {
      const int uses = (count - 1 - s) / nslot + 1;  // half-tiles s, s + nslot, ...
      tc::mbar_wait_brief(bar(fullb + s), (uses - 1) & 1, &no_abort, p.drain_limit);
    }
  }
  tc::cp_async_wait_all();
  if (drain && (warp == kWQk || warp == kWPv) && mma_issued && tc::elect_one()) {
    const uint32_t db = bar(warp == kWQk ? kDrainQk : kDrainPv);
    tc::mma_commit(db);
    volatile int no_abort = 0;
    tc::mbar_wait_brief(db, 0, &no_abort, p.drain_limit);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kWQk) tc::tmem_dealloc(tbase, 512);
}

// ---------------------------------------------------------------------------
// Host side: launch of one instantiation.
template <int D, int N, bool LISTED>
cudaError_t launch_dn(const SegParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                      cudaStream_t stream) {
  using C = Cfg<D, N>;
  // the shared-memory opt-in is a function attribute of the device's
  // context: set it once per context
  constexpr int kDevs = 64;
  static std::atomic<unsigned long long> configured[kDevs] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const unsigned long long ctx = current_context_id();
  if (dev < 0 || dev >= kDevs || ctx == 0 ||
      configured[dev].load(std::memory_order_acquire) != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(
        seg_kernel<D, N, LISTED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kDevs)
      configured[dev].store(current_context_id(), std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(C::NTHREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, seg_kernel<D, N, LISTED>, p, map_k, map_v);
}

template <int D, bool LISTED>
cudaError_t launch_d(const SegParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                     cudaStream_t stream) {
  switch (p.N) {
    case 16: return launch_dn<D, 16, LISTED>(p, map_k, map_v, stream);
    case 32: return launch_dn<D, 32, LISTED>(p, map_k, map_v, stream);
    case 48: return launch_dn<D, 48, LISTED>(p, map_k, map_v, stream);
    case 64: return launch_dn<D, 64, LISTED>(p, map_k, map_v, stream);
    default: return cudaErrorInvalidValue;
  }
}

// one head dim each, compiled in a translation unit of its own
cudaError_t launch_64(const SegParams &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s);
cudaError_t launch_128(const SegParams &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s);
cudaError_t launch_256(const SegParams &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s);

}  // namespace seg
}  // namespace vae4
