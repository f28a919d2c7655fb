// Launch parameters of the block-scaled cache's kernels, shared by the host entry
// points and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vae4 {

// Block scales outside this range (or NaN) are reported as invalid: within it
// no weight or sum of the FP32 softmax state can overflow.
constexpr float kMinScale = 9.094947017729282e-13f;  // 2^-40
constexpr float kMaxScale = 1099511627776.f;         // 2^40

// One block of a sequence that sparse attention visits (one KV head).
struct alignas(16) BlockEntry {
  int32_t phys;   // physical page; -1: the page id or a scale is invalid
  int32_t box0;   // first 16-token box of the block in its page
  int32_t tok0;   // first token of the block in the sequence
  uint32_t mask;  // bit i: query i attends to the block
  float alpha;    // softmax_scale * s_K * log2(e): a score in log2 units per raw product
  float lgv;      // log2(s_V)
  float inv_sv;   // 1 / s_V
  int32_t pad;
};

// n a multiple of 16 up to 65536 -> the multiplier of div16
inline unsigned long long reciprocal16(int n) {
  const unsigned long long d = (unsigned long long)n / 16;
  return ((1ull << 38) + d - 1) / d;
}

// The stream record of one (sequence, KV head) under sparse attention.
struct alignas(16) BlockStream {
  int32_t n16;  // tokens of the listed blocks, rounded up to 16 (0: nothing to visit)
  int32_t ql;   // live queries (0 if the stream has nothing to visit)
  int32_t n;    // tokens of the listed blocks (the sequence's last block may be partial)
  int32_t L;    // the sequence's length
};

// Attention over a block-scaled cache: the split kernel and its combine.
// Strides are in elements (bytes for the caches).
struct SegParams {
  const void *q;               // fp16 [B][Qmax][Hq][D]
  int64_t q_sb, q_si, q_sh;
  void *out;                   // the same shape
  int64_t o_sb, o_si, o_sh;
  // token t of KV head h in page ph: base + ph * ps + (t % page) * ts + h * hs
  const uint8_t *k_base, *v_base;
  int64_t k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;
  int64_t n_pages;
  int32_t cpasync;             // strides are multiples of 8 but not all of 16 (8-byte copies)
  int32_t box_log2;            // log2 of the keys per tensor copy (4, 5 or 6)
  const int32_t *bt;
  int64_t bt_sb;
  int32_t max_pages;
  const int32_t *seq;          // i32 [B] or [B][2]
  int32_t seq_sb, seq_has_qlen;
  int32_t seq_capacity;        // most tokens of a sequence
  const float *scales;         // f32 [n_pages][2][Hkv][page / blk]
  int64_t s_page, s_kv, s_head;
  int32_t blk;
  // groups of units: the sequences (unit_heads = Hkv), or sparse attention's
  // streams (unit_heads = 1), with their (tokens, queries) pairs
  const int32_t *pairs;
  int32_t pair_sb, has_qlen, groups, unit_heads, capacity;
  const BlockEntry *list;      // sparse: [B * Hkv][list_cap], else null
  const BlockStream *streams;  // sparse: [B * Hkv]
  int32_t list_cap;
  float *ws_ml;                // f32 [2 ctas][N][2]
  float *ws_o;                 // f32 [2 ctas][N][D]
  int2 *tab;                   // (first CTA, parts) [B * Hkv][n_rg]
  uint32_t *status;
  int32_t B, Qmax, Hkv, G, D, page, e5m2;
  int32_t page_blocks;         // page / blk
  unsigned long long page_m, blk_m;  // reciprocals for the device's divisions (seg_tc.cuh)
  int32_t N, n_rg;             // rows per unit, row groups
  int32_t ctas;
  float sm_scale;
  long long wait_limit;        // SM cycles before a pipeline wait gives up
  long long drain_limit;       // SM cycles the wind-down waits for copies and MMAs in flight
};

// The visit-list kernel's parameters.
struct ListParams {
  const int32_t *ids;            // i32 [B][Qmax][Hkv][k]
  int64_t i_sb, i_si, i_sh;
  int32_t k;
  const int32_t *bt;
  int64_t bt_sb;
  int32_t max_pages;
  const int32_t *seq;
  int32_t seq_sb, seq_has_qlen;
  const float *scales;
  int64_t s_page, s_kv, s_head;
  int64_t n_pages;
  BlockEntry *list;
  BlockStream *streams;
  int2 *tab;                     // (first CTA, parts) [B * Hkv][n_rg], cleared here
  int32_t n_rg;
  uint32_t *status;
  int32_t B, Qmax, Hkv, page, blk, capacity, list_cap;
  float alpha;                   // softmax_scale * log2(e)
};

// The cache writer's parameters; index 0: K, 1: V.
struct AppendParams {
  const void *x[2];              // f16 or bf16 [B][Qmax][Hkv][D]
  int64_t x_sb[2], x_si[2], x_sh[2];
  uint8_t *c[2];                 // u8 [n_pages][page][Hkv][D]
  int64_t c_ps[2], c_ts[2], c_hs[2];
  int64_t n_pages;
  const int32_t *bt;
  int64_t bt_sb;
  int32_t max_pages;
  const int32_t *seq;
  int32_t seq_sb, seq_has_qlen;
  float *scales;
  int64_t s_page, s_kv, s_head;
  uint8_t *bounds;               // u8 [n_pages][Hkv][page / blk][2][D], or null
  int64_t b_page, b_head, b_blk, b_mm;
  uint32_t *status;              // may be null
  int32_t B, Qmax, Hkv, D, page, blk;
  int32_t touched;               // most blocks a sequence's new tokens can touch
  int32_t nb;                    // blocks per page
  unsigned long long page_m, blk_m;  // reciprocals of page and blk (div16)
};

// The block scores' parameters.
struct ScoreParams {
  const void *q;                 // fp16 [B][Qmax][Hq][D]
  int64_t q_sb, q_si, q_sh;
  const uint8_t *bounds;
  int64_t b_page, b_head, b_blk, b_mm;
  const float *scales;
  int64_t s_page, s_kv, s_head;
  int64_t n_pages;
  const int32_t *bt;
  int64_t bt_sb;
  int32_t max_pages;
  const int32_t *seq;
  int32_t seq_sb, seq_has_qlen;
  float *scores;                 // f32 [B][Qmax][Hkv][cols]
  int64_t o_sb, o_si, o_sh;
  int32_t cols;
  uint32_t *status;              // may be null
  int32_t B, Qmax, Hkv, G, D, nb, blk;  // nb: blocks per page
  int32_t num_sms;               // SMs the grid is sized for
  int32_t qn, parts;             // queries per CTA, CTAs that share them (set at the launch)
  float sm_scale;
};

// The block choice's parameters.
struct SelectParams {
  const float *scores;           // f32 [B][Qmax][Hkv][cols]
  int64_t s_sb, s_si, s_sh;
  int32_t cols;
  const int32_t *seq;
  int32_t seq_sb, seq_has_qlen;
  int32_t *ids;                  // i32 [B][Qmax][Hkv][k]
  int64_t i_sb, i_si, i_sh;
  int32_t k;
  uint32_t *status;              // may be null
  int32_t B, Qmax, Hkv, blk, sink, local;
};

}  // namespace vae4
