// C-ABI entry point of chunk attention.  See include/verify_attn_e4m3.h for the contract.
#include "api_prepare.h"
#include "chunk_params.h"

using namespace vae4;

namespace {

struct ChunkPlan {
  int ctas;
  int64_t split_off, ml_off, o_off, total;
};

// workspace: status | split units [ctas] | (max, sum) [2 ctas][R][2] | unnormalised
// O [2 ctas][R][D]
int plan_chunk(int64_t B, int64_t Hkv, int64_t G, int64_t Qmax, int64_t D, int64_t cap, int sms,
               ChunkPlan *o) {
  const int64_t R = chunk_rows((int)D);
  // a group of CTAs for every tile at most (each unit counts one more for its set-up)
  const int64_t units = B * Hkv * ((Qmax * G + R - 1) / R);
  const int64_t tiles = units * ((cap + 127) / 128 + 1);
  // The device counts the batch's work in G-ths of a key, and divides a unit's by products
  // with its tiles: both have to stay inside 63 bits.
  if ((double)G * cap * (cap / 128 + 1) >= 0x1p62 || (double)units * G * (cap + 1024) >= 0x1p62)
    return VAE4_ERR_SHAPE;
  o->ctas = (int)std::min<int64_t>(std::max(1, std::min(sms, kMaxChunkCtas) / chunk_group((int)D)), tiles);
  o->split_off = kStatusBytes;
  o->ml_off = align_up(o->split_off + o->ctas * (int64_t)sizeof(ChunkSplit), 256);
  o->o_off = align_up(o->ml_off + 2ll * o->ctas * R * 2 * 4, 256);
  o->total = o->o_off + 2ll * o->ctas * R * D * 4;
  return VAE4_OK;
}

int check_sizes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Qmax, int64_t D) {
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (Hq < 1 || Hkv < 1 || Hkv > kMaxBlockedHeads || Qmax < 1 || Qmax > kMaxChunk || B < 0 ||
      B > 65535 || Hq > INT32_MAX / 2)
    return VAE4_ERR_SHAPE;
  if (Hq % Hkv != 0) return VAE4_ERR_GQA;
  // rows of a KV head, and of a sequence, in 32 bits on the device
  if (Qmax * (Hq / Hkv) >= (1ll << 30) || Qmax * Hq >= (1ll << 31)) return VAE4_ERR_SHAPE;
  return VAE4_OK;
}

}  // namespace

extern "C" {

int64_t verify_attn_e4m3_chunk_workspace_bytes(int B, int Hq, int Hkv, int Qmax, int D, int max_seq_len,
                                               int num_sms) {
  if (B < 1 || max_seq_len < 1 || max_seq_len > INT32_MAX / 2 || num_sms < 0) return VAE4_ERR_SHAPE;
  int rc = check_sizes(B, Hq, Hkv, Qmax, D);
  if (rc) return rc;
  int sms = num_sms;
  if (sms == 0) {
    rc = device_sms(&sms);
    if (rc) return rc;
  }
  ChunkPlan plan;
  rc = plan_chunk(B, Hkv, Hq / Hkv, Qmax, D, max_seq_len, sms, &plan);
  return rc ? rc : plan.total;
}

int verify_attn_e4m3_chunk(const vae4_tensor *q, const vae4_tensor *k_cache, const vae4_tensor *v_cache,
                           const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                           const vae4_tensor *scales, const vae4_tensor *out,
                           const vae4_tensor *workspace, vae4_stream stream, const vae4_options *opt) {
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !scales || !out || !workspace)
    return VAE4_ERR_NULL;
  vae4_options o;
  memset(&o, 0, sizeof(o));
  if (opt) o = *opt;
  if ((o.flags & ~(VAE4_FLAG_WARP_MMA | VAE4_FLAG_KV_E5M2 | VAE4_FLAG_TEST_SHORT_WAITS)) != 0)
    return VAE4_ERR_OPTIONS;
  if (o.hilo_pv != 0 && o.hilo_pv != 1) return VAE4_ERR_OPTIONS;
  if ((o.flags & VAE4_FLAG_WARP_MMA) || o.hilo_pv) return VAE4_ERR_UNSUPPORTED;
  if (!(o.softmax_scale >= 0.f)) return VAE4_ERR_OPTIONS;
  if (o.partition_tokens != 0) return VAE4_ERR_PARTITION;
  for (const vae4_tensor *t : {q, out}) {
    if ((t->dtype != VAE4_F16 && t->dtype != VAE4_BF16) || t->dtype != q->dtype) return VAE4_ERR_DTYPE;
    if (t->ndim != 4) return VAE4_ERR_SHAPE;
    for (int k = 0; k < 4; ++k)
      if (t->shape[k] != q->shape[k] || t->shape[k] < 0) return VAE4_ERR_SHAPE;
    if (t->stride[3] != 1) return VAE4_ERR_STRIDE;
    for (int k = 0; k < 3; ++k)
      if (t->stride[k] % 8 != 0 || t->stride[k] < 0 || t->stride[k] >= ((int64_t)1 << 40))
        return VAE4_ERR_STRIDE;
    if (!al16(t->data)) return VAE4_ERR_MISALIGNED;
  }
  const int64_t B = q->shape[0], Qmax = q->shape[1], Hq = q->shape[2], D = q->shape[3];
  if (overlaps(out, 3, D)) return VAE4_ERR_STRIDE;
  KvSrc src;
  int rc = check_kv(k_cache, v_cache, D, &src);
  if (rc) return rc;
  const int64_t Hkv = src.Hkv, page = src.page;
  rc = check_sizes(B, Hq, Hkv, Qmax, D);
  if (rc) return rc;
  rc = check_table(block_table, B);
  if (rc) return rc;
  int has_qlen = 0;
  rc = check_seq(seq_lens, B, &has_qlen);
  if (rc) return rc;
  const bool per_head = scales->ndim == 2;
  if (per_head) {  // F32 [Hkv][2]
    if (scales->dtype != VAE4_F32) return VAE4_ERR_DTYPE;
    if (scales->shape[0] != Hkv || scales->shape[1] != 2) return VAE4_ERR_SHAPE;
    if (scales->stride[1] != 1 || scales->stride[0] < 0 || scales->stride[0] >= ((int64_t)1 << 40))
      return VAE4_ERR_STRIDE;
    if ((reinterpret_cast<uintptr_t>(scales->data) & 3u) != 0) return VAE4_ERR_MISALIGNED;
  } else {
    rc = check_block_scales(scales, src.n_pages, Hkv, page);
    if (rc) return rc;
  }
  if (workspace->dtype != VAE4_U8) return VAE4_ERR_DTYPE;
  if (workspace->ndim != 1 || workspace->stride[0] != 1) return VAE4_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(workspace->data) & 255u) != 0) return VAE4_ERR_WORKSPACE;
  const int64_t table_cap = block_table->shape[1] * page;
  const int64_t cap = o.max_seq_len > 0 ? o.max_seq_len : table_cap;
  if (o.max_seq_len < 0 || o.num_sms < 0 || cap > table_cap || cap > INT32_MAX / 2) return VAE4_ERR_SHAPE;
  if (B == 0) return VAE4_OK;
  int sms = o.num_sms;
  if (sms == 0) {
    rc = device_sms(&sms);
    if (rc) return rc;
  }
  ChunkPlan plan;
  rc = plan_chunk(B, Hkv, Hq / Hkv, Qmax, D, cap, sms, &plan);
  if (rc) return rc;
  if (workspace->shape[0] < plan.total) return VAE4_ERR_WORKSPACE;
  if (!q->data || !src.kb || !src.vb || !block_table->data || !seq_lens->data || !scales->data ||
      !out->data || !workspace->data)
    return VAE4_ERR_NULL;
  uint8_t *ws = static_cast<uint8_t *>(workspace->data);
  ChunkParams p;
  memset(&p, 0, sizeof(p));
  p.q = q->data;
  p.q_sb = q->stride[0];
  p.q_si = q->stride[1];
  p.q_sh = q->stride[2];
  p.out = out->data;
  p.o_sb = out->stride[0];
  p.o_si = out->stride[1];
  p.o_sh = out->stride[2];
  p.k_base = src.kb;
  p.v_base = src.vb;
  p.k_ps = src.k_ps;
  p.k_ts = src.k_ts;
  p.k_hs = src.k_hs;
  p.v_ps = src.v_ps;
  p.v_ts = src.v_ts;
  p.v_hs = src.v_hs;
  p.n_pages = src.n_pages;
  p.wide = al16(src.kb) && al16(src.vb);
  for (int64_t s : {src.k_ps, src.k_ts, src.k_hs, src.v_ps, src.v_ts, src.v_hs})
    if (s % 16 != 0) p.wide = 0;
  p.bt = static_cast<const int32_t *>(block_table->data);
  p.bt_sb = block_table->stride[0];
  p.seq = static_cast<const int32_t *>(seq_lens->data);
  p.seq_sb = (int32_t)seq_lens->stride[0];
  p.seq_has_qlen = has_qlen;
  p.capacity = (int32_t)cap;
  p.scales = static_cast<const float *>(scales->data);
  const int64_t blk = per_head ? page : page / scales->shape[3];
  p.s_page = per_head ? 0 : scales->stride[0];
  p.s_kv = scales->stride[1];
  p.s_head = per_head ? scales->stride[0] : scales->stride[2];
  p.page_blocks = (int32_t)(page / blk);
  p.page_m = reciprocal16((int)page);
  p.blk_m = reciprocal16((int)blk);
  p.split = reinterpret_cast<ChunkSplit *>(ws + plan.split_off);
  p.ws_ml = reinterpret_cast<float *>(ws + plan.ml_off);
  p.ws_o = reinterpret_cast<float *>(ws + plan.o_off);
  p.status = reinterpret_cast<uint32_t *>(ws);
  p.B = (int32_t)B;
  p.Qmax = (int32_t)Qmax;
  p.Hkv = (int32_t)Hkv;
  p.G = (int32_t)(Hq / Hkv);
  p.D = (int32_t)D;
  p.page = (int32_t)page;
  p.bf16 = q->dtype == VAE4_BF16;
  p.e5m2 = (o.flags & VAE4_FLAG_KV_E5M2) != 0;
  p.ctas = plan.ctas;
  // (the product of two FP32 numbers is exact in 64 bits, and may be too small or too large
  // for 32)
  const double alpha = (double)(o.softmax_scale > 0.f ? o.softmax_scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  int e = 1;
  p.alpha = (float)(2 * (std::isfinite(alpha) ? std::frexp(alpha, &e) : alpha));
  p.alpha_e = e - 1;
  p.wait_limit = (o.flags & VAE4_FLAG_TEST_SHORT_WAITS) ? kShortWaitCycles : kWaitLimitCycles;
  p.drain_limit = kWaitLimitCycles;
  if (launch_chunk(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  if (launch_chunk_combine(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

}  // extern "C"
