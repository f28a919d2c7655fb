// C-ABI entry points of the block-scaled cache: the writer, attention with
// block scales, the block scores, the choice of blocks and sparse attention.
// See include/verify_attn_e4m3.h for the contract of every function.
#include "api_prepare.h"

using namespace vae4;

namespace {

int run_attention(const Prepared &pr, cudaStream_t st) {
  if (pr.sparse && launch_block_list(pr.lp, st) != cudaSuccess) return VAE4_ERR_CUDA;
  if (launch_seg(pr.gp, st) != cudaSuccess) return VAE4_ERR_CUDA;
  if (launch_seg_combine(pr.gp, st) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

// bytes of workspace of attention over a block-scaled cache (blocks = 0: dense)
int64_t attention_bytes(int B, int Hq, int Hkv, int Qmax, int D, int max_seq_len, int block_tokens,
                        int blocks, int num_sms) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Qmax < 1 || Qmax > kMaxQmax || max_seq_len < 1 ||
      max_seq_len > INT32_MAX / 2)
    return VAE4_ERR_SHAPE;
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return VAE4_ERR_GQA;
  const int64_t rows = (int64_t)Qmax * (Hq / Hkv);
  if (align_up(rows, 16) > kMaxRowsPad) return VAE4_ERR_UNSUPPORTED;
  int sms = num_sms;
  if (sms < 0) return VAE4_ERR_SHAPE;
  if (sms == 0) {
    const int rc = device_sms(&sms);
    if (rc) return rc;
  }
  BlockPlan plan;
  const int rc =
      plan_blocks(B, Hkv, Qmax, rows, D, max_seq_len, block_tokens, blocks, sms, &plan);
  return rc ? rc : plan.total;
}

}  // namespace

extern "C" {

int verify_attn_e4m3_append(const vae4_tensor *k_new, const vae4_tensor *v_new,
                            const vae4_tensor *k_cache, const vae4_tensor *v_cache,
                            const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                            const vae4_tensor *block_scales, const vae4_tensor *k_bounds,
                            uint32_t *dev_status, int32_t flags, vae4_stream stream) {
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_lens || !block_scales)
    return VAE4_ERR_NULL;
  if ((flags & ~VAE4_FLAG_KV_E5M2) != 0) return VAE4_ERR_OPTIONS;
  for (const vae4_tensor *t : {k_new, v_new}) {
    if ((t->dtype != VAE4_F16 && t->dtype != VAE4_BF16) || t->dtype != k_new->dtype)
      return VAE4_ERR_DTYPE;
    if (t->ndim != 4) return VAE4_ERR_SHAPE;
    for (int k = 0; k < 4; ++k)
      if (t->shape[k] != k_new->shape[k] || t->shape[k] < 0) return VAE4_ERR_SHAPE;
    if (t->stride[3] != 1) return VAE4_ERR_STRIDE;
    for (int k = 0; k < 3; ++k)
      if (t->stride[k] % 8 != 0 || t->stride[k] < 0 || t->stride[k] >= ((int64_t)1 << 40))
        return VAE4_ERR_STRIDE;
    if (!al16(t->data)) return VAE4_ERR_MISALIGNED;
  }
  const int64_t B = k_new->shape[0], Q = k_new->shape[1], Hkv = k_new->shape[2], D = k_new->shape[3];
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (Q < 1 || Q > INT32_MAX / 2 || Hkv < 1 || Hkv > 32767 || B > 65535) return VAE4_ERR_SHAPE;
  KvSrc src;
  int rc = check_kv(k_cache, v_cache, D, &src);
  if (rc) return rc;
  if (src.Hkv != Hkv) return VAE4_ERR_SHAPE;
  if (overlaps(k_cache, 3, D) || overlaps(v_cache, 3, D)) return VAE4_ERR_STRIDE;
  rc = check_table(block_table, B);
  if (rc) return rc;
  int has_qlen = 0;
  rc = check_seq(seq_lens, B, &has_qlen);
  if (rc) return rc;
  rc = check_block_scales(block_scales, src.n_pages, Hkv, src.page);
  if (rc) return rc;
  if (overlaps(block_scales, 3, block_scales->shape[3])) return VAE4_ERR_STRIDE;
  const int64_t nb = block_scales->shape[3], blk = src.page / nb;
  if (k_bounds) {
    rc = check_bounds(k_bounds, src.n_pages, Hkv, nb, D);
    if (rc) return rc;
    if (overlaps(k_bounds, 4, D)) return VAE4_ERR_STRIDE;
  }
  if (block_table->shape[1] * src.page > INT32_MAX / 2) return VAE4_ERR_SHAPE;
  if (B == 0) return VAE4_OK;
  if (!k_new->data || !v_new->data || !src.kb || !src.vb || !block_table->data || !seq_lens->data ||
      !block_scales->data || (k_bounds && !k_bounds->data))
    return VAE4_ERR_NULL;
  AppendParams p;
  memset(&p, 0, sizeof(p));
  const vae4_tensor *x[2] = {k_new, v_new};
  const vae4_tensor *c[2] = {k_cache, v_cache};
  for (int w = 0; w < 2; ++w) {
    p.x[w] = x[w]->data;
    p.x_sb[w] = x[w]->stride[0];
    p.x_si[w] = x[w]->stride[1];
    p.x_sh[w] = x[w]->stride[2];
    p.c[w] = static_cast<uint8_t *>(c[w]->data);
    p.c_ps[w] = c[w]->stride[0];
    p.c_ts[w] = c[w]->stride[1];
    p.c_hs[w] = c[w]->stride[2];
  }
  p.n_pages = src.n_pages;
  p.bt = static_cast<const int32_t *>(block_table->data);
  p.bt_sb = block_table->stride[0];
  p.max_pages = (int32_t)block_table->shape[1];
  p.seq = static_cast<const int32_t *>(seq_lens->data);
  p.seq_sb = (int32_t)seq_lens->stride[0];
  p.seq_has_qlen = has_qlen;
  p.scales = static_cast<float *>(block_scales->data);
  p.s_page = block_scales->stride[0];
  p.s_kv = block_scales->stride[1];
  p.s_head = block_scales->stride[2];
  if (k_bounds) {
    p.bounds = static_cast<uint8_t *>(k_bounds->data);
    p.b_page = k_bounds->stride[0];
    p.b_head = k_bounds->stride[1];
    p.b_blk = k_bounds->stride[2];
    p.b_mm = k_bounds->stride[3];
  }
  p.status = dev_status;
  p.B = (int32_t)B;
  p.Qmax = (int32_t)Q;
  p.Hkv = (int32_t)Hkv;
  p.D = (int32_t)D;
  p.page = (int32_t)src.page;
  p.blk = (int32_t)blk;
  p.touched = (int32_t)((Q + blk - 2) / blk + 1);
  p.nb = (int32_t)nb;
  p.page_m = reciprocal16(p.page);
  p.blk_m = reciprocal16(p.blk);
  if (launch_append(p, k_new->dtype == VAE4_BF16, (flags & VAE4_FLAG_KV_E5M2) != 0, cu(stream)) !=
      cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_block_scaled(const vae4_tensor *q, const vae4_tensor *k_cache,
                                  const vae4_tensor *v_cache, const vae4_tensor *block_table,
                                  const vae4_tensor *seq_lens, const vae4_tensor *block_scales,
                                  const vae4_tensor *out, const vae4_tensor *workspace,
                                  vae4_stream stream, const vae4_options *opt) {
  Prepared pr;
  const int rc = prepare(q, nullptr, k_cache, v_cache, block_table, seq_lens, block_scales, out,
                         workspace, opt, &pr, true);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  return run_attention(pr, cu(stream));
}

int verify_attn_e4m3_sparse(const vae4_tensor *q, const vae4_tensor *k_cache,
                            const vae4_tensor *v_cache, const vae4_tensor *block_table,
                            const vae4_tensor *seq_lens, const vae4_tensor *block_scales,
                            const vae4_tensor *block_ids, const vae4_tensor *out,
                            const vae4_tensor *workspace, vae4_stream stream,
                            const vae4_options *opt) {
  if (!block_ids) return VAE4_ERR_NULL;
  Prepared pr;
  const int rc = prepare(q, nullptr, k_cache, v_cache, block_table, seq_lens, block_scales, out,
                         workspace, opt, &pr, true, block_ids);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  return run_attention(pr, cu(stream));
}

int64_t verify_attn_e4m3_sparse_workspace_bytes(int B, int Hq, int Hkv, int Qmax, int D,
                                                int max_seq_len, int block_tokens, int blocks,
                                                int num_sms) {
  if (blocks < 1 || blocks > INT32_MAX / 32) return VAE4_ERR_SHAPE;
  if (block_tokens < 16 || block_tokens % 16 != 0 || block_tokens > 65536)
    return VAE4_ERR_UNSUPPORTED;
  return attention_bytes(B, Hq, Hkv, Qmax, D, max_seq_len, block_tokens, blocks, num_sms);
}

int64_t verify_attn_e4m3_block_scaled_workspace_bytes(int B, int Hq, int Hkv, int Qmax, int D,
                                                      int max_seq_len, int num_sms) {
  return attention_bytes(B, Hq, Hkv, Qmax, D, max_seq_len, 16, 0, num_sms);
}

int verify_attn_e4m3_block_scores(const vae4_tensor *q, const vae4_tensor *k_bounds,
                                  const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                                  const vae4_tensor *block_scales, const vae4_tensor *scores,
                                  int32_t block_tokens, float softmax_scale, uint32_t *dev_status,
                                  int32_t flags, vae4_stream stream) {
  if (!q || !k_bounds || !block_table || !seq_lens || !block_scales || !scores) return VAE4_ERR_NULL;
  if ((flags & ~VAE4_FLAG_KV_E5M2) != 0 || !(softmax_scale >= 0.f)) return VAE4_ERR_OPTIONS;
  int rc = check_qo(q);
  if (rc) return rc;
  const int64_t B = q->shape[0], Qmax = q->shape[1], Hq = q->shape[2], D = q->shape[3];
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (Qmax < 1 || Qmax > kMaxQmax || Hq < 1 || B > 65535) return VAE4_ERR_SHAPE;
  if (k_bounds->ndim != 5 || k_bounds->shape[0] < 1 || k_bounds->shape[0] > 0x7fffffff ||
      k_bounds->shape[1] < 1 || k_bounds->shape[2] < 1)
    return VAE4_ERR_SHAPE;
  const int64_t n_pages = k_bounds->shape[0], Hkv = k_bounds->shape[1], nb = k_bounds->shape[2];
  rc = check_bounds(k_bounds, n_pages, Hkv, nb, D);
  if (rc) return rc;
  if (Hkv > kMaxBlockedHeads) return VAE4_ERR_SHAPE;
  if (Hq % Hkv != 0) return VAE4_ERR_GQA;
  if (align_up(Qmax * (Hq / Hkv), 16) > kMaxRowsPad) return VAE4_ERR_UNSUPPORTED;
  if (block_tokens < 16 || block_tokens % 16 != 0 || nb * block_tokens > 65536)
    return VAE4_ERR_UNSUPPORTED;
  rc = check_table(block_table, B);
  if (rc) return rc;
  int has_qlen = 0;
  rc = check_seq(seq_lens, B, &has_qlen);
  if (rc) return rc;
  rc = check_block_scales(block_scales, n_pages, Hkv, nb * block_tokens);
  if (rc) return rc;
  if (block_scales->shape[3] != nb) return VAE4_ERR_SHAPE;
  if (block_table->shape[1] * nb * block_tokens > INT32_MAX / 2) return VAE4_ERR_SHAPE;
  if (scores->dtype != VAE4_F32) return VAE4_ERR_DTYPE;
  if (scores->ndim != 4 || scores->shape[0] != B || scores->shape[1] != Qmax ||
      scores->shape[2] != Hkv || scores->shape[3] < 1 || scores->shape[3] > INT32_MAX / 2)
    return VAE4_ERR_SHAPE;
  if (scores->stride[3] != 1) return VAE4_ERR_STRIDE;
  for (int k = 0; k < 3; ++k)
    if (scores->stride[k] < 0 || scores->stride[k] >= ((int64_t)1 << 40)) return VAE4_ERR_STRIDE;
  if (overlaps(scores, 3, scores->shape[3])) return VAE4_ERR_STRIDE;
  if ((reinterpret_cast<uintptr_t>(scores->data) & 3u) != 0) return VAE4_ERR_MISALIGNED;
  if (B == 0) return VAE4_OK;
  if (!q->data || !k_bounds->data || !block_table->data || !seq_lens->data || !block_scales->data ||
      !scores->data)
    return VAE4_ERR_NULL;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc) return rc;
  ScoreParams p;
  memset(&p, 0, sizeof(p));
  p.q = q->data;
  p.q_sb = q->stride[0];
  p.q_si = q->stride[1];
  p.q_sh = q->stride[2];
  p.bounds = static_cast<const uint8_t *>(k_bounds->data);
  p.b_page = k_bounds->stride[0];
  p.b_head = k_bounds->stride[1];
  p.b_blk = k_bounds->stride[2];
  p.b_mm = k_bounds->stride[3];
  p.scales = static_cast<const float *>(block_scales->data);
  p.s_page = block_scales->stride[0];
  p.s_kv = block_scales->stride[1];
  p.s_head = block_scales->stride[2];
  p.n_pages = n_pages;
  p.bt = static_cast<const int32_t *>(block_table->data);
  p.bt_sb = block_table->stride[0];
  p.max_pages = (int32_t)block_table->shape[1];
  p.seq = static_cast<const int32_t *>(seq_lens->data);
  p.seq_sb = (int32_t)seq_lens->stride[0];
  p.seq_has_qlen = has_qlen;
  p.scores = static_cast<float *>(scores->data);
  p.o_sb = scores->stride[0];
  p.o_si = scores->stride[1];
  p.o_sh = scores->stride[2];
  p.cols = (int32_t)scores->shape[3];
  p.status = dev_status;
  p.B = (int32_t)B;
  p.Qmax = (int32_t)Qmax;
  p.Hkv = (int32_t)Hkv;
  p.G = (int32_t)(Hq / Hkv);
  p.D = (int32_t)D;
  p.nb = (int32_t)nb;
  p.blk = block_tokens;
  p.num_sms = sms;
  p.sm_scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)D);
  if (launch_block_scores(p, (flags & VAE4_FLAG_KV_E5M2) != 0, cu(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_select_blocks(const vae4_tensor *scores, const vae4_tensor *seq_lens,
                                   const vae4_tensor *block_ids, int32_t block_tokens,
                                   int32_t sink_blocks, int32_t local_blocks, uint32_t *dev_status,
                                   vae4_stream stream) {
  if (!scores || !seq_lens || !block_ids) return VAE4_ERR_NULL;
  if (scores->dtype != VAE4_F32) return VAE4_ERR_DTYPE;
  if (scores->ndim != 4 || scores->shape[0] < 0 || scores->shape[0] > 65535 || scores->shape[1] < 1 ||
      scores->shape[2] < 1 || scores->shape[2] > 65535 || scores->shape[3] < 1 ||
      scores->shape[3] > INT32_MAX / 2 || scores->shape[1] > INT32_MAX / 2)
    return VAE4_ERR_SHAPE;
  if (scores->stride[3] != 1) return VAE4_ERR_STRIDE;
  for (int k = 0; k < 3; ++k)
    if (scores->stride[k] < 0 || scores->stride[k] >= ((int64_t)1 << 40)) return VAE4_ERR_STRIDE;
  if ((reinterpret_cast<uintptr_t>(scores->data) & 3u) != 0) return VAE4_ERR_MISALIGNED;
  const int64_t B = scores->shape[0], Qmax = scores->shape[1], Hkv = scores->shape[2];
  int rc = check_ids(block_ids, B, Qmax, Hkv);
  if (rc) return rc;
  if (overlaps(block_ids, 3, block_ids->shape[3])) return VAE4_ERR_STRIDE;
  int has_qlen = 0;
  rc = check_seq(seq_lens, B, &has_qlen);
  if (rc) return rc;
  if (block_tokens < 16 || block_tokens % 16 != 0 || block_tokens > 65536) return VAE4_ERR_UNSUPPORTED;
  const int64_t k = block_ids->shape[3];
  if (sink_blocks < 0 || local_blocks < 0 || (int64_t)sink_blocks + local_blocks > k)
    return VAE4_ERR_OPTIONS;
  if (B == 0) return VAE4_OK;
  if (!scores->data || !seq_lens->data || !block_ids->data) return VAE4_ERR_NULL;
  SelectParams p;
  memset(&p, 0, sizeof(p));
  p.scores = static_cast<const float *>(scores->data);
  p.s_sb = scores->stride[0];
  p.s_si = scores->stride[1];
  p.s_sh = scores->stride[2];
  p.cols = (int32_t)scores->shape[3];
  p.seq = static_cast<const int32_t *>(seq_lens->data);
  p.seq_sb = (int32_t)seq_lens->stride[0];
  p.seq_has_qlen = has_qlen;
  p.ids = static_cast<int32_t *>(block_ids->data);
  p.i_sb = block_ids->stride[0];
  p.i_si = block_ids->stride[1];
  p.i_sh = block_ids->stride[2];
  p.k = (int32_t)k;
  p.status = dev_status;
  p.B = (int32_t)B;
  p.Qmax = (int32_t)Qmax;
  p.Hkv = (int32_t)Hkv;
  p.blk = block_tokens;
  p.sink = sink_blocks;
  p.local = local_blocks;
  if (launch_select_blocks(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

}  // extern "C"
