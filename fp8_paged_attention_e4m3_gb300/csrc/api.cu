// C-ABI entry points: argument validation and kernel launches (the checks and
// the plan are in api_prepare.h).  See include/verify_attn_e4m3.h for the
// contract of every function.
#include "api_prepare.h"

using namespace vae4;

namespace {

// Validation and parameters of the bridge call (kv, block table, lengths and
// scales follow the verify step's rules; outputs are dense FP16 K and V).
int prepare_bridge(const vae4_tensor *kv, const vae4_tensor *bt, const vae4_tensor *seq,
                   const vae4_tensor *sc, const vae4_tensor *ko, const vae4_tensor *vo,
                   uint32_t *status, int32_t flags, vae4::BridgeParams *bp, bool *empty) {
  if (!kv || !bt || !seq || !sc || !ko || !vo) return VAE4_ERR_NULL;
  if ((flags & ~(VAE4_FLAG_KV_E5M2 | VAE4_FLAG_BRIDGE_RAW)) != 0) return VAE4_ERR_OPTIONS;
  if (kv->dtype != VAE4_U8 || bt->dtype != VAE4_I32 || seq->dtype != VAE4_I32 ||
      sc->dtype != VAE4_F32 || ko->dtype != VAE4_F16 || vo->dtype != VAE4_F16)
    return VAE4_ERR_DTYPE;
  if (kv->ndim != 5 || kv->shape[1] != 2 || kv->shape[0] < 1 || kv->shape[2] < 1)
    return VAE4_ERR_SHAPE;
  const int64_t n_pages = kv->shape[0], Hkv = kv->shape[2], page = kv->shape[3], D = kv->shape[4];
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (page < 16 || page % 16 != 0 || page > 65536) return VAE4_ERR_UNSUPPORTED;
  if (kv->stride[4] != 1 || kv->stride[3] != D || kv->stride[2] != page * D ||
      kv->stride[1] != Hkv * page * D || kv->stride[0] != 2 * Hkv * page * D)
    return VAE4_ERR_STRIDE;
  if (!al16(kv->data)) return VAE4_ERR_MISALIGNED;
  // outputs: F16 [B][Hkv][cap][D], d contiguous, rows on 16-byte boundaries
  for (const vae4_tensor *o : {ko, vo}) {
    if (o->ndim != 4 || o->shape[1] != Hkv || o->shape[3] != D || o->shape[2] < 1)
      return VAE4_ERR_SHAPE;
    if (o->shape[0] != ko->shape[0] || o->shape[2] != ko->shape[2]) return VAE4_ERR_SHAPE;
    if (o->stride[3] != 1) return VAE4_ERR_STRIDE;
    for (int k = 0; k < 3; ++k)
      if (o->stride[k] < 0 || o->stride[k] % 8 != 0) return VAE4_ERR_STRIDE;
    if (o->stride[0] != ko->stride[0] || o->stride[1] != ko->stride[1] ||
        o->stride[2] != ko->stride[2])
      return VAE4_ERR_STRIDE;
    if (!al16(o->data)) return VAE4_ERR_MISALIGNED;
  }
  const int64_t B = ko->shape[0], cap = ko->shape[2];
  if (B > 65535 || cap > INT32_MAX / 2) return VAE4_ERR_SHAPE;
  if (bt->ndim != 2 || bt->shape[0] != B || bt->shape[1] < 1) return VAE4_ERR_SHAPE;
  if (bt->stride[1] != 1 || bt->stride[0] < 0) return VAE4_ERR_STRIDE;
  if (bt->shape[1] * page < cap) return VAE4_ERR_SHAPE;  // the table must address cap tokens
  if (seq->ndim == 1) {
    if (seq->shape[0] != B) return VAE4_ERR_SHAPE;
  } else if (seq->ndim == 2) {
    if (seq->shape[0] != B || seq->shape[1] != 2) return VAE4_ERR_SHAPE;
    if (seq->stride[1] != 1) return VAE4_ERR_STRIDE;
  } else {
    return VAE4_ERR_SHAPE;
  }
  if (seq->stride[0] < 0 || seq->stride[0] > INT32_MAX) return VAE4_ERR_STRIDE;
  if (sc->ndim != 2 || sc->shape[0] != Hkv || sc->shape[1] != 2) return VAE4_ERR_SHAPE;
  if (sc->stride[1] != 1 || sc->stride[0] < 0 || sc->stride[0] > INT32_MAX) return VAE4_ERR_STRIDE;
  *empty = B == 0;
  if (B > 0 && (!kv->data || !bt->data || !seq->data || !sc->data || !ko->data || !vo->data))
    return VAE4_ERR_NULL;
  vae4::BridgeParams &p = *bp;
  memset(&p, 0, sizeof(p));
  p.kv = static_cast<const uint8_t *>(kv->data);
  p.n_pages = n_pages;
  p.bt = static_cast<const int32_t *>(bt->data);
  p.bt_sb = bt->stride[0];
  p.seq = static_cast<const int32_t *>(seq->data);
  p.seq_sb = (int32_t)seq->stride[0];
  p.scales = static_cast<const float *>(sc->data);
  p.scale_sh = (int32_t)sc->stride[0];
  p.k_out = static_cast<uint16_t *>(ko->data);
  p.v_out = static_cast<uint16_t *>(vo->data);
  p.o_sb = ko->stride[0];
  p.o_sh = ko->stride[1];
  p.o_st = ko->stride[2];
  p.status = status;
  p.B = (int32_t)B;
  p.Hkv = (int32_t)Hkv;
  p.D = (int32_t)D;
  p.page = (int32_t)page;
  p.cap = (int32_t)cap;
  return VAE4_OK;
}

}  // namespace

extern "C" {

int verify_attn_e4m3_bridge_fp16(const vae4_tensor *kv_pages, const vae4_tensor *block_table,
                                 const vae4_tensor *seq_lens, const vae4_tensor *kv_scales,
                                 const vae4_tensor *k_out, const vae4_tensor *v_out,
                                 uint32_t *dev_status, int32_t flags, vae4_stream stream) {
  vae4::BridgeParams bp;
  bool empty = false;
  int rc = prepare_bridge(kv_pages, block_table, seq_lens, kv_scales, k_out, v_out, dev_status,
                          flags, &bp, &empty);
  if (rc) return rc;
  if (empty) return VAE4_OK;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc) return rc;
  if (vae4::launch_bridge(bp, sms, (flags & VAE4_FLAG_KV_E5M2) != 0,
                          (flags & VAE4_FLAG_BRIDGE_RAW) != 0,
                          reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_ex(const vae4_tensor *q, const vae4_tensor *kv_pages,
                        const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                        const vae4_tensor *kv_scales, const vae4_tensor *out,
                        const vae4_tensor *workspace, vae4_stream stream,
                        const vae4_options *opt) {
  Prepared pr;
  int rc = prepare(q, kv_pages, nullptr, nullptr, block_table, seq_lens, kv_scales, out,
                   workspace, opt, &pr);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_split(pr, st) != cudaSuccess) return VAE4_ERR_CUDA;
  if (vae4::launch_combine(pr.cp, st) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_kv(const vae4_tensor *q, const vae4_tensor *k_cache,
                        const vae4_tensor *v_cache, const vae4_tensor *block_table,
                        const vae4_tensor *seq_lens, const vae4_tensor *kv_scales,
                        const vae4_tensor *out, const vae4_tensor *workspace,
                        vae4_stream stream, const vae4_options *opt) {
  Prepared pr;
  int rc = prepare(q, nullptr, k_cache, v_cache, block_table, seq_lens, kv_scales, out, workspace,
                   opt, &pr);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_split(pr, st) != cudaSuccess) return VAE4_ERR_CUDA;
  if (vae4::launch_combine(pr.cp, st) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_partials(const vae4_tensor *q, const vae4_tensor *kv_pages,
                              const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                              const vae4_tensor *kv_scales, const vae4_tensor *out,
                              const vae4_tensor *workspace, vae4_stream stream,
                              const vae4_options *opt) {
  Prepared pr;
  int rc = prepare(q, kv_pages, nullptr, nullptr, block_table, seq_lens, kv_scales, out,
                   workspace, opt, &pr);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  if (launch_split(pr, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_combine(const vae4_tensor *q, const vae4_tensor *kv_pages,
                             const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                             const vae4_tensor *kv_scales, const vae4_tensor *out,
                             const vae4_tensor *workspace, vae4_stream stream,
                             const vae4_options *opt) {
  Prepared pr;
  int rc = prepare(q, kv_pages, nullptr, nullptr, block_table, seq_lens, kv_scales, out,
                   workspace, opt, &pr);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  if (vae4::launch_combine(pr.cp, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_kv_read(const vae4_tensor *q, const vae4_tensor *kv_pages,
                             const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                             const vae4_tensor *kv_scales, const vae4_tensor *out,
                             const vae4_tensor *workspace, vae4_stream stream,
                             const vae4_options *opt) {
  Prepared pr;
  int rc = prepare(q, kv_pages, nullptr, nullptr, block_table, seq_lens, kv_scales, out,
                   workspace, opt, &pr);
  if (rc) return rc;
  if (pr.empty) return VAE4_OK;
  if (vae4::launch_kv_read(pr.sp, pr.num_sms, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3(const vae4_tensor *q, const vae4_tensor *kv_pages,
                     const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                     const vae4_tensor *kv_scales, const vae4_tensor *out,
                     const vae4_tensor *workspace, vae4_stream stream) {
  return verify_attn_e4m3_ex(q, kv_pages, block_table, seq_lens, kv_scales, out, workspace,
                             stream, nullptr);
}

int verify_attn_e4m3_plan(int B, int Hkv, int max_seq_len, int partition_tokens, int num_sms,
                          int32_t *partition_tokens_out, int32_t *partitions_out) {
  if (!partition_tokens_out || !partitions_out) return VAE4_ERR_NULL;
  int T = 0, P = 0;
  const int rc = do_plan(B, Hkv, max_seq_len, partition_tokens, num_sms, &T, &P);
  if (rc) return rc;
  *partition_tokens_out = T;
  *partitions_out = P;
  return VAE4_OK;
}

int64_t verify_attn_e4m3_workspace_bytes(int B, int Hq, int Hkv, int Qmax, int D,
                                         int max_seq_len, int partition_tokens, int num_sms) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Qmax < 1 || Qmax > kMaxQmax || max_seq_len < 1)
    return VAE4_ERR_SHAPE;
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return VAE4_ERR_GQA;
  if (align_up((int64_t)Qmax * (Hq / Hkv), 16) > kMaxRowsPad) return VAE4_ERR_UNSUPPORTED;
  const int64_t rows_pad = ws_rows(Qmax * (Hq / Hkv));
  int sms = num_sms;
  if (sms < 0) return VAE4_ERR_SHAPE;
  if (sms == 0) {
    const int rc = device_sms(&sms);
    if (rc) return rc;
  }
  int T = 0, P = 0;
  const int rc = do_plan(B, Hkv, max_seq_len, partition_tokens, sms, &T, &P);
  if (rc) return rc;
  return ws_layout(ws_slots(B, Hkv, P, partition_tokens, sms, vae4_tc_groups(Qmax * (Hq / Hkv))),
                   (int)rows_pad, D, (int64_t)B * Hkv)
      .total;
}

int verify_attn_e4m3_abi_version(void) { return VAE4_ABI_VERSION; }

const char *verify_attn_e4m3_strerror(int code) {
  switch (code) {
    case VAE4_OK: return "ok";
    case VAE4_ERR_NULL: return "a required pointer is NULL";
    case VAE4_ERR_DTYPE: return "wrong dtype";
    case VAE4_ERR_SHAPE: return "inconsistent or out-of-range shape";
    case VAE4_ERR_STRIDE: return "unsupported strides";
    case VAE4_ERR_MISALIGNED: return "base address or row not 16-byte aligned";
    case VAE4_ERR_UNSUPPORTED: return "head dim, page, block or row count not supported";
    case VAE4_ERR_GQA: return "q heads not a multiple of KV heads";
    case VAE4_ERR_WORKSPACE: return "workspace too small or not 256-byte aligned";
    case VAE4_ERR_CUDA: return "CUDA runtime error";
    case VAE4_ERR_PARTITION: return "partition_tokens must be a positive multiple of 16 giving at most 8192 partitions";
    case VAE4_ERR_OPTIONS: return "invalid options";
    default: return "unknown error";
  }
}

int verify_attn_e4m3_read_status(const vae4_tensor *workspace, int32_t *host_status,
                                 vae4_stream stream) {
  if (!workspace || !workspace->data || !host_status) return VAE4_ERR_NULL;
  if (workspace->dtype != VAE4_U8) return VAE4_ERR_DTYPE;
  if (workspace->ndim != 1 || workspace->shape[0] < kStatusBytes) return VAE4_ERR_WORKSPACE;
  if (cudaMemcpyAsync(host_status, workspace->data, sizeof(int32_t), cudaMemcpyDeviceToHost,
                      reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_clear_status(const vae4_tensor *workspace, vae4_stream stream) {
  if (!workspace || !workspace->data) return VAE4_ERR_NULL;
  if (workspace->dtype != VAE4_U8) return VAE4_ERR_DTYPE;
  if (workspace->ndim != 1 || workspace->shape[0] < kStatusBytes) return VAE4_ERR_WORKSPACE;
  if (cudaMemsetAsync(workspace->data, 0, sizeof(int32_t),
                      reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_decode_table(void *dev_out, int32_t *scale_log2, int32_t flags,
                                  vae4_stream stream) {
  if (!dev_out || !scale_log2) return VAE4_ERR_NULL;
  if (!al16(dev_out)) return VAE4_ERR_MISALIGNED;
  if ((flags & ~(VAE4_FLAG_WARP_MMA | VAE4_FLAG_KV_E5M2)) != 0) return VAE4_ERR_OPTIONS;
  if ((flags & VAE4_FLAG_WARP_MMA) && (flags & VAE4_FLAG_KV_E5M2)) return VAE4_ERR_UNSUPPORTED;
  const bool integer_path = (flags & VAE4_FLAG_WARP_MMA) != 0;
  const bool e5m2 = (flags & VAE4_FLAG_KV_E5M2) != 0;
  *scale_log2 = integer_path ? -8 : 0;
  if (vae4::launch_decode_table(static_cast<uint16_t *>(dev_out), integer_path, e5m2,
                                reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return VAE4_ERR_CUDA;
  return VAE4_OK;
}

}  // extern "C"
