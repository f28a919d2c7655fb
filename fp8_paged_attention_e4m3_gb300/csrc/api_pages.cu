// C-ABI entry points of the pages' lives: copying pages of a cache, and a pool's fork,
// resize and compaction.  See include/verify_attn_e4m3.h for the contract of every
// function.
#include "api_prepare.h"
#include "page_params.h"

using namespace vae4;

namespace {

constexpr int64_t kMaxCells = (int64_t)1 << 30;  // entries of a table; vectors of a page

// A page's part of one tensor: n[k] x .. runs of `bytes` bytes (dimensions of one or
// that continue their neighbour are merged into the run)
int make_slab(void *base, int64_t ps, const int64_t *n, const int64_t *s, int64_t bytes, int vec,
              int64_t first, PageSlab *o) {
  o->base = static_cast<uint8_t *>(base);
  o->ps = ps;
  int64_t dn[3], ds[3];
  int dims = 0;
  for (int k = 0; k < 3; ++k)
    if (n[k] > 1) {
      dn[dims] = n[k];
      ds[dims++] = s[k];
    }
  // innermost first: the smallest stride
  for (int a = 0; a < dims; ++a)
    for (int b = a + 1; b < dims; ++b)
      if (ds[b] > ds[a]) {
        std::swap(ds[a], ds[b]);
        std::swap(dn[a], dn[b]);
      }
  while (dims > 0 && ds[dims - 1] == bytes) bytes *= dn[--dims];
  int64_t total = bytes / vec;
  for (int k = 0; k < 3; ++k) {
    const int d = k - (3 - dims);  // outer dimensions of one, then the rest
    o->n[k] = d >= 0 ? (int32_t)dn[d] : 1;
    o->s[k] = d >= 0 ? ds[d] : 0;
    total *= o->n[k];
  }
  if (first + total > kMaxCells) return VAE4_ERR_SHAPE;
  o->run = (int32_t)(bytes / vec);
  o->first = (int32_t)first;
  o->vecs = (int32_t)total;
  return VAE4_OK;
}

// block table I32 [B][columns], counts I32 [n_pages]
int check_pool_state(const vae4_tensor *bt, const vae4_tensor *counts, uint32_t *status,
                     PoolParams *o) {
  if (bt->ndim != 2 || bt->shape[0] < 0) return bt->dtype != VAE4_I32 ? VAE4_ERR_DTYPE : VAE4_ERR_SHAPE;
  const int rc = check_table(bt, bt->shape[0]);
  if (rc) return rc;
  if (counts->dtype != VAE4_I32) return VAE4_ERR_DTYPE;
  if (counts->ndim != 1 || counts->shape[0] < 1 || counts->shape[0] > kMaxCells) return VAE4_ERR_SHAPE;
  if (counts->stride[0] != 1) return VAE4_ERR_STRIDE;
  if (bt->shape[0] > kMaxCells || bt->shape[0] * bt->shape[1] > kMaxCells) return VAE4_ERR_SHAPE;
  // rows are written: they must not share memory
  if (overlaps(bt, 1, bt->shape[1]) || bt->stride[0] >= ((int64_t)1 << 40)) return VAE4_ERR_STRIDE;
  for (const vae4_tensor *t : {bt, counts})
    if ((reinterpret_cast<uintptr_t>(t->data) & 3u) != 0) return VAE4_ERR_MISALIGNED;
  o->bt = static_cast<int32_t *>(bt->data);
  o->bt_sb = bt->stride[0];
  o->B = (int32_t)bt->shape[0];
  o->cols = (int32_t)bt->shape[1];
  o->counts = static_cast<int32_t *>(counts->data);
  o->n_pages = (int32_t)counts->shape[0];
  o->status = status;
  return VAE4_OK;
}

// pairs: I32 [n][2]; written ones must not overlap
int check_pairs(const vae4_tensor *t, bool written) {
  if (t->dtype != VAE4_I32) return VAE4_ERR_DTYPE;
  if (t->ndim != 2 || t->shape[0] < 0 || t->shape[0] > INT32_MAX / 2 || t->shape[1] != 2)
    return VAE4_ERR_SHAPE;
  if (t->stride[1] != 1 || t->stride[0] < 0 || t->stride[0] >= ((int64_t)1 << 40))
    return VAE4_ERR_STRIDE;
  if (written && overlaps(t, 1, 2)) return VAE4_ERR_STRIDE;
  if ((reinterpret_cast<uintptr_t>(t->data) & 3u) != 0) return VAE4_ERR_MISALIGNED;
  return VAE4_OK;
}

}  // namespace

extern "C" {

int verify_attn_e4m3_copy_pages(const vae4_tensor *k_cache, const vae4_tensor *v_cache,
                                const vae4_tensor *pairs, const vae4_tensor *block_scales,
                                const vae4_tensor *k_bounds, uint32_t *dev_status,
                                vae4_stream stream) {
  if (!k_cache || !v_cache || !pairs) return VAE4_ERR_NULL;
  if (k_cache->ndim != 4) return k_cache->dtype != VAE4_U8 ? VAE4_ERR_DTYPE : VAE4_ERR_SHAPE;
  const int64_t D = k_cache->shape[3];
  KvSrc src;
  int rc = check_kv(k_cache, v_cache, D, &src);
  if (rc) return rc;
  if (D != 64 && D != 128 && D != 256) return VAE4_ERR_UNSUPPORTED;
  if (overlaps(k_cache, 3, D) || overlaps(v_cache, 3, D)) return VAE4_ERR_STRIDE;
  if (src.Hkv > 32767) return VAE4_ERR_SHAPE;
  int64_t nb = 0;
  if (block_scales) {
    rc = check_block_scales(block_scales, src.n_pages, src.Hkv, src.page);
    if (rc) return rc;
    if (overlaps(block_scales, 3, block_scales->shape[3])) return VAE4_ERR_STRIDE;
    nb = block_scales->shape[3];
  }
  if (k_bounds) {
    if (!block_scales) {  // the blocks per page are the bounds' own
      if (k_bounds->ndim != 5) return k_bounds->dtype != VAE4_U8 ? VAE4_ERR_DTYPE : VAE4_ERR_SHAPE;
      nb = k_bounds->shape[2];
      if (nb < 1 || src.page % nb != 0 || (src.page / nb) % 16 != 0) return VAE4_ERR_UNSUPPORTED;
    }
    rc = check_bounds(k_bounds, src.n_pages, src.Hkv, nb, D);
    if (rc) return rc;
    if (overlaps(k_bounds, 4, D)) return VAE4_ERR_STRIDE;
  }
  rc = check_pairs(pairs, false);
  if (rc) return rc;
  CopyParams p;
  memset(&p, 0, sizeof(p));
  int64_t first = 0;
  const vae4_tensor *kv[2] = {k_cache, v_cache};
  for (int w = 0; w < 2; ++w) {
    const vae4_tensor *t = kv[w];
    bool wide = al16(t->data);
    for (int d = 0; d < 3; ++d) wide = wide && (t->stride[d] % 16 == 0 || t->shape[d] == 1);
    const int64_t n[3] = {t->shape[1], t->shape[2], 1}, s[3] = {t->stride[1], t->stride[2], 0};
    p.vec[w] = wide ? 16 : 8;
    rc = make_slab(t->data, t->stride[0], n, s, D, p.vec[w], first, &p.slab[w]);
    if (rc) return rc;
    first = align_up(first + p.slab[w].vecs, 32);
  }
  for (int w = 2; w < 4; ++w) p.slab[w].first = INT32_MAX;
  if (k_bounds) {
    const vae4_tensor *t = k_bounds;
    const int64_t n[3] = {t->shape[1], t->shape[2], t->shape[3]},
                  s[3] = {t->stride[1], t->stride[2], t->stride[3]};
    p.vec[2] = 16;
    rc = make_slab(t->data, t->stride[0], n, s, D, 16, first, &p.slab[2]);
    if (rc) return rc;
    first = align_up(first + p.slab[2].vecs, 32);
  }
  if (block_scales) {
    const vae4_tensor *t = block_scales;
    const int64_t n[3] = {t->shape[1], t->shape[2], 1}, s[3] = {4 * t->stride[1], 4 * t->stride[2], 0};
    p.vec[3] = 4;
    rc = make_slab(t->data, 4 * t->stride[0], n, s, 4 * nb, 4, first, &p.slab[3]);
    if (rc) return rc;
    first = align_up(first + p.slab[3].vecs, 32);
  }
  p.vecs = (int32_t)first;
  p.pairs = static_cast<const int32_t *>(pairs->data);
  p.pair_sb = pairs->stride[0];
  p.n = (int32_t)pairs->shape[0];
  p.n_pages = src.n_pages;
  p.status = dev_status;
  if (p.n == 0) return VAE4_OK;
  if (!src.kb || !src.vb || !pairs->data || (block_scales && !block_scales->data) ||
      (k_bounds && !k_bounds->data))
    return VAE4_ERR_NULL;
  if (launch_copy_pages(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_fork_pages(const vae4_tensor *block_table, const vae4_tensor *ref_counts,
                                const vae4_tensor *parents, uint32_t *dev_status,
                                vae4_stream stream) {
  if (!block_table || !ref_counts || !parents) return VAE4_ERR_NULL;
  ForkParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_pool_state(block_table, ref_counts, dev_status, &p.pool);
  if (rc) return rc;
  if (p.pool.B > kMaxForkRows) return VAE4_ERR_SHAPE;
  if (parents->dtype != VAE4_I32) return VAE4_ERR_DTYPE;
  if (parents->ndim != 1 || parents->shape[0] != p.pool.B) return VAE4_ERR_SHAPE;
  if (parents->stride[0] != 1 && p.pool.B > 1) return VAE4_ERR_STRIDE;
  p.parents = static_cast<const int32_t *>(parents->data);
  if (p.pool.B == 0) return VAE4_OK;
  if (!p.pool.bt || !p.pool.counts || !p.parents) return VAE4_ERR_NULL;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc) return rc;
  if (launch_fork_pages(p, sms, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int64_t verify_attn_e4m3_pages_workspace_bytes(int64_t n_pages) {
  if (n_pages < 1 || n_pages > kMaxCells) return VAE4_ERR_SHAPE;
  return kPoolGrid * 32 * 8 + align_up(4 * n_pages, 256);  // sums of the warps | list
}

int verify_attn_e4m3_resize_pages(const vae4_tensor *block_table, const vae4_tensor *seq_lens,
                                  const vae4_tensor *ref_counts, const vae4_tensor *copies,
                                  const vae4_tensor *workspace, int32_t page_tokens,
                                  uint32_t *dev_status, vae4_stream stream) {
  if (!block_table || !seq_lens || !ref_counts || !copies || !workspace) return VAE4_ERR_NULL;
  ResizeParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_pool_state(block_table, ref_counts, dev_status, &p.pool);
  if (rc) return rc;
  if (p.pool.B > kMaxResizeRows) return VAE4_ERR_SHAPE;
  int has_qlen = 0;
  rc = check_seq(seq_lens, p.pool.B, &has_qlen);
  if (rc) return rc;
  rc = check_pairs(copies, true);
  if (rc) return rc;
  if (copies->shape[0] != p.pool.B) return VAE4_ERR_SHAPE;
  if (page_tokens < 16 || page_tokens % 16 != 0 || page_tokens > 65536) return VAE4_ERR_UNSUPPORTED;
  if ((int64_t)p.pool.cols * page_tokens > INT32_MAX / 2) return VAE4_ERR_SHAPE;
  if (workspace->dtype != VAE4_U8) return VAE4_ERR_DTYPE;
  if (workspace->ndim != 1 || workspace->stride[0] != 1) return VAE4_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(workspace->data) & 255u) != 0 ||
      workspace->shape[0] < verify_attn_e4m3_pages_workspace_bytes(p.pool.n_pages))
    return VAE4_ERR_WORKSPACE;
  p.seq = static_cast<const int32_t *>(seq_lens->data);
  p.seq_sb = (int32_t)seq_lens->stride[0];
  p.seq_has_qlen = has_qlen;
  p.page = page_tokens;
  p.copies = static_cast<int32_t *>(copies->data);
  p.copies_sb = copies->stride[0];
  p.sums = static_cast<int2 *>(workspace->data);
  p.list = reinterpret_cast<int32_t *>(p.sums + kPoolGrid * 32);
  if (p.pool.B == 0) return VAE4_OK;
  if (!p.pool.bt || !p.pool.counts || !p.seq || !p.copies || !workspace->data) return VAE4_ERR_NULL;
  if (launch_resize_pages(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

int verify_attn_e4m3_compact_pages(const vae4_tensor *block_table, const vae4_tensor *ref_counts,
                                   const vae4_tensor *moves, uint32_t *dev_status,
                                   vae4_stream stream) {
  if (!block_table || !ref_counts || !moves) return VAE4_ERR_NULL;
  CompactParams p;
  memset(&p, 0, sizeof(p));
  int rc = check_pool_state(block_table, ref_counts, dev_status, &p.pool);
  if (rc) return rc;
  rc = check_pairs(moves, true);
  if (rc) return rc;
  p.moves = static_cast<int32_t *>(moves->data);
  p.moves_sb = moves->stride[0];
  p.n = (int32_t)moves->shape[0];
  if (p.n == 0 && (!dev_status || p.pool.B == 0)) return VAE4_OK;  // (else entries are looked at)
  if ((!p.pool.bt && p.pool.B > 0) || !p.pool.counts || (!p.moves && p.n > 0)) return VAE4_ERR_NULL;
  if (launch_compact_pages(p, cu(stream)) != cudaSuccess) return VAE4_ERR_CUDA;
  return VAE4_OK;
}

}  // extern "C"
