// Visit lists of sparse attention: for every (sequence, KV head) the blocks
// that at least one of its queries attends to, in ascending order, each with
// a bit per query, its page, and its scales ready for the softmax.  A block
// that several queries chose is then read once.
//
// One CTA per stream: a 16-bit query mask per block of the sequence in shared
// memory, set from the queries' lists (an OR, so the order and repetitions of
// the ids do not matter), then a compaction in block order.
#include "common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kListThreads = 512;
constexpr int kListWarps = kListThreads / 32;

__global__ void __launch_bounds__(kListThreads) block_list_kernel(const ListParams p) {
  extern __shared__ uint32_t masks[];  // two blocks per word
  __shared__ int wcnt[kListWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, stream = b * p.Hkv + h;
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool bad_l = L < 0 || L > p.capacity;
  const bool bad = bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L);
  if (bad && h == 0 && tid == 0)
    atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
  const int nblk = bad || n == 0 || L == 0 ? 0 : (L - 1) / p.blk + 1;
  const int words = (nblk + 1) / 2;
  for (int x = tid; x < words; x += kListThreads) masks[x] = 0u;
  __syncthreads();
  if (nblk > 0) {
    for (int x = tid; x < n * p.k; x += kListThreads) {
      const int i = x / p.k, kk = x - i * p.k;
      const int id = p.ids[(int64_t)b * p.i_sb + (int64_t)i * p.i_si + (int64_t)h * p.i_sh + kk];
      // a block that starts past the query's position has nothing for it
      if (id >= 0 && id < nblk && (int64_t)id * p.blk <= L - n + i)
        atomicOr(&masks[id >> 1], (1u << i) << (16 * (id & 1)));
    }
  }
  __syncthreads();
  auto mask_of = [&](int x) -> uint32_t { return (masks[x >> 1] >> (16 * (x & 1))) & 0xFFFFu; };
  const int seg = ((nblk + kListWarps - 1) / kListWarps + 31) & ~31;
  const int x0 = min(warp * seg, nblk), x1 = min(x0 + seg, nblk);
  int cnt = 0;
  for (int x = x0; x < x1; x += 32)
    cnt += __popc(__ballot_sync(0xffffffffu, x + lane < x1 && mask_of(x + lane) != 0u));
  if (lane == 0) wcnt[warp] = cnt;
  __syncthreads();
  int base = 0, total = 0;
  for (int k = 0; k < kListWarps; ++k) {
    if (k < warp) base += wcnt[k];
    total += wcnt[k];
  }
  BlockEntry *out = p.list + (int64_t)stream * p.list_cap;
  for (int x = x0; x < x1; x += 32) {
    const int j = x + lane;
    const uint32_t mk = j < x1 ? mask_of(j) : 0u;
    const uint32_t any = __ballot_sync(0xffffffffu, mk != 0u);
    if (mk != 0u) {
      const int64_t t0 = (int64_t)j * p.blk;
      const int lp = (int)(t0 / p.page), slot = (int)(t0 - (int64_t)lp * p.page);
      const int phys = p.bt[(int64_t)b * p.bt_sb + lp];
      BlockEntry e{-1, slot >> 4, (int)t0, mk, 0.f, 0.f, 1.f, 0};
      if (phys >= 0 && phys < p.n_pages) {
        const float *s = p.scales + (int64_t)phys * p.s_page + (int64_t)h * p.s_head + slot / p.blk;
        const float sk = s[0], sv = s[p.s_kv];
        if (sk >= kMinScale && sk <= kMaxScale && sv >= kMinScale && sv <= kMaxScale) {
          e.phys = phys;
          e.alpha = p.alpha * sk;
          e.lgv = log2f(sv);
          e.inv_sv = 1.f / sv;
        } else {
          atomicOr(p.status, VAE4_STATUS_BAD_SCALE);
        }
      } else {
        atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
      }
      out[base + __popc(any & ((1u << lane) - 1u))] = e;
    }
    base += __popc(any);
  }
  if (tid == 0) {
    BlockStream s{0, 0, 0, 0};
    if (total > 0) {
      // only the sequence's last block can be partial
      const bool last = mask_of(nblk - 1) != 0u;
      s.n = total * p.blk - (last ? nblk * p.blk - L : 0);
      s.n16 = (s.n + 15) & ~15;
      s.ql = n;
      s.L = L;
    }
    p.streams[stream] = s;
    for (int r = 0; r < p.n_rg; ++r) p.tab[stream * p.n_rg + r] = make_int2(0, 0);
  }
}

}  // namespace

cudaError_t launch_block_list(const ListParams &p, cudaStream_t stream) {
  const int nblk = (p.capacity + p.blk - 1) / p.blk;
  const int smem = (nblk + 1) / 2 * 4;
  if (smem > 48 * 1024) {  // beyond the default dynamic shared-memory limit
    const cudaError_t e =
        cudaFuncSetAttribute(block_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  block_list_kernel<<<dim3((unsigned)p.Hkv, (unsigned)p.B), kListThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vae4
