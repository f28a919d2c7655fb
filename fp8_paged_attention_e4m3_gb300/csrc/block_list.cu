// Visit lists of sparse attention: for every (sequence, KV head) the blocks
// that at least one of its queries attends to, in ascending order, each with
// a bit per query, its page, and its scales ready for the softmax.  A block
// that several queries chose is then read once.
//
// One CTA per stream: a 16-bit query mask per block of the sequence in shared
// memory, set from the queries' lists (an OR, so the order and repetitions of
// the ids do not matter); every thread counts the blocks in its share of the
// masks, a scan over the CTA places them, and then the entries are filled in,
// one per thread, so that the loads of their pages and scales are all under
// way together.  (Filling them in as they were found, 32 blocks of a warp's
// share after another, took 31.5 us for 16384 blocks; this takes 6.)
#include <algorithm>
#include <atomic>

#include "block_common.cuh"
#include "kernels.h"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kListThreads = 512;
constexpr int kListWarps = kListThreads / 32;

__global__ void __launch_bounds__(kListThreads) block_list_kernel(const ListParams p) {
  extern __shared__ __align__(16) uint32_t masks[];  // two blocks per word
  __shared__ int wsum[kListWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, stream = b * p.Hkv + h;
  // the split kernel may be placed already (it waits for this grid), and this
  // grid for the previous call's kernels, which read the lists
  await_previous();
  const int L = p.seq[(int64_t)b * p.seq_sb];
  const int n = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
  const bool bad_l = L < 0 || L > p.capacity;
  const bool bad = bad_l || n < 0 || n > p.Qmax || (L > 0 && n > L);
  if (bad && h == 0 && tid == 0)
    atomicOr(p.status, bad_l ? VAE4_STATUS_BAD_LENGTH : VAE4_STATUS_BAD_QLEN);
  const int nblk = bad || n == 0 || L == 0 ? 0 : (L - 1) / p.blk + 1;
  const int quads = (nblk + 7) / 8;  // eight blocks (16 bytes) each
  uint4 *m4 = reinterpret_cast<uint4 *>(masks);
  for (int x = tid; x < quads; x += kListThreads) m4[x] = make_uint4(0u, 0u, 0u, 0u);
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
  // ---- this thread's share: quads q0 .. q1
  const int per = (quads + kListThreads - 1) / kListThreads;
  const int q0 = min(tid * per, quads), q1 = min(q0 + per, quads);
  auto count4 = [](uint4 v) -> int {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    int c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) c += ((w[e] & 0xFFFFu) != 0u) + ((w[e] >> 16) != 0u);
    return c;
  };
  int mine = 0;
  for (int x = q0; x < q1; ++x) mine += count4(m4[x]);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  const int ws = lane < kListWarps ? wsum[lane] : 0;
  const int base = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
  const int total = __reduce_add_sync(0xffffffffu, ws);
  BlockEntry *out = p.list + (int64_t)stream * p.list_cap;
  int at = base + incl - mine;
  for (int x = q0; x < q1 && mine > 0; ++x) {
    const uint4 v = m4[x];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t mk = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      if (mk != 0u) *reinterpret_cast<int2 *>(&out[at++].tok0) = make_int2((8 * x + e) * p.blk, (int)mk);
    }
  }
  const bool last = nblk > 0 && ((masks[(nblk - 1) >> 1] >> (16 * ((nblk - 1) & 1))) & 0xFFFFu) != 0u;
  __syncthreads();
  // ---- pages and scales
  for (int x = tid; x < total; x += kListThreads) {
    const int tok0 = out[x].tok0;
    const int lp = tok0 / p.page, slot = tok0 - lp * p.page;
    const int phys = p.bt[(int64_t)b * p.bt_sb + lp];
    int2 head = make_int2(-1, slot >> 4);
    float4 tail = make_float4(0.f, 0.f, 1.f, 0.f);
    if (phys >= 0 && phys < p.n_pages) {
      const float *s = p.scales + (int64_t)phys * p.s_page + (int64_t)h * p.s_head + slot / p.blk;
      const float sk = s[0], sv = s[p.s_kv];
      if (sk >= kMinScale && sk <= kMaxScale && sv >= kMinScale && sv <= kMaxScale) {
        head.x = phys;
        tail = make_float4(p.alpha * sk, log2f(sv), 1.f / sv, 0.f);
      } else {
        atomicOr(p.status, VAE4_STATUS_BAD_SCALE);
      }
    } else {
      atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
    }
    *reinterpret_cast<int2 *>(&out[x].phys) = head;
    *reinterpret_cast<float4 *>(&out[x].alpha) = tail;
  }
  if (tid == 0) {
    BlockStream s{0, 0, 0, 0};
    if (total > 0) {
      // only the sequence's last block can be partial
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
  const int smem = (nblk + 7) / 8 * 16;
  if (smem > 48 * 1024) {  // beyond the default dynamic shared-memory limit
    // The limit belongs to the function in the device's context, whatever host
    // thread sets it: once per context, to the most that any call needs, so that
    // none lowers it between another's setting and launch.
    constexpr int kDevs = 64;
    static std::atomic<unsigned long long> configured[kDevs] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    if (dev < 0 || dev >= kDevs || ctx == 0 ||
        configured[dev].load(std::memory_order_acquire) != ctx) {
      const cudaError_t e =
          cudaFuncSetAttribute(block_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kMaxListBlocks * 2);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < kDevs)
        configured[dev].store(current_context_id(), std::memory_order_release);
    }
  }
  return launch_dependent(block_list_kernel, dim3((unsigned)p.Hkv, (unsigned)p.B), kListThreads,
                          (size_t)smem, stream, p);
}

}  // namespace vae4
