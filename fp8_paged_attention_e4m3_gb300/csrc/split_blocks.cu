// Split (partition) stage of attention over a block-scaled cache, dense or
// over sparse attention's visit lists: the plain form of the computation,
// FP32 products in shared memory.
//
// A partition walks its keys in 16-key boxes (a box lies in one block, so it
// has one s_K and one s_V).  With t = alpha (q . dec(K)) the score in log2
// units and g = log2 s_V, the weight of a key is w = 2^(t + g - m), m the
// running maximum of t + g: O += w dec(V) and l += w / s_V, so
// O / l = sum e^z s_V dec(V) / sum e^z for any m.
#include "common.cuh"
#include "kernels.h"
#include "plan.cuh"
#include "verify_attn_e4m3.h"

namespace vae4 {

namespace {

constexpr int kThreads = 256;

constexpr int smem_floats(int D, int rows) {
  return rows * D /* O */ + rows * (D / 2 + 1) /* q, half2 */ + 2 * 16 * (D + 1) /* K, V */ +
         rows * 16 /* w */ + 3 * rows /* m, l, factor */;
}

template <bool E5M2>
__global__ void __launch_bounds__(kThreads) split_blocks_kernel(const SplitParams p) {
  extern __shared__ float sm[];
  const int D = p.D, rows = p.rows;
  float *o_s = sm;
  __half2 *q_s = reinterpret_cast<__half2 *>(o_s + rows * D);
  float *k_s = reinterpret_cast<float *>(q_s + rows * (D / 2 + 1));
  float *v_s = k_s + 16 * (D + 1), *w_s = v_s + 16 * (D + 1);
  float *m_s = w_s + rows * 16, *l_s = m_s + rows, *f_s = l_s + rows;
  __shared__ int bad_s;
  const int tid = threadIdx.x;
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const bool list = p.bs.list != nullptr;
  const int stream = b * p.Hkv + h;
  const float ninf = -__int_as_float(0x7f800000);
  const float klog2e = 1.4426950408889634f;
  int L, ql, Lv, T = p.T;
  if (list) {
    const BlockStream s = p.bs.streams[stream];
    L = s.L;
    ql = s.ql;
    Lv = s.n;
    if (Lv == 0) return;
    T = max(64, plan_t_from_len(s.n16, p.P));
    if (part == 0 && tid == 0) p.plan_tab[stream] = make_int2(stream * p.P, (s.n16 + T - 1) / T);
  } else {
    L = p.seq[(int64_t)b * p.seq_sb];
    ql = p.seq_has_qlen ? p.seq[(int64_t)b * p.seq_sb + 1] : p.Qmax;
    if (L <= 0 || L > p.capacity || ql <= 0 || ql > p.Qmax || ql > L) return;  // the combine reports
    Lv = L;
  }
  const int k0 = part * T;
  if (k0 >= Lv) return;
  const int k1 = min(k0 + T, Lv);
  for (int x = tid; x < rows * D; x += kThreads) o_s[x] = 0.f;
  for (int x = tid; x < rows; x += kThreads) {
    m_s[x] = ninf;
    l_s[x] = 0.f;
  }
  for (int x = tid; x < rows * (D / 2); x += kThreads) {
    const int r = x / (D / 2), c = x - r * (D / 2), i = r / p.G, g = r - i * p.G;
    __half2 v = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
    if (i < ql)
      v = *reinterpret_cast<const __half2 *>(static_cast<const __half *>(p.q) + (int64_t)b * p.q_sb +
                                             (int64_t)i * p.q_si + (int64_t)(h * p.G + g) * p.q_sh + 2 * c);
    q_s[r * (D / 2 + 1) + c] = v;
  }
  if (tid == 0) bad_s = 0;
  __syncthreads();
  for (int k = k0; k < k1; k += 16) {
    int phys, slot, pos;
    uint32_t mask = 0xFFFFu;
    float alpha = 0.f, lgv = 0.f, inv_sv = 1.f;
    bool bad = false;
    if (list) {
      const int e = k / p.bs.blk;
      const BlockEntry t = p.bs.list[(int64_t)stream * p.bs.list_cap + e];
      phys = t.phys;
      slot = 16 * t.box0 + k - e * p.bs.blk;
      pos = t.tok0 + k - e * p.bs.blk;
      mask = t.mask;
      alpha = t.alpha;
      lgv = t.lgv;
      inv_sv = t.inv_sv;
      bad = phys < 0;
    } else {
      pos = k;
      slot = k % p.page;
      phys = p.bt[(int64_t)b * p.bt_sb + k / p.page];
      bad = phys < 0 || phys >= p.n_pages;
      if (bad && tid == 0) atomicOr(p.status, VAE4_STATUS_BAD_BLOCK);
      if (!bad) {
        const float *s = p.bs.scales + (int64_t)phys * p.bs.s_page + (int64_t)h * p.bs.s_head + slot / p.bs.blk;
        const float sk = s[0], sv = s[p.bs.s_kv];
        bad = !(sk >= kMinScale && sk <= kMaxScale && sv >= kMinScale && sv <= kMaxScale);
        if (bad && tid == 0) atomicOr(p.status, VAE4_STATUS_BAD_SCALE);
        alpha = p.sm_scale * klog2e * sk;
        lgv = log2f(sv);
        inv_sv = 1.f / sv;
      }
    }
    if (bad) {  // the same for every thread
      if (tid == 0) bad_s = 1;
      break;
    }
    for (int x = tid; x < 16 * (D / 2); x += kThreads) {
      const int t = x / (D / 2), c = x - t * (D / 2);
      float2 kv = make_float2(0.f, 0.f), vv = kv;
      if (k + t < k1) {
        const uint32_t kr = *reinterpret_cast<const uint16_t *>(
            p.k_base + (int64_t)phys * p.k_ps + (int64_t)(slot + t) * p.k_ts + (int64_t)h * p.k_hs + 2 * c);
        const uint32_t vr = *reinterpret_cast<const uint16_t *>(
            p.v_base + (int64_t)phys * p.v_ps + (int64_t)(slot + t) * p.v_ts + (int64_t)h * p.v_hs + 2 * c);
        const uint32_t kh = fp8x2_to_f16x2<E5M2>(kr), vh = fp8x2_to_f16x2<E5M2>(vr);
        kv = __half22float2(*reinterpret_cast<const __half2 *>(&kh));
        vv = __half22float2(*reinterpret_cast<const __half2 *>(&vh));
      }
      k_s[t * (D + 1) + 2 * c] = kv.x;
      k_s[t * (D + 1) + 2 * c + 1] = kv.y;
      v_s[t * (D + 1) + 2 * c] = vv.x;
      v_s[t * (D + 1) + 2 * c + 1] = vv.y;
    }
    __syncthreads();
    for (int x = tid; x < rows * 16; x += kThreads) {
      const int r = x >> 4, t = x & 15, i = r / p.G;
      float s = 0.f;
      for (int c = 0; c < D / 2; ++c) {
        const float2 q = __half22float2(q_s[r * (D / 2 + 1) + c]);
        s += q.x * k_s[t * (D + 1) + 2 * c] + q.y * k_s[t * (D + 1) + 2 * c + 1];
      }
      const bool see = k + t < k1 && i < ql && pos + t <= L - ql + i && ((mask >> i) & 1u);
      w_s[x] = see ? s * alpha + lgv : ninf;
    }
    __syncthreads();
    for (int r = tid; r < rows; r += kThreads) {
      float mx = m_s[r];
      for (int t = 0; t < 16; ++t) mx = fmaxf(mx, w_s[r * 16 + t]);
      const float f = mx == m_s[r] ? 1.f : exp2f(m_s[r] - mx);
      float l = l_s[r] * f;
      for (int t = 0; t < 16; ++t) {
        const float w = mx == ninf ? 0.f : exp2f(w_s[r * 16 + t] - mx);
        w_s[r * 16 + t] = w;
        l += w * inv_sv;
      }
      m_s[r] = mx;
      l_s[r] = l;
      f_s[r] = f;
    }
    __syncthreads();
    for (int x = tid; x < rows * D; x += kThreads) {
      const int r = x / D, d = x - r * D;
      float o = o_s[x] * f_s[r];
      for (int t = 0; t < 16; ++t) o += w_s[r * 16 + t] * v_s[t * (D + 1) + d];
      o_s[x] = o;
    }
    __syncthreads();
  }
  __syncthreads();
  const int64_t base = ((int64_t)stream * p.P + part) * p.rows_pad;
  for (int r = tid; r < rows; r += kThreads) {
    p.ws_ml[(base + r) * 2] = m_s[r];
    p.ws_ml[(base + r) * 2 + 1] = bad_s ? -1.f : l_s[r];
  }
  for (int x = tid; x < rows * D; x += kThreads) p.ws_o[base * D + x] = o_s[x] * 0.00390625f;
}

}  // namespace

cudaError_t launch_split_blocks(const SplitParams &p, cudaStream_t stream) {
  const int smem = smem_floats(p.D, p.rows) * 4;
  auto fn = p.kv_e5m2 ? split_blocks_kernel<true> : split_blocks_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fn<<<dim3((unsigned)p.P, (unsigned)p.Hkv, (unsigned)p.B), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vae4
