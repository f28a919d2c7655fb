// Host launcher of the split kernel over block-scaled caches: the TMA tensor
// maps of K and V and the choice of the instantiation.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <string.h>

#include <mutex>

#include "seg_tc.cuh"

namespace vae4 {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

bool mappable(const uint8_t *base, int64_t ps, int64_t ts, int64_t hs) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ps % 16 == 0 && ts % 16 == 0 &&
         hs % 16 == 0 && ps < ((int64_t)1 << 40) && ts < ((int64_t)1 << 40) &&
         hs < ((int64_t)1 << 40);
}

// The 5-D tensor map of one cache: coordinates (byte within a swizzled row,
// token in the page, row of the key, KV head, page); a box is 2^box_log2 keys
// of one head, in shared memory D / IB blocks of that many rows of IB bytes.
bool encode(CUtensorMap *map, const uint8_t *base, int64_t ps, int64_t ts, int64_t hs,
            const SegParams &p) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int D = p.D, IB = D < 128 ? D : 128;
  const cuuint64_t dims[5] = {(cuuint64_t)IB, (cuuint64_t)p.page, (cuuint64_t)(D / IB),
                              (cuuint64_t)p.Hkv, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)ts, (cuuint64_t)IB, (cuuint64_t)hs, (cuuint64_t)ps};
  const cuuint32_t box[5] = {(cuuint32_t)IB, 1u << p.box_log2, (cuuint32_t)(D / IB), 1u, 1u};
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  // fetches into L2 no wider than what lies together: in a token-major cache
  // of several heads the neighbouring bytes are another head's
  const int64_t run = ts == D ? 256 : D;
  const CUtensorMapL2promotion promotion = run >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : run >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                        : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<uint8_t *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            IB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            promotion,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_seg(const SegParams &p_in, cudaStream_t stream) {
  SegParams p = p_in;
  if (p.n_pages > 0x7fffffff) return cudaErrorInvalidValue;  // 32-bit page coordinate
  // the largest copy that a page (a listed block) is a multiple of: segments
  // start at multiples of 64 keys, so it never crosses one
  const int unit = p.list ? p.blk : p.page;
  p.box_log2 = unit % 64 == 0 ? 6 : unit % 32 == 0 ? 5 : 4;
  p.page_blocks = p.page / p.blk;
  p.page_m = reciprocal16(p.page);
  p.blk_m = reciprocal16(p.blk);
  CUtensorMap map_k, map_v;
  memset(&map_k, 0, sizeof(map_k));
  memset(&map_v, 0, sizeof(map_v));
  p.cpasync = 0;
  if (!mappable(p.k_base, p.k_ps, p.k_ts, p.k_hs) || !mappable(p.v_base, p.v_ps, p.v_ts, p.v_hs) ||
      !encode(&map_k, p.k_base, p.k_ps, p.k_ts, p.k_hs, p) ||
      !encode(&map_v, p.v_base, p.v_ps, p.v_ts, p.v_hs, p)) {
    p.cpasync = 1;
    p.box_log2 = 4;
  }
  switch (p.D) {
    case 64: return seg::launch_64(p, map_k, map_v, stream);
    case 128: return seg::launch_128(p, map_k, map_v, stream);
    case 256: return seg::launch_256(p, map_k, map_v, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace vae4
