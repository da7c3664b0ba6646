// Tensor maps for bulk tensor copies.
#pragma once

#include <cuda.h>

#include <mutex>

#include "fade_internal.cuh"

namespace fade {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// Per-head fp16 vectors [rows][tokens][heads][d] of any strides, boxes of 64 channels under the 128-byte
// swizzle. grouped: a box holds `heads_box` heads of `tokens_box` tokens (a token's heads one after
// another), coordinates (channel, head, token, row); otherwise tokens of one head, coordinates
// (channel, token, head, row). A stride that no coordinate but 0 uses does not matter; a dimension of
// stride 0 (a broadcast one) gets extent 1, and its coordinates have to be 0.
inline fade_status_t encode_heads(CUtensorMap* m, const char* name, const fade_heads_t& x, int d,
                                  long long heads, long long tokens, long long rows, int heads_box,
                                  int tokens_box, bool grouped) {
  EncodeFn fn = encode_fn();
  if (!fn) return set_error(FADE_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(grouped ? heads : tokens),
                        (cuuint64_t)(grouped ? tokens : heads), (cuuint64_t)rows};
  cuuint64_t strides[3] = {(cuuint64_t)(grouped ? x.head_stride : x.token_stride) * 2,
                           (cuuint64_t)(grouped ? x.token_stride : x.head_stride) * 2,
                           (cuuint64_t)x.row_stride * 2};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] == 0) dims[i + 1] = 1;
    if (dims[i + 1] == 1) strides[i] = (cuuint64_t)d * 2;
  }
  const cuuint32_t box[4] = {64u, (cuuint32_t)(grouped ? heads_box : tokens_box),
                             (cuuint32_t)(grouped ? tokens_box : 1), 1u};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, x.x, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(FADE_ERR_CUDA, "cuTensorMapEncodeTiled (%s) failed (%d)", name, (int)r);
  return FADE_OK;
}

// One box of a map of encode_heads, into shared memory, counted on an mbarrier.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                         int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

}  // namespace fade
