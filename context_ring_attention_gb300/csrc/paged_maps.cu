// Tensor maps of the paged cache's tensor-core kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged_internal.h"

namespace ra {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encoder() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

bool encode(void* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(static_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_rows(void* map, const void* base, int64_t rows, int d, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  return encode(map, base, 2, dims, strides, boxes);
}

bool encode_packed(void* map, const void* base, const PagedStrides& s, int64_t tokens, int64_t heads, int d, int group,
                   int box) {
  // (an axis of one element has no stride that matters)
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? s.head : d) * 2, (cuuint64_t)(tokens > 1 ? s.token : d) * 2};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)box};
  return encode(map, base, 3, dims, strides, boxes);
}

}  // namespace ra
