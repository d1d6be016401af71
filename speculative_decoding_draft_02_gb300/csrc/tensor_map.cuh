// tensor_map.cuh — tensor maps of any rank, on the host: the caches' and the queries' of
// the attentions.
#pragma once
#include <cuda.h>

#include <atomic>

#include "common.cuh"

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps; null while there is none (asked for again then).
EncodeFn tensor_map_encoder() {
  static std::atomic<EncodeFn> kept{nullptr};
  EncodeFn f = kept.load();
  if (!f) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    f = (EncodeFn)fn;
    kept.store(f);
  }
  return f;
}

// A tensor map of RANK dimensions: dims and box in elements (dimension 0 contiguous),
// strides in bytes for dimensions 1.. (multiples of 16); zeros outside.
template <int RANK>
bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base,
              const uint64_t (&dims)[RANK], const uint64_t (&strides)[RANK - 1],
              const uint32_t (&box)[RANK], CUtensorMapSwizzle swizzle) {
  const EncodeFn encode = tensor_map_encoder();
  if (!encode) return false;
  cuuint64_t d[RANK], s[RANK - 1];
  cuuint32_t b[RANK], step[RANK];
  for (int i = 0; i < RANK; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    step[i] = 1;
    if (i + 1 < RANK) s[i] = strides[i];
  }
  return encode(map, type, RANK, const_cast<void *>(base), d, s, b, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
