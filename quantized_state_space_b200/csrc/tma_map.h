// Host side of TMA tensor maps: the driver's encoder, looked up at run time (the
// library does not link libcuda).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace ssmq {

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up once per process; NULL when the driver has none
inline EncodeFn tensor_map_encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A tiled map of `rank` dimensions without interleave, element strides 1, zeros
// beyond the tensor.  The encoder needs the thread's context, which a thread
// whose first CUDA call this is does not have yet: the current device is then
// set again and the call repeated.
inline cudaError_t encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* p,
                                const cuuint64_t* dims, const cuuint64_t* strides,
                                const cuuint32_t* box, CUtensorMapSwizzle swizzle,
                                CUtensorMapL2promotion promotion) {
  const EncodeFn fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 2; ++i) {
    if (fn(map, type, (cuuint32_t)rank, const_cast<void*>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
      return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
  }
  return cudaErrorInvalidValue;
}

}  // namespace ssmq
