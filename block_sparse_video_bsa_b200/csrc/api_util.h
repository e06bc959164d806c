// Host-side helpers the C entry points share: pointer checks, the device check
// and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bsa {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The kernels use tcgen05 / TMA: sm_100 only.  BSA_OK, BSA_ERR_UNSUPPORTED or
// BSA_ERR_CUDA; cached per device.
int check_device();

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or NULL where the driver has none.
EncodeTiledFn encode_fn();

int cuda_status(cudaError_t e);

}  // namespace bsa
