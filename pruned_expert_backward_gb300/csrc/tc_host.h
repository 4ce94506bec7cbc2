// Host helpers of the tensor-core kernels (defined in gemm_tc.cu).
#pragma once

#include <cuda.h>

namespace lrm {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // cuTensorMapEncodeTiled, or NULL where the driver has none
int sm_count();             // of the current device
bool device_ok();           // the current device is an sm_103

}  // namespace lrm
