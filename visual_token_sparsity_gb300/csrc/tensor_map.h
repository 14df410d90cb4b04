// The driver's encoder of TMA tensor maps, looked up once (salience.cu).
#pragma once

#include <cuda.h>

namespace sv {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// nullptr when the driver has none
EncodeTiledFn tensor_map_encoder();

}  // namespace sv
