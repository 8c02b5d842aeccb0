#pragma once

#include <cuda.h>

#include "common.cuh"

namespace moedc_host {

// A tiled map of `dims` dimensions, the innermost first; stride in bytes, of all but the
// innermost.  Reads outside give zeros.  False when the driver refuses.
bool tensor_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int dims,
                const cuuint64_t* size, const cuuint64_t* stride, const cuuint32_t* box);

}  // namespace moedc_host
