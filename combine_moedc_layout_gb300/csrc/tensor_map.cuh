#pragma once

#include <cuda.h>

#include "common.cuh"

namespace moedc {

// One matrix in boxes of four heights: a stage's rows are one copy, as each costs some 200
// clocks beside its bytes.
struct BoxMaps {
    CUtensorMap by[4];
};

}  // namespace moedc

namespace moedc_host {

// A tiled map of `dims` dimensions, the innermost first; stride in bytes, of all but the
// innermost.  Reads outside give zeros.  False when the driver refuses.
bool tensor_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int dims,
                const cuuint64_t* size, const cuuint64_t* stride, const cuuint32_t* box);

// [rows][width] of 16-bit elements, ld elements from row to row, in boxes of 64 elements x
// box_rows in the 128-byte swizzle (matmul_pair.cu).
bool map_rows16(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t ld, int box_rows);

}  // namespace moedc_host
