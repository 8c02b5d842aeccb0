// The pair kernel's 16-bit forms: forward, gradient of the rows, gradient of the weights.
#include "matmul_pair.cuh"
#include "tensor_map.cuh"

namespace moedc_host {
namespace {

constexpr CUtensorMapDataType k16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
constexpr CUtensorMapSwizzle kSwizzle = CU_TENSOR_MAP_SWIZZLE_128B;

// [rows][width] with ld elements from row to row, boxes of 64 elements x box_rows
bool map_rows(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t ld, int box_rows)
{
    const cuuint64_t size[2] = {(cuuint64_t)width, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return tensor_map(map, k16, kSwizzle, base, 2, size, stride, box);
}

int64_t col_tiles(const moedc::MmArgs& a)
{
    const int tile = a.gated ? moedc::kMmHalf : moedc::kMmTile;
    return (a.N + (int64_t)tile - 1) / tile;
}
int64_t most_units(const moedc::MmArgs& a)
{
    return ((int64_t)a.rows / moedc::kMmTile + (a.E < a.rows ? a.E : a.rows)) * col_tiles(a);
}

}  // namespace

int launch_mm_forward(const moedc::MmArgs& a, const void* x, int64_t ldx, const void* w, cudaStream_t stream)
{
    CUtensorMap l, r, all;   // left in boxes of 32 rows and of 128
    const cuuint64_t K = a.K, N = a.N, parts = a.gated ? 2 : 1;
    const cuuint64_t size[4] = {K, N, parts, (cuuint64_t)a.E}, stride[3] = {2 * K, 2 * K * N, 2 * K * N * parts};
    const cuuint32_t box[4] = {64, moedc::kMmHalf, 1, 1};
    if (!map_rows(&l, x, a.K, a.rows, ldx, 32) || !map_rows(&all, x, a.K, a.rows, ldx, moedc::kMmHalf) ||
         !tensor_map(&r, k16, kSwizzle, w, 4, size, stride, box))
        return MOEDC_ERR_CUDA;
    return launch_mm_pair<moedc::kMmForward>(a, most_units(a), l, r, all, stream);
}

int launch_mm_dx(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* w, cudaStream_t stream)
{
    CUtensorMap l, r, all;   // left in boxes of 32 rows and of 128
    const cuuint64_t size[3] = {(cuuint64_t)a.N, (cuuint64_t)a.K, (cuuint64_t)a.E};
    const cuuint64_t stride[2] = {2 * (cuuint64_t)a.N, 2 * (cuuint64_t)a.N * a.K};
    const cuuint32_t box[3] = {64, 64, 1};
    if (!map_rows(&l, dout, a.K, a.rows, ldd, 32) || !map_rows(&all, dout, a.K, a.rows, ldd, moedc::kMmHalf) ||
         !tensor_map(&r, k16, kSwizzle, w, 3, size, stride, box))
        return MOEDC_ERR_CUDA;
    return launch_mm_pair<moedc::kMmDx>(a, most_units(a), l, r, all, stream);
}

int launch_mm_dw(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* x, int64_t ldx, cudaStream_t stream)
{
    CUtensorMap l, r;
    if (!map_rows(&l, dout, a.M, a.rows, ldd, 64) || !map_rows(&r, x, a.N, a.rows, ldx, 64)) return MOEDC_ERR_CUDA;
    const int64_t units = a.E * col_tiles(a) * ((a.M + (int64_t)moedc::kMmTile - 1) / moedc::kMmTile);
    return launch_mm_pair<moedc::kMmDw>(a, units, l, r, l, stream);
}

}  // namespace moedc_host
