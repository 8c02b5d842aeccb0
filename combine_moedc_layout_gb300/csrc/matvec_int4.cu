// Products of packed expert rows with 4-bit weights and group scales:
//   out[r][n] = sum_k x[r'][k] (q[e][n][k] - z[e][n][k/g]) s[e][n][k/g]
// for the expert e whose rows hold r.  Each warp owns one output channel of
// one expert (with SwiGLU: a gate row and its up row) and walks the expert's
// rows four at a time, so that a weight is unpacked once for four rows.
#include <climits>

#include "lm_common.cuh"

namespace moedc {

constexpr int kMvThreads = 256;
constexpr int kMvWarps = kMvThreads / kWarp;
constexpr int kMvRows = 4;

struct MatvecArgs {
    const void* x;
    int64_t ldx;
    int x_rows, Kd;
    const uint8_t* wq;
    const void* scales;
    int scale_dtype;
    const uint8_t* zeros;
    int group, E, N;
    const int32_t *offsets, *counts, *src;
    int top_k, rows;
    int32_t* status;
};

__device__ __forceinline__ float load_scale(const void* s, int dtype, int64_t i)
{
    return dtype == MOEDC_F32   ? __ldg(static_cast<const float*>(s) + i)
           : dtype == MOEDC_F16 ? __half2float(static_cast<const __half*>(s)[i])
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(s)[i]);
}

// The x row of packed row r, or -1 (outside x: read as zero).
__device__ __forceinline__ int64_t x_row(const MatvecArgs& a, int r, bool& bad)
{
    int64_t t = r;
    if (a.src) {
        const int i = __ldg(a.src + r);
        t = i < 0 ? -1 : i / a.top_k;
    }
    if (t >= a.x_rows || t < 0) {
        bad = true;
        return -1;
    }
    return t;
}

template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kMvThreads)
matvec_int4_kernel(MatvecArgs a, T* __restrict__ out)
{
    pdl_enter();
    const int lane = threadIdx.x % kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kMvWarps;
    const int groups = a.Kd / a.group;
    const int wrows = SWIGLU ? 2 * a.N : a.N;
    bool bad = false, over = false;
    for (int64_t it = (int64_t)blockIdx.x * kMvWarps + threadIdx.x / kWarp;
         it < (int64_t)a.E * a.N; it += nwarps) {
        const int e = (int)(it / a.N), n = (int)(it - (int64_t)e * a.N);
        int64_t beg = a.offsets ? __ldg(a.offsets + e) : 0;
        int64_t end = beg + (a.counts ? __ldg(a.counts + e) : a.rows);
        if (beg < 0) beg = 0;
        if (end > a.rows) {
            end = a.rows;
            over = true;
        }
        for (int64_t r0 = beg; r0 < end; r0 += kMvRows) {
            const T* xr[kMvRows];
#pragma unroll
            for (int i = 0; i < kMvRows; ++i) {
                const int64_t t = r0 + i < end ? x_row(a, (int)(r0 + i), bad) : -1;
                xr[i] = t >= 0 ? static_cast<const T*>(a.x) + t * a.ldx : nullptr;
            }
            float acc[2][kMvRows] = {};
#pragma unroll
            for (int half = 0; half < (SWIGLU ? 2 : 1); ++half) {
                const int64_t wrow = (int64_t)e * wrows + n + (half ? a.N : 0);
                for (int k = lane * 8; k < a.Kd; k += kWarp * 8) {
                    const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(
                        a.wq + wrow * (a.Kd / 2) + k / 2));
                    const int64_t g = wrow * groups + k / a.group;
                    const float s = load_scale(a.scales, a.scale_dtype, g);
                    const float z = a.zeros ? (float)__ldg(a.zeros + g) : 8.0f;
                    float w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = ((float)((q >> (4 * j)) & 15u) - z) * s;
#pragma unroll
                    for (int i = 0; i < kMvRows; ++i) {
                        if (!xr[i]) continue;
                        const Pack<T, 8> v = *reinterpret_cast<const Pack<T, 8>*>(xr[i] + k);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[half][i] = fmaf(w[j], to_f32(v.v[j]), acc[half][i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kMvRows; ++i) {
                float v = warp_sum(acc[0][i]);
                if (SWIGLU) {
                    const float b = warp_sum(acc[1][i]);
                    v = v / (1.0f + expf(-v)) * b;
                }
                if (lane == 0 && r0 + i < end) out[(r0 + i) * a.N + n] = from_f32<T>(v);
            }
        }
    }
    if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    if (over) raise_status(a.status, MOEDC_ERR_CAPACITY);
}

}  // namespace moedc

namespace moedc_host {
namespace {

template <typename T, bool SWIGLU>
int launch_matvec(const moedc::MatvecArgs& a, void* out, cudaStream_t stream)
{
    auto* k = moedc::matvec_int4_kernel<T, SWIGLU>;
    const int64_t want = ((int64_t)a.E * a.N + moedc::kMvWarps - 1) / moedc::kMvWarps;
    const int64_t most = resident_blocks((const void*)k, moedc::kMvThreads, 0);
    clear_stale_error();
    launch(k, (int)(want < most ? want : most), moedc::kMvThreads, 0, stream, a,
           static_cast<T*>(out));
    return launch_status();
}

}  // namespace
}  // namespace moedc_host

extern "C" int moedc_matvec_int4(const void* x, int64_t ldx, int dtype, int x_rows, int Kd,
                                 const void* wq, const void* scales, int scale_dtype,
                                 const uint8_t* zeros, int group, int E, int N, int flags,
                                 const int32_t* offsets, const int32_t* counts,
                                 const int32_t* src, int top_k, int rows, void* out,
                                 int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    if ((dtype != MOEDC_BF16 && dtype != MOEDC_F16) || !lm_dtype_ok(scale_dtype)) return MOEDC_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return MOEDC_ERR_ARG;
    if (Kd < group || Kd % group != 0 || E < 1 || E > MOEDC_MAX_E || N < 1 || x_rows < 0 ||
        rows < 0 || (flags & ~MOEDC_SWIGLU) != 0 || (flags && N > INT32_MAX / 2))
        return MOEDC_ERR_ARG;
    if ((offsets == nullptr) != (counts == nullptr) || (!offsets && E != 1)) return MOEDC_ERR_ARG;
    if (src && top_k < 1) return MOEDC_ERR_ARG;
    if (!wq || !scales || !dev_status || ldx < Kd || ldx % 8 != 0) return MOEDC_ERR_ARG;
    if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(scales, lm_dtype_size(scale_dtype)) ||
        !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(src, 4) || !aligned(out, 2) ||
        !aligned(dev_status, 4))
        return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!out || (x_rows > 0 && !x)) return MOEDC_ERR_ARG;
    const moedc::MatvecArgs a{x, ldx, x_rows, Kd, static_cast<const uint8_t*>(wq), scales,
                              scale_dtype, zeros, group, E, N, offsets, counts, src, top_k, rows,
                              dev_status};
    const bool swiglu = (flags & MOEDC_SWIGLU) != 0;
    if (dtype == MOEDC_F16)
        return swiglu ? launch_matvec<__half, true>(a, out, stream)
                      : launch_matvec<__half, false>(a, out, stream);
    return swiglu ? launch_matvec<__nv_bfloat16, true>(a, out, stream)
                  : launch_matvec<__nv_bfloat16, false>(a, out, stream);
}
