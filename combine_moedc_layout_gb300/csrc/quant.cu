// Rows or 128 x 128 blocks of bf16, f16 or binary32 to e4m3 codes with binary32 scales, by
// the rule of dispatch: a = max |x|, scale = max(a, 1e-4) / 448, code = e4m3(x / scale).
//
// Bound by HBM: every element is read once and kept in registers between the maximum and
// the codes.  A thread owns 16 neighbouring channels, so that eight lanes hold a group of
// 128 and store 128 bytes of codes; for blocks, 512 threads hold the 128 rows, each of them
// two.  65536 x 7168 bf16 rows: 263 us, 5.4 TB/s; 32800 x 7168 in blocks: 144 us, 4.9 TB/s.  The
// quotients, not HBM, were the bound while each was a division.
#include "quotient.cuh"

namespace moedc {

// 16 channels as they come from memory
template <typename T> struct Quant16 {
    static constexpr int units = (int)sizeof(T);   // of 16 bytes
    static constexpr int per = kVec<T>;
    uint4 u[units];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < units; ++i) u[i] = ld_global_nc(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < units; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ float top() const
    {
        if constexpr (sizeof(T) == 2) {
            // two at a time; the maximum leaves NaN out as fmaxf does
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
            T2 m = __habs2(*reinterpret_cast<const T2*>(w));
#pragma unroll
            for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const T2*>(w + i)));
            // (a 0 for the first one's NaN)
            return fmaxf(fmaxf(0.0f, to_f32(m.x)), to_f32(m.y));
        }
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < units; ++i) {
            float f[per];
            Unit<T, per>::widen(u[i], f);
#pragma unroll
            for (int j = 0; j < per; ++j) t = fmaxf(t, fabsf(f[j]));
        }
        return t;
    }
    __device__ __forceinline__ uint4 codes(float sc) const
    {
        using Q = Quotient<sizeof(T) == 4 ? 2 : 1>;
        const Q by = Q::by(sc);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < units; ++i) {
            float f[per];
            Unit<T, per>::widen(u[i], f);
#pragma unroll
            for (int j = 0; j < per; j += 4)
                q[(i * per + j) / 4] = by.codes(f[j], f[j + 1]) | by.codes(f[j + 2], f[j + 3]) << 16;
        }
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
};

__device__ __forceinline__ float group_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
}

template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, int64_t ld, int64_t rows, int Kd,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    pdl_enter();
    const int per_row = Kd / 16;
    const int64_t n = rows * per_row;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    // n is a multiple of 8: the lanes of a group are in or out together; the loop's bound is
    // the warp's, as the shuffles want all of its lanes
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i - threadIdx.x % kWarp < n; i += step) {
        const int64_t row = i / per_row;
        const int c = (int)(i - row * per_row) * 16;
        Quant16<T> v;
        if (i < n) v.load(x + row * ld + c);
        else v.clear();
        const float sc = __fdiv_rn(fmaxf(group_max(v.top()), 1e-4f), 448.0f);
        if (i < n) {
            *reinterpret_cast<uint4*>(codes + row * Kd + c) = v.codes(sc);
            if (threadIdx.x % 8 == 0) scales[row * (Kd / 128) + c / 128] = sc;
        }
    }
}

constexpr int kQuantBlock = 512;

template <typename T>
__global__ void __launch_bounds__(kQuantBlock, sizeof(T) == 4 ? 2 : 3) quant_blocks_kernel(const T* __restrict__ x, int64_t ld, int64_t blocks, int rows,
                                                           int Kd, uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    pdl_enter();
    constexpr int kRows = kQuantBlock / 8, kEach = 128 / kRows;   // rows at once, of a thread
    __shared__ float s_top[2][kQuantBlock / kWarp];
    const int groups = Kd / 128, down = (rows + 127) / 128;
    int turn = 0;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const int g = (int)(b % groups);
        const int64_t rest = b / groups;
        const int64_t e = rest / down;
        const int r0 = (int)(rest - e * down) * 128 + threadIdx.x / 8;
        const int c = g * 128 + threadIdx.x % 8 * 16;
        Quant16<T> v[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (r0 + kRows * i < rows) v[i].load(x + (e * rows + r0 + kRows * i) * ld + c);
            else v[i].clear();
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) top = fmaxf(top, v[i].top());
        top = warp_max(top);
        // two sets in turn: a warp may be at the next block while another reads this one's
        if (threadIdx.x % kWarp == 0) s_top[turn][threadIdx.x / kWarp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQuantBlock / kWarp; ++w) top = fmaxf(top, s_top[turn][w]);
        const float sc = __fdiv_rn(fmaxf(top, 1e-4f), 448.0f);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (r0 + kRows * i < rows) *reinterpret_cast<uint4*>(codes + (e * rows + r0 + kRows * i) * Kd + c) = v[i].codes(sc);
        if (threadIdx.x == 0) scales[b] = sc;
    }
}

}  // namespace moedc

namespace moedc_host {
namespace {

template <typename T>
void launch_quant(const void* x, int64_t ld, int E, int rows, int Kd, int block_rows, void* codes, float* scales,
                  cudaStream_t stream)
{
    const T* p = static_cast<const T*>(x);
    const int64_t sms = sm_count();
    if (block_rows == 1) {
        const int64_t all = (int64_t)E * rows, want = (all * (Kd / 16) + 255) / 256, most = 32 * sms;
        launch(moedc::quant_rows_kernel<T>, (int)(want < most ? want : most), 256, 0, stream, p, ld, all, Kd,
               static_cast<uint8_t*>(codes), scales);
    } else {
        const int64_t blocks = (int64_t)E * ((rows + 127) / 128) * (Kd / 128), most = 16 * sms;
        launch(moedc::quant_blocks_kernel<T>, (int)(blocks < most ? blocks : most), moedc::kQuantBlock, 0, stream, p, ld, blocks, rows, Kd,
               static_cast<uint8_t*>(codes), scales);
    }
}

}  // namespace
}  // namespace moedc_host

extern "C" int moedc_quant_e4m3(const void* x, int64_t ldx, int dtype, int E, int rows, int Kd, int block_rows, void* codes,
                                float* scales, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!lm_dtype_ok(dtype) || E < 1 || rows < 0 || Kd < 128 || Kd % 128 != 0 || (block_rows != 1 && block_rows != 128) ||
        ldx < Kd || ldx % (16 / lm_dtype_size(dtype)) != 0 || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!x || !codes || !scales) return MOEDC_ERR_ARG;
    clear_stale_error();
    if (dtype == MOEDC_F32) launch_quant<float>(x, ldx, E, rows, Kd, block_rows, codes, scales, stream);
    else if (dtype == MOEDC_F16) launch_quant<__half>(x, ldx, E, rows, Kd, block_rows, codes, scales, stream);
    else launch_quant<__nv_bfloat16>(x, ldx, E, rows, Kd, block_rows, codes, scales, stream);
    return launch_status();
}
