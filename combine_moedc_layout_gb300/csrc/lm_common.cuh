// Element types of the language-model operators (router, sorted rows, 4-bit
// products): bf16, f16 or binary32 in memory, binary32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace moedc {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// one rounding, to nearest even
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// V consecutive elements: one 16-byte access (V = 16 / sizeof(T)) or one element
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

// One access of V elements as it moves through registers: 16 bytes, or one
// element.  Kept as words: arrays of the 16-bit classes end up in local memory.
template <typename T, int V> struct Unit {
    static_assert(V * sizeof(T) == 16, "a unit is 16 bytes or one element");
    using Raw = uint4;
    static __device__ __forceinline__ void widen(const Raw& r, float (&f)[V])
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                f[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xffffu)));
                f[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
            } else {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
    static __device__ __forceinline__ Raw round(const float (&f)[V])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else if constexpr (std::is_same<T, __half>::value)
                w[i] = (uint32_t)__half_as_ushort(__float2half_rn(f[2 * i])) |
                       (uint32_t)__half_as_ushort(__float2half_rn(f[2 * i + 1])) << 16;
            else
                w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <typename T> struct Unit<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ void widen(const Raw& r, float (&f)[1]) { f[0] = to_f32(r); }
    static __device__ __forceinline__ Raw round(const float (&f)[1]) { return from_f32<T>(f[0]); }
};

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

}  // namespace moedc

namespace moedc_host {

inline bool lm_dtype_ok(int d) { return d == MOEDC_BF16 || d == MOEDC_F16 || d == MOEDC_F32; }
inline int lm_dtype_size(int d) { return d == MOEDC_F32 ? 4 : 2; }

}  // namespace moedc_host
