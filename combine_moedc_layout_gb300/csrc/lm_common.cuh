// Element types of the language-model operators (router, sorted rows, 4-bit
// products): bf16, f16 or binary32 in memory, binary32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
