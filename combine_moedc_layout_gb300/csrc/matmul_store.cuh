// Stores of the epilogues whose threads own a row of the output each.
#pragma once

#include "matmul.cuh"

namespace moedc {

__device__ __forceinline__ uint32_t mm_pack16(float lo, float hi, bool f16)
{
    if (!f16) return pack_bf16x2(lo, hi);
    return (uint32_t)__half_as_ushort(__float2half_rn(lo)) | (uint32_t)__half_as_ushort(__float2half_rn(hi)) << 16;
}

// A warp's 32 rows, 64 bytes of each lane's own one: through shared memory, so that four
// lanes store a row's 64 bytes and no sector is written in halves.  `rows` of them and
// `bytes` (in 16s) of each exist; the first begins at `to`.
__device__ __forceinline__ void mm_store_rows(uint8_t* buf, const uint4 (&q)[4], uint8_t* to, int64_t stride, int rows, int bytes)
{
    const int lane = threadIdx.x % kWarp;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = q[c];
    __syncwarp();
    const int c = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = k * 8 + (lane >> 2);
        const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
        if (r < rows && c * 16 < bytes) *reinterpret_cast<uint4*>(to + r * stride + c * 16) = v;
    }
}

// 32 values of each lane's row from column n on, as far as N, rounded once to 16 bits.
// out: the first row's column 0; vec: 16-byte stores fit.
__device__ __forceinline__ void mm_store32(uint8_t* buf, uint16_t* out, int64_t ld, int n, int N, int rows, bool vec, bool f16,
                                           const float* v)
{
    if (vec) {
        uint4 q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float* f = v + 8 * c;
            q[c] = make_uint4(mm_pack16(f[0], f[1], f16), mm_pack16(f[2], f[3], f16), mm_pack16(f[4], f[5], f16),
                              mm_pack16(f[6], f[7], f16));
        }
        mm_store_rows(buf, q, reinterpret_cast<uint8_t*>(out + n), 2 * ld, rows, 2 * min(N - n, 32));
    } else if ((int)(threadIdx.x % kWarp) < rows) {
        uint16_t* row = out + threadIdx.x % kWarp * ld + n;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (n + j < N) row[j] = (uint16_t)mm_pack16(v[j], 0.0f, f16);
    }
}
__device__ __forceinline__ void mm_store32(uint8_t* buf, float* out, int64_t ld, int n, int N, int rows, const float* v)
{
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        uint4 q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float* f = v + h + 4 * c;
            q[c] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        }
        mm_store_rows(buf, q, reinterpret_cast<uint8_t*>(out + n + h), 4 * ld, rows, 4 * min(N - n - h, 16));
    }
}

}  // namespace moedc
