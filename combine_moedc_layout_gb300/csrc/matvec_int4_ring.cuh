// What the two ring kernels of the 4-bit expert products share: the records of x,
// scales in registers, the weights' tensor map.
#pragma once

#include <type_traits>

#include "matvec_int4.cuh"
#include "mbarrier.cuh"
#include "tensor_map.cuh"

namespace moedc {

constexpr int kMvChunk = 256;                          // channels of a stage (of one part of K)
// A record of x: 256 channels in f16, then (16-byte aligned, for TMA) 2^12 / scale.
// 576 bytes apart, the rows that a quarter-warp reads lie in different halves of the
// banks.
constexpr int kMvRecord = kMvChunk * 2 + 64;
constexpr int kMvFactor = kMvChunk * 2 + 32;

// Scales and zero points of R weight rows for one stage, in registers as they come
// from memory.
template <int GROUP, typename S, int R> struct MvScales {
    static constexpr int n = kMvChunk / GROUP;                 // groups
    static constexpr int words = n * (int)sizeof(S) / 4;
    static constexpr int zwords = n == 8 ? 2 : 1;
    uint32_t s[R][words];
    uint32_t z[R][zwords];

    static __device__ __forceinline__ void load_row(uint32_t (&s)[words], const S* p, bool whole, int have)
    {
        if (whole) {
            if constexpr (words == 1) {
                s[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            } else if constexpr (words == 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                s[0] = v.x, s[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < words / 4; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
                    s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
                }
            }
        } else if constexpr (sizeof(S) == 4) {
#pragma unroll
            for (int i = 0; i < n; ++i) s[i] = __float_as_uint(__ldg(reinterpret_cast<const float*>(p) + min(i, have - 1)));
        } else {
#pragma unroll
            for (int i = 0; i < n; i += 2) {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
                s[i / 2] = (uint32_t)__ldg(h + min(i, have - 1)) | (uint32_t)__ldg(h + min(i + 1, have - 1)) << 16;
            }
        }
    }
    static __device__ __forceinline__ void load_zeros(uint32_t (&z)[zwords], const uint8_t* p, bool whole, int have)
    {
        if (whole) {
            if constexpr (n == 2) {
                z[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
            } else if constexpr (n == 4) {
                z[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
                z[0] = v.x, z[1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < zwords; ++i) z[i] = 0;
#pragma unroll
            for (int i = 0; i < n; ++i) z[i / 4] |= (uint32_t)__ldg(p + min(i, have - 1)) << (8 * (i % 4));
        }
    }
    // Of a unit's rows: where their scales and zero points begin.  Without zero
    // points z stays 8.
    struct Rows {
        const S* s[R];
        const uint8_t* z[R];
    };
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < zwords; ++i) z[r][i] = 0x08080808u;
    }
    // the groups from q on; `have` of them exist (all, where they come as one load)
    __device__ __forceinline__ void load(const Rows& rows, int q, int have, bool whole, bool zeros)
    {
        // written out: as a loop the compiler spills more (490 against 462 us in the warp
        // tiles' largest case)
        static_assert(R <= 2);
        load_row(s[0], rows.s[0] + q, whole, have);
        if constexpr (R == 2) load_row(s[1], rows.s[1] + q, whole, have);
        if (zeros) {
            load_zeros(z[0], rows.z[0] + q, whole, have);
            if constexpr (R == 2) load_zeros(z[1], rows.z[1] + q, whole, have);
        }
    }
    // whether a row's groups of a stage are one aligned load
    static __device__ __forceinline__ bool aligned_groups(const MatvecArgs& a, int groups)
    {
        constexpr int bytes = n * (int)sizeof(S) < 16 ? n * (int)sizeof(S) : 16;
        return groups % n == 0 && reinterpret_cast<uintptr_t>(a.scales) % bytes == 0 &&
               reinterpret_cast<uintptr_t>(a.zeros) % n == 0;
    }
    __device__ __forceinline__ float scale(int row, int q) const
    {
        if constexpr (sizeof(S) == 4) {
            return __uint_as_float(s[row][q]);
        } else {
            const uint32_t w = s[row][q / 2];
            if constexpr (std::is_same<S, __nv_bfloat16>::value)
                return __uint_as_float(q % 2 ? w & 0xffff0000u : w << 16);
            else
                return __half2float(__ushort_as_half((unsigned short)(q % 2 ? w >> 16 : w & 0xffffu)));
        }
    }
    // the zero point as the weights' f16 subnormals, of the low nibbles
    __device__ __forceinline__ uint32_t zero_f16(int row, int q) const
    {
        return ((z[row][q / 4] >> (8 * (q % 4))) & 0xffu) * 0x00010001u;
    }
};

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

}  // namespace moedc

namespace moedc_host {

constexpr int kMvSmem = 227 * 1024;

// Rows of Kd / 2 bytes, boxes of box_rows x 128 bytes in the 128-byte swizzle.  False
// when the driver refuses.
bool matvec_weight_map(CUtensorMap* map, const void* wq, int Kd, int64_t rows, int box_rows);

// Records of x by packed row, [row][stage]: 64 of their channels in the 128-byte
// swizzle, and 16 bytes of them (the factor) as they are, in boxes of box_rows rows of one stage.
bool matvec_x_maps(CUtensorMap* channels, CUtensorMap* factors, const uint8_t* records, int chunks, int rows, int box_rows);

// matvec_int4_tc.cu: many rows to an expert.  Its records of x are by packed row.
bool matvec_tc_takes(int E, int rows, int group);
int launch_matvec_tc(const moedc::MatvecArgs& a, int group, void* out, cudaStream_t stream);

}  // namespace moedc_host
