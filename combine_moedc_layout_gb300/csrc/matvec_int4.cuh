// What the kernels of the 4-bit expert products share: arguments and units of
// work.
#pragma once

#include <climits>

#include "lm_common.cuh"

namespace moedc {

struct MatvecArgs {
    const void* x;
    int64_t ldx;
    int x_rows, Kd;
    const uint8_t* wq;
    const void* scales;
    int scale_dtype;
    const uint8_t* zeros;
    int E, N;
    const int32_t *offsets, *counts, *src;
    int top_k, rows;
    int32_t* status;
    bool swiglu, f16;   // f16: the type of the outputs (else bf16)
    // of the kernel with prepared x:
    const uint8_t* records;   // [x_rows + 1][channels / 256], the last row zeros
    int lk;             // log2 of the parts of K
    int chunk_rows;     // rows of a unit, at most: 8, 16 or 32
    int stages, stage_bytes;
    unsigned wait_extra;
};

// Rows [r0, r0 + m) of expert e and the tile's first output channel.
struct MvUnit {
    int e, n0, r0, m;
};

// First and last row of an expert, inside [0, rows].
__device__ __forceinline__ void expert_rows(const MatvecArgs& a, int e, int& beg, int& end,
                                            bool& over)
{
    int64_t b = a.offsets ? __ldg(a.offsets + e) : 0;
    int64_t n = b + (a.counts ? __ldg(a.counts + e) : a.rows);
    if (b < 0) b = 0;
    if (n > a.rows) {
        n = a.rows;
        over = true;
    }
    beg = (int)(b < n ? b : 0);
    end = (int)(b < n ? n : 0);
}

// s_pre[e]: chunks of the experts before e; s_beg[e], s_end[e]: its rows
__device__ __forceinline__ MvUnit mv_unit(const MatvecArgs& a, const int32_t* s_pre,
                                          const int32_t* s_beg, const int32_t* s_end, int tiles,
                                          int tile_n, int unit)
{
    int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (s_pre[mid] * tiles <= unit) lo = mid; else hi = mid - 1;
    }
    const int chunks = s_pre[lo + 1] - s_pre[lo];
    const int in = unit - s_pre[lo] * tiles;
    const int tile = in / chunks, chunk = in - tile * chunks;   // chunks of one tile are neighbours
    MvUnit u;
    u.e = lo;
    u.n0 = tile * tile_n;
    u.r0 = s_beg[lo] + chunk * a.chunk_rows;
    u.m = min(a.chunk_rows, s_end[lo] - u.r0);
    return u;
}

// The x row of packed row r; the row of zeros where there is none.
__device__ __forceinline__ int x_row(const MatvecArgs& a, int r, bool& bad)
{
    int t = r;
    if (a.src) {
        const int i = __ldg(a.src + r);
        t = i < 0 ? -1 : i / a.top_k;
    }
    if (t >= 0 && t < a.x_rows) return t;
    bad = true;
    return a.x_rows;
}

__device__ __forceinline__ void store16(uint16_t* p, float v, bool f16)
{
    *p = f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// By the whole block: the rows of every expert, and the chunks of the experts
// before each one.  True for a thread that saw an expert pass the end of the rows
// (or more units than there are numbers: none are left then).
template <int kThreads>
__device__ __forceinline__ bool mv_chunks(const MatvecArgs& a, int tiles, int64_t* s_scan, int32_t* s_pre,
                                          int32_t* s_beg, int32_t* s_end)
{
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    bool over = false;
    const int per = (a.E + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per;
    int64_t sum = 0;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
        int beg, end;
        expert_rows(a, e, beg, end, over);
        const int c = (end - beg) / a.chunk_rows + ((end - beg) % a.chunk_rows != 0);
        s_beg[e] = beg;
        s_end[e] = end;
        s_pre[e] = c;
        sum += c;
    }
    int64_t incl = sum;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == kWarp - 1) s_scan[warp] = incl;
    __syncthreads();
    int64_t base = incl - sum;
    for (int w = 0; w < warp; ++w) base += s_scan[w];
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
        const int c = s_pre[e];
        s_pre[e] = (int)base;
        base += c;
    }
    if (e0 < a.E && e0 + per >= a.E) {
        const bool fits = base * tiles <= INT_MAX;
        s_pre[a.E] = fits ? (int)base : 0;
        over |= !fits;
    }
    __syncthreads();
    return over;
}

}  // namespace moedc

namespace moedc_host {

// matvec_int4_small.cu: one launch, nothing prepared
bool matvec_small_takes(int Kd, int E, int N, bool swiglu, int rows);
int launch_matvec_small(const moedc::MatvecArgs& a, int group, void* out, cudaStream_t stream);

}  // namespace moedc_host
