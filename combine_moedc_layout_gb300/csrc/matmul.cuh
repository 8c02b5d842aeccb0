// What the products of packed expert rows with 16-bit or e4m3 weights share: arguments
// and units of work.
#pragma once

#include <climits>

#include "lm_common.cuh"

namespace moedc {

// out = x W^T, dx = dout W (of matmul_pair.cu)
enum MmMode { kMmForward, kMmDx };

struct MmArgs {
    int E;
    int N;              // columns of the output (with `gated`, of each of the two products)
    int K;              // elements of a row of x that a product adds up 
    int M;              // dW: rows of the output
    int rows, x_rows;
    int slots;          // rows of an expert's slots where there are no offsets
    int top_k;
    const int32_t *offsets, *counts, *src;
    bool packed;        // e4m3: src has been followed, x holds `rows` rows in packed order
    int32_t* status;
    // e4m3: scale of row r (row i of expert e's slots) and channels 128 g ..: xs[r * xs_r +
    // g * xs_g] (xs[e * xs_e + i * xs_r + g * xs_g]); ws [E][1 or 2][blocks][K / 128]
    const float *xs, *ws;
    int64_t xs_e, xs_r, xs_g;
    void* out;
    void* extra;        // gated: both products; the codes' scales (e4m3)
    bool gated, f16;    // f16: 16-bit outputs are f16 (else bf16)
    bool f32;           // dW: binary32 output
    bool codes;         // e4m3 output
    bool vec;           // 16-byte stores fit the output
    unsigned wait_extra;
};

// First and last row of an expert, inside [0, rows].
__device__ __forceinline__ void mm_expert_rows(const MmArgs& a, int e, int& beg, int& end, bool& over)
{
    int64_t b = a.offsets ? __ldg(a.offsets + e) : (int64_t)e * a.slots;
    const int64_t most = a.offsets ? a.rows : b + a.slots;
    int64_t n = b + (a.counts ? __ldg(a.counts + e) : a.rows);
    if (b < 0) b = 0;
    if (n > most) {
        n = most;
        over = true;
    }
    beg = (int)(b < n ? b : 0);
    end = (int)(b < n ? n : 0);
}

// Row of x, as the caller has it, of packed row r; -1 where there is none.
__device__ __forceinline__ int mm_x_row(const MmArgs& a, int r)
{
    if (!a.src) return r;
    const int i = __ldg(a.src + r);
    const int t = i < 0 ? -1 : i / a.top_k;
    return t < a.x_rows ? t : -1;
}

// -0: of packed rows that src led outside of x
constexpr uint32_t kMmLostScale = 0x80000000u;

// silu(g) u.  exp(-|g|) does not overflow, so that the sigmoid goes down to the smallest
// binary32 numbers; the quotient, of numbers between 1 and 2, is the fast one of two ulps.
__device__ __forceinline__ float mm_silu_mul(float g, float u)
{
    const float e = expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + e);
    return g * (g < 0.0f ? e * r : r) * u;
}

// By the whole block: the rows of every expert, and the chunks of chunk_rows rows of the
// experts before each one.  True for a thread that saw an expert pass the end of its rows
// (or more units than there are numbers: none are left then).  Ends with a barrier.
template <int kThreads>
__device__ __forceinline__ bool mm_chunks(const MmArgs& a, int chunk_rows, int tiles, int64_t* s_scan, int32_t* s_pre,
                                          int32_t* s_beg, int32_t* s_end)
{
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    bool over = false;
    const int per = (a.E + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per;
    int64_t sum = 0;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
        int beg, end;
        mm_expert_rows(a, e, beg, end, over);
        const int c = (end - beg) / chunk_rows + ((end - beg) % chunk_rows != 0);
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

// Order of an expert's units: eight tiles of columns for one chunk of rows, for the next
// chunk, then the next eight.  What is written at one time lies together in the rows of the
// output (chunk after chunk for one tile: 167 us against 147 for 8192 x 4096 x 4096), and
// operands of both sides are in L2 for their next use.
constexpr int kMmTogether = 8;
__device__ __forceinline__ void mm_order(int in, int tiles, int chunks, int& tile, int& chunk)
{
    const int group = in / (kMmTogether * chunks), rest = in - group * (kMmTogether * chunks);
    const int width = min(kMmTogether, tiles - group * kMmTogether);
    chunk = rest / width;
    tile = group * kMmTogether + rest - chunk * width;
}

}  // namespace moedc

namespace moedc_host {

// By pairs of SMs (matmul_pair.cu, matmul_dw.cu).  Leading dimensions in elements.
int launch_mm_forward(const moedc::MmArgs& a, const void* x, int64_t ldx, const void* w, cudaStream_t stream);
int launch_mm_dx(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* w, cudaStream_t stream);
int launch_mm_dw(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* x, int64_t ldx, cudaStream_t stream);
// e4m3, by single SMs: the tokens on the tile's rows (matmul_rows.cu), no src
int launch_mm_rows(const moedc::MmArgs& a, const void* x, const void* w, cudaStream_t stream);
// the weights on the tile's rows (matmul_stream.cu): few rows to an expert.  share: blocks may
// share a tile's channels, which changes the order of the sums
int launch_mm_stream(const moedc::MmArgs& a, const void* x, const void* w, bool share, cudaStream_t stream);

}  // namespace moedc_host
