// Token rows sorted by expert into one packed buffer, the weighted way back,
// and their gradients.
//
// With row[t][k] the packed row of entry (t, k):
//   sort         rows[row[t][k]] = x[t]
//   unsort       y[t] = sum_k w[t][k] rows[row[t][k]]   (w = 1: sort's gradient)
//   unsort_grad  drows[row[t][k]] = w[t][k] dy[t],  dw[t][k] = <dy[t], rows[row[t][k]]>
// All four move rows: HBM traffic bounds them.  4096 tokens, top 8 of 256 experts, 7168
// channels in bf16: sort 92 us by itself (under the counts before it, which it
// overlaps, 183 us with unsort), unsort 77-79 us (529 MB, 6.7 TB/s), unsort_grad
// 148-161 us (998 MB).
#include <climits>

#include "block_layout.cuh"
#include "lm_common.cuh"

namespace moedc {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / kWarp;

// Exclusive prefix over the experts of the aligned counts (s_off[0..E]) and of
// the padding before each group (s_pad[0..E]: padding rows of the groups
// before it), by one warp over the counts in shared memory.  Counts are clamped
// to [0, rows] and the sums saturate at `rows`, so that no count, whatever it
// holds, leads out of the buffer.
__device__ __forceinline__ void group_offsets(int E, int align, int rows, int32_t* s_off,
                                              int32_t* s_pad, const int32_t* s_cnt)
{
    if (threadIdx.x < kWarp) {
        const int lane = threadIdx.x;
        int64_t off = 0, live = 0;
        for (int e0 = 0; e0 < E; e0 += kWarp) {
            const int e = e0 + lane;
            const int64_t c = e < E ? s_cnt[e] : 0;
            const int64_t a = (c + align - 1) / align * align;
            int64_t ia = a, ic = c;
#pragma unroll
            for (int d = 1; d < kWarp; d <<= 1) {
                const int64_t ya = __shfl_up_sync(0xffffffffu, ia, d);
                const int64_t yc = __shfl_up_sync(0xffffffffu, ic, d);
                if (lane >= d) { ia += ya; ic += yc; }
            }
            if (e < E) {
                const int64_t o = off + ia - a, l = live + ic - c;
                s_off[e] = (int)min(o, (int64_t)rows);
                s_pad[e] = (int)min(o - l, (int64_t)rows);
            }
            off += __shfl_sync(0xffffffffu, ia, kWarp - 1);
            live += __shfl_sync(0xffffffffu, ic, kWarp - 1);
        }
        if (lane == 0) {
            s_off[E] = (int)min(off, (int64_t)rows);
            s_pad[E] = (int)min(off - live, (int64_t)rows);
        }
    }
    __syncthreads();
}

struct SortArgs {
    int64_t ldx;               // in units
    int units, T, K, E, align, rows;
    int32_t *row, *src, *offsets;
    int32_t* status;
};

// Units of one row that a lane carries at a time.
#ifndef MOEDC_SORT_UNITS
#define MOEDC_SORT_UNITS 4
#endif
constexpr int kSortUnits = MOEDC_SORT_UNITS;

// The entries' rows, once the block's shared memory holds offsets, padding and
// counts: a warp takes (token, slice) items, reads its part of the token's row
// once and writes it to the row of each entry; then the rows that no entry
// reaches.  route(t, e, s) gives lane k < K the expert and the slot of (t, k).
// U: the unit of one access (16 bytes, or one element where rows are not
// 16-byte multiples).
template <typename U, int kThreads, typename Route>
__device__ __forceinline__ void sort_rows(const SortArgs& a, const U* __restrict__ x,
                                          U* __restrict__ sorted, const int32_t* s_off,
                                          const int32_t* s_pad, const int32_t* s_cnt, Route route)
{
    constexpr int kWarps = kThreads / kWarp;
    const int lane = threadIdx.x % kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kWarps;
    const int64_t warp0 = (int64_t)blockIdx.x * kWarps + threadIdx.x / kWarp;
    const int slices = a.units ? (a.units + kSortUnits * kWarp - 1) / (kSortUnits * kWarp) : 1;
    const int64_t items = (int64_t)a.T * slices;
    bool dropped = false;
    auto load = [&](int64_t it, int& e, int& s, U (&v)[kSortUnits]) {
        e = s = -1;
        if (it >= items) return;
        const int64_t t = it / slices;
        const int u0 = (int)(it - t * slices) * kSortUnits * kWarp + lane;
        if (lane < a.K) route(t, e, s);
#pragma unroll
        for (int j = 0; j < kSortUnits; ++j)
            if (u0 + j * kWarp < a.units) v[j] = __ldg(x + t * a.ldx + u0 + j * kWarp);
    };
    int e, s;
    U v[kSortUnits];
    load(warp0, e, s, v);
    for (int64_t it = warp0; it < items; it += nwarps) {
        // the next item's row travels while this one is stored
        int ne, ns;
        U nv[kSortUnits];
        load(it + nwarps, ne, ns, nv);
        const int64_t t = it / slices;
        const int u0 = (int)(it - t * slices) * kSortUnits * kWarp + lane;
        int r = -1;
        if (e >= 0 && e < a.E && s >= 0) {
            const int64_t at = (int64_t)s_off[e] + s;
            if (at < a.rows) r = (int)at;
            else dropped = true;
        }
        if (u0 == lane && lane < a.K) {
            a.row[t * a.K + lane] = r;
            if (r >= 0) a.src[r] = (int)(t * a.K + lane);
        }
        for (int k = 0; k < a.K; ++k) {
            const int rk = __shfl_sync(0xffffffffu, r, k);
            if (rk < 0) continue;
            U* to = sorted + (int64_t)rk * a.units + u0;
#pragma unroll
            for (int j = 0; j < kSortUnits; ++j)
                if (u0 + j * kWarp < a.units) to[j * kWarp] = v[j];
        }
        e = ne;
        s = ns;
#pragma unroll
        for (int j = 0; j < kSortUnits; ++j) v[j] = nv[j];
    }
    // the rows that no entry reaches: padding of each group, and the tail
    const int64_t live = (int64_t)s_off[a.E] - s_pad[a.E];
    for (int64_t p = warp0; p < a.rows - live; p += nwarps) {
        int lo = 0, hi = a.E;   // last group g with s_pad[g] <= p
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_pad[mid] <= p) lo = mid; else hi = mid - 1;
        }
        const int64_t r = (int64_t)s_off[lo] + (lo < a.E ? s_cnt[lo] : 0) + (p - s_pad[lo]);
        if (r < 0 || r >= a.rows) continue;
        if (lane == 0) a.src[r] = -1;
        U zero{};
        for (int u = lane; u < a.units; u += kWarp) sorted[r * a.units + u] = zero;
    }
    if (dropped) raise_status(a.status, MOEDC_ERR_CAPACITY);
}

constexpr int kSortAhead = 64 << 20;       // bytes of x brought to L2 ahead, at most

// After the layout: slots and counts from memory.
template <typename U>
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(SortArgs a, const U* __restrict__ x, const int32_t* __restrict__ topk_idx,
            const int32_t* __restrict__ slot, const int32_t* __restrict__ counts, U* __restrict__ sorted)
{
    extern __shared__ int32_t s_mem[];   // off [E + 1], pad [E + 1], cnt [E]
    // While the layout runs, the token rows come to L2 (as many as may stay there).  No
    // value is used before the wait.
    if (a.units) {
        const int64_t lines = ((int64_t)a.units * (int)sizeof(U) + 127) / 128;
        const int64_t most = min(a.T * lines, (int64_t)kSortAhead / 128);
        for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < most; i += (int64_t)gridDim.x * kSortThreads) {
            const int64_t t = i / lines;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                reinterpret_cast<const char*>(x + t * a.ldx) + (i - t * lines) * 128));
        }
    }
    pdl_enter();
    int32_t *s_off = s_mem, *s_pad = s_off + a.E + 1, *s_cnt = s_pad + a.E + 1;
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) s_cnt[e] = min(max(__ldg(counts + e), 0), a.rows);
    __syncthreads();
    group_offsets(a.E, a.align, a.rows, s_off, s_pad, s_cnt);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += kSortThreads) a.offsets[e] = s_off[e];
    sort_rows<U, kSortThreads>(a, x, sorted, s_off, s_pad, s_cnt, [&](int64_t t, int& e, int& s) {
        e = __ldg(topk_idx + t * a.K + threadIdx.x % kWarp);
        s = __ldg(slot + t * a.K + threadIdx.x % kWarp);
    });
}

// Up to MOEDC_FUSED_MAX_ENTRIES entries in one launch: every block rebuilds the
// layout in its shared memory, nothing waits on another block.
template <typename U, int kThreads>
__global__ void __launch_bounds__(kThreads)
sort_small_kernel(SortArgs a, const U* __restrict__ x, const int32_t* __restrict__ topk_idx,
                  int32_t* __restrict__ counts, U* __restrict__ sorted)
{
    extern __shared__ int32_t s_mem[];
    pdl_enter();
    const int n = a.T * a.K;
    int32_t *s_off = s_mem, *s_pad = s_off + a.E + 1, *s_cnt = s_pad + a.E + 1;
    int32_t *s_idx = s_cnt + a.E, *s_slot = s_idx + n, *s_wcnt = s_slot + n;
    block_layout<kThreads>(topk_idx, n, a.E, s_idx, s_slot, s_wcnt, s_cnt);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < a.E; e += kThreads) counts[e] = s_cnt[e];
        bool bad = false;
        for (int i = threadIdx.x; i < n; i += kThreads) bad |= s_idx[i] < -1 || s_idx[i] >= a.E;
        if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    }
    // counts of more than `rows` (a buffer that is too small) saturate the offsets
    group_offsets(a.E, a.align, a.rows, s_off, s_pad, s_cnt);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = s_off[e];
    sort_rows<U, kThreads>(a, x, sorted, s_off, s_pad, s_cnt, [&](int64_t t, int& e, int& s) {
        e = s_idx[t * a.K + threadIdx.x % kWarp];
        s = s_slot[t * a.K + threadIdx.x % kWarp];
    });
}

// Packed rows are read once and y is not read again here: no L1 lines for the
// one, no L2 priority for the other (16-byte units).
__device__ __forceinline__ uint4 ld_row(const uint4* p) { return ld_global_nc(p); }
template <typename R> __device__ __forceinline__ R ld_row(const R* p) { return __ldg(p); }
__device__ __forceinline__ void st_row(uint4* p, uint4 v) { st_global_cs(p, v); }
template <typename R> __device__ __forceinline__ void st_row(R* p, R v) { *p = v; }

// Units in flight per lane, over a batch of B rows (as many as K needs, at most 8).
template <int V, int B> constexpr int kUnsortUnits = (V == 1 ? 32 : 16) / B;

// A warp takes (token, slice) items.  The loads of a batch of rows are
// straight-line code (entries without a row read row 0 and are left out of the
// sum), so all of them are in flight together: 4096 tokens, top-8, 7168 channels
// in bf16 take 79 us (6.7 TB/s), 89 us with one row at a time.
template <typename T, int V, int B>
__global__ void __launch_bounds__(kSortThreads, 2)
unsort_kernel(const T* __restrict__ sorted, int rows, int H, const int32_t* __restrict__ row,
              const float* __restrict__ weights, int tokens, int K, T* __restrict__ y)
{
    pdl_enter();
    using P = Unit<T, V>;
    using Raw = typename P::Raw;
    constexpr int kU = kUnsortUnits<V, B>;
    const int lane = threadIdx.x % kWarp;
    const int units = H / V;
    const int slices = (units + kU * kWarp - 1) / (kU * kWarp);
    const int64_t items = (int64_t)tokens * slices;
    const int64_t nwarps = (int64_t)gridDim.x * kSortWarps;
    const Raw* base = reinterpret_cast<const Raw*>(sorted);
    // lane k: the row and the weight of entry k
    auto route = [&](int64_t it, int& r, float& w) {
        r = -1;
        w = 1.0f;
        if (it < items && lane < K) {
            const int64_t i = it / slices * K + lane;
            r = __ldg(row + i);
            if (r >= rows) r = -1;
            if (weights) w = __ldg(weights + i);
        }
    };
    int64_t it = (int64_t)blockIdx.x * kSortWarps + threadIdx.x / kWarp;
    int r;
    float w;
    route(it, r, w);
    for (; it < items; it += nwarps) {
        const int64_t t = it / slices;
        const int u0 = (int)(it - t * slices) * kU * kWarp + lane;
        float acc[kU][V] = {};
        int nr;
        float nw;
        for (int k0 = 0; k0 < K; k0 += B) {
            Raw v[B][kU];
            float wk[B];
            int rk[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                rk[b] = __shfl_sync(0xffffffffu, r, (k0 + b) & 31);
                wk[b] = __shfl_sync(0xffffffffu, w, (k0 + b) & 31);
                if (k0 + b >= K) rk[b] = -1;
            }
            if (rows > 0) {
#pragma unroll
                for (int b = 0; b < B; ++b)
#pragma unroll
                    for (int j = 0; j < kU; ++j) {
                        const int u = u0 + j * kWarp;
                        v[b][j] = ld_row(base + (int64_t)max(rk[b], 0) * units + (u < units ? u : 0));
                    }
            }
            if (k0 == 0) route(it + nwarps, nr, nw);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (rk[b] < 0) continue;
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    float f[V];
                    P::widen(v[b][j], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[j][i] = fmaf(wk[b], f[i], acc[j][i]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            const int u = u0 + j * kWarp;
            if (u >= units) continue;
            st_row(reinterpret_cast<Raw*>(y) + t * units + u, P::round(acc[j]));
        }
        r = nr;
        w = nw;
    }
}

// A block takes entries; dy is read again for each of a token's, from L2.  One
// 16-byte unit at a time keeps 32 registers and 64 warps an SM (two: 48 registers,
// 170 us instead of 148 at 4096 tokens, top-8, 7168 channels in bf16).  The rows that no
// entry reaches are cleared at the end.
template <typename T, int V>
__global__ void __launch_bounds__(kSortThreads, 8)
unsort_grad_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ sorted, int rows,
                   int H, const int32_t* __restrict__ row, const int32_t* __restrict__ src,
                   const float* __restrict__ weights, int tokens, int K, T* __restrict__ dsorted,
                   float* __restrict__ dweights)
{
    __shared__ float s_part[2][kSortWarps];
    pdl_enter();
    using P = Unit<T, V>;
    using Raw = typename P::Raw;
    constexpr int kU = V == 1 ? 4 : 1;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int units = H / V;
    const int64_t entries = (int64_t)tokens * K;
    int turn = 0;
    for (int64_t i = blockIdx.x; i < entries; i += gridDim.x) {
        const int64_t t = i / K;
        const int r = __ldg(row + i);
        const bool ok = r >= 0 && r < rows;
        float dot = 0.0f;
        if (ok) {
            const float w = __ldg(weights + i);
            const Raw* g = reinterpret_cast<const Raw*>(dy + t * lddy);
            const Raw* e = reinterpret_cast<const Raw*>(sorted) + (int64_t)r * units;
            Raw* o = reinterpret_cast<Raw*>(dsorted) + (int64_t)r * units;
            for (int u0 = threadIdx.x; u0 < units; u0 += kU * kSortThreads) {
                Raw d[kU], v[kU];
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    const int u = u0 + j * kSortThreads;
                    if (u < units) {
                        d[j] = __ldg(g + u);
                        if (dweights) v[j] = __ldg(e + u);
                    }
                }
#pragma unroll
                for (int j = 0; j < kU; ++j) {
                    const int u = u0 + j * kSortThreads;
                    if (u >= units) continue;
                    float a[V], b[V];
                    P::widen(d[j], a);
                    if (dweights) {
                        P::widen(v[j], b);
#pragma unroll
                        for (int c = 0; c < V; ++c) dot = fmaf(a[c], b[c], dot);
                    }
#pragma unroll
                    for (int c = 0; c < V; ++c) a[c] *= w;
                    o[u] = P::round(a);
                }
            }
        }
        if (!dweights) continue;
        // one barrier an entry: the partial sums of the next one go to the other half
        dot = warp_sum(dot);
        if (lane == 0) s_part[turn][warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < kSortWarps; ++j) s += s_part[turn][j];
            dweights[i] = ok ? s : 0.0f;
        }
        turn ^= 1;
    }
    const int64_t nwarps = (int64_t)gridDim.x * kSortWarps;
    for (int64_t r = (int64_t)blockIdx.x * kSortWarps + warp; r < rows; r += nwarps) {
        if (__ldg(src + r) >= 0) continue;
        for (int u = lane; u < units; u += kWarp) reinterpret_cast<Raw*>(dsorted)[r * units + u] = Raw{};
    }
}

}  // namespace moedc

namespace moedc_host {
namespace {

int sort_blocks(const void* kernel, size_t smem, int64_t want)
{
    const int64_t most = resident_blocks(kernel, moedc::kSortThreads, smem);
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

// whether rows of H elements at these places can be read 16 bytes at a time
bool rows_vec(int dtype, int H, int64_t ld, const void* a, const void* b, const void* c)
{
    const int v = 16 / lm_dtype_size(dtype);
    return H % v == 0 && ld % v == 0 && aligned(a, 16) && aligned(b, 16) && aligned(c, 16);
}

// the parts of moedc_sort's workspace, each on a 256-byte boundary
struct SortWorkspace {
    size_t slot, in_rank, per_rank, layout, total;
};
SortWorkspace sort_workspace(int T, int K, int E)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    SortWorkspace w;
    w.slot = 0;
    w.in_rank = up((size_t)T * K * sizeof(int32_t));
    w.per_rank = w.in_rank + up((size_t)T);
    w.layout = w.per_rank + 256;
    w.total = w.layout + up(moedc_layout_workspace_bytes(T, K, E, 1));
    return w;
}

template <typename U>
int launch_sort(const moedc::SortArgs& a, const void* x, const int32_t* topk_idx, const int32_t* slot,
                int32_t* counts, void* sorted, cudaStream_t stream)
{
    const U* from = static_cast<const U*>(x);
    U* to = static_cast<U*>(sorted);
    const int per = moedc::kSortUnits * moedc::kWarp;
    // without tokens there are the rows to clear
    const int64_t items = a.T ? (int64_t)a.T * (a.units ? (a.units + per - 1) / per : 1) : a.rows;
    size_t smem = (3 * (size_t)a.E + 2) * sizeof(int32_t);
    clear_stale_error();
    if (!slot) {
        const int n = a.T * a.K;
        const bool narrow = n <= moedc::kFusedNarrow * moedc::kFusedIdsPerThread;
        const int threads = narrow ? moedc::kFusedNarrow : moedc::kFusedWide;
        smem += (2 * (size_t)n + (size_t)(threads / moedc::kWarp) * a.E) * sizeof(int32_t);
        auto* k = narrow ? moedc::sort_small_kernel<U, moedc::kFusedNarrow>
                         : moedc::sort_small_kernel<U, moedc::kFusedWide>;
        // more than the default shared memory needs the limit raised; the layout kernels
        // take such shapes instead
        const int64_t want = (items + threads / moedc::kWarp - 1) / (threads / moedc::kWarp);
        const int64_t most = resident_blocks((const void*)k, threads, smem);
        clear_stale_error();
        launch(k, (int)(want < 1 ? 1 : want < most ? want : most), threads, smem, stream, a, from, topk_idx,
               counts, to);
        return launch_status();
    }
    auto* k = moedc::sort_kernel<U>;
    const int blocks = sort_blocks((const void*)k, smem, (items + moedc::kSortWarps - 1) / moedc::kSortWarps);
    clear_stale_error();
    launch(k, blocks, moedc::kSortThreads, smem, stream, a, from, topk_idx, slot, counts, to);
    return launch_status();
}

// Whether the layout of this shape fits a block of the single launch (its
// default 48 KB of shared memory).
bool sort_small(int T, int K, int E)
{
    const int64_t n = (int64_t)T * K;
    if (n > MOEDC_FUSED_MAX_ENTRIES) return false;
    const int warps = (n <= moedc::kFusedNarrow * moedc::kFusedIdsPerThread ? moedc::kFusedNarrow : moedc::kFusedWide) / moedc::kWarp;
    return ((3 + (size_t)warps) * E + 2 + 2 * (size_t)n) * sizeof(int32_t) <= 48 * 1024;
}

template <typename T, int V, int B>
int launch_unsort(const void* sorted, int rows, int H, const int32_t* row, const float* w,
                  int tokens, int K, void* y, cudaStream_t stream)
{
    auto* k = moedc::unsort_kernel<T, V, B>;
    const int per = moedc::kUnsortUnits<V, B> * moedc::kWarp;
    const int64_t items = (int64_t)tokens * ((H / V + per - 1) / per);
    const int blocks = sort_blocks((const void*)k, 0, (items + moedc::kSortWarps - 1) / moedc::kSortWarps);
    clear_stale_error();
    launch(k, blocks, moedc::kSortThreads, 0, stream, static_cast<const T*>(sorted), rows, H, row,
           w, tokens, K, static_cast<T*>(y));
    return launch_status();
}

template <typename T, int V>
int launch_unsort_k(const void* sorted, int rows, int H, const int32_t* row, const float* w,
                    int tokens, int K, void* y, cudaStream_t stream)
{
    return K <= 2   ? launch_unsort<T, V, 2>(sorted, rows, H, row, w, tokens, K, y, stream)
           : K <= 4 ? launch_unsort<T, V, 4>(sorted, rows, H, row, w, tokens, K, y, stream)
                    : launch_unsort<T, V, 8>(sorted, rows, H, row, w, tokens, K, y, stream);
}

template <typename T, int V>
int launch_unsort_grad(const void* dy, int64_t lddy, const void* sorted, int rows, int H,
                       const int32_t* row, const int32_t* src, const float* w, int tokens, int K,
                       void* dsorted, float* dw, cudaStream_t stream)
{
    auto* k = moedc::unsort_grad_kernel<T, V>;
    const int64_t want = (int64_t)tokens * K > rows ? (int64_t)tokens * K : rows;
    const int blocks = sort_blocks((const void*)k, 0, want);
    clear_stale_error();
    launch(k, blocks, moedc::kSortThreads, 0, stream, static_cast<const T*>(dy), lddy,
           static_cast<const T*>(sorted), rows, H, row, src, w, tokens, K,
           static_cast<T*>(dsorted), dw);
    return launch_status();
}

bool rows_args_ok(int dtype, int T, int H, int K, int rows)
{
    return lm_dtype_ok(dtype) && T >= 0 && H >= 1 && K >= 1 && K <= MOEDC_MAX_K && rows >= 0 &&
           (int64_t)T * K <= INT32_MAX;
}

}  // namespace
}  // namespace moedc_host

extern "C" size_t moedc_sort_rows(int T, int K, int E, int align)
{
    if (!moedc_host::layout_args_ok(T, K, E, 1, 1) || align < 1 || align > MOEDC_SORT_MAX_ALIGN)
        return 0;
    const int64_t n = (int64_t)T * K;
    const int64_t rows = n + (n < E ? n : E) * (int64_t)(align - 1);
    return rows <= INT32_MAX ? (size_t)rows : 0;
}

extern "C" size_t moedc_sort_workspace_bytes(int T, int K, int E)
{
    if (!moedc_host::layout_args_ok(T, K, E, 1, 1)) return 0;
    return moedc_host::sort_workspace(T, K, E).total;
}

extern "C" int moedc_sort(const void* x, int64_t ldx, int dtype, int T, int H,
                          const int32_t* topk_idx, int K, int E, int align, int rows,
                          void* sorted, int32_t* row, int32_t* src, int32_t* offsets,
                          int32_t* counts, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!rows_args_ok(dtype, T, H, K, rows) || !layout_args_ok(T, K, E, 1, 1) || align < 1 ||
        align > MOEDC_SORT_MAX_ALIGN)
        return MOEDC_ERR_ARG;
    if (!offsets || !counts || !dev_status || (rows > 0 && !src)) return MOEDC_ERR_ARG;
    if (T > 0 && (!topk_idx || !row)) return MOEDC_ERR_ARG;
    // x and sorted come together; without them only the maps are made
    if (T > 0 && rows > 0 && (x == nullptr) != (sorted == nullptr)) return MOEDC_ERR_ARG;
    const int size = lm_dtype_size(dtype);
    if ((x && ldx < H) || !aligned(x, size) || !aligned(sorted, size) || !aligned(topk_idx, 4) ||
        !aligned(row, 4) || !aligned(src, 4) || !aligned(offsets, 4) || !aligned(counts, 4) ||
        !aligned(dev_status, 4))
        return MOEDC_ERR_ARG;
    const SortWorkspace ws = sort_workspace(T, K, E);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < ws.total) return MOEDC_ERR_ARG;
    const int32_t* slot = nullptr;
    if (!sort_small(T, K, E)) {
        char* base = static_cast<char*>(workspace);
        int32_t* s = reinterpret_cast<int32_t*>(base + ws.slot);
        const int st = launch_layout(topk_idx, T, K, E, 1, INT32_MAX, counts,
                                     reinterpret_cast<int32_t*>(base + ws.per_rank),
                                     reinterpret_cast<uint8_t*>(base + ws.in_rank), s,
                                     base + ws.layout, ws.total - ws.layout, dev_status, stream);
        if (st != MOEDC_OK) return st;
        slot = s;
    }
    // without `sorted` the maps alone; without tokens every row of it is cleared all the same
    if (!sorted || rows == 0) H = 0;
    moedc::SortArgs a{ldx, H, T, K, E, align, rows, row, src, offsets, dev_status};
    if (rows_vec(dtype, H, x ? ldx : 0, x, sorted, nullptr)) {
        a.ldx = ldx * size / 16;
        a.units = H * size / 16;
        return launch_sort<uint4>(a, x, topk_idx, slot, counts, sorted, stream);
    }
    return size == 4 ? launch_sort<uint32_t>(a, x, topk_idx, slot, counts, sorted, stream)
                     : launch_sort<uint16_t>(a, x, topk_idx, slot, counts, sorted, stream);
}

extern "C" int moedc_unsort(const void* sorted, int dtype, int rows, int H, const int32_t* row,
                            const float* topk_weights, int T, int K, void* y, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!rows_args_ok(dtype, T, H, K, rows)) return MOEDC_ERR_ARG;
    const int size = lm_dtype_size(dtype);
    if (!aligned(sorted, size) || !aligned(y, size) || !aligned(row, 4) || !aligned(topk_weights, 4))
        return MOEDC_ERR_ARG;
    if (T == 0) return MOEDC_OK;
    if ((rows > 0 && !sorted) || !row || !y) return MOEDC_ERR_ARG;
    const bool vec = rows_vec(dtype, H, 0, sorted, y, nullptr);
#define MOEDC_UNSORT(T_) \
    (vec ? launch_unsort_k<T_, moedc::kVec<T_>>(sorted, rows, H, row, topk_weights, T, K, y, stream) \
         : launch_unsort_k<T_, 1>(sorted, rows, H, row, topk_weights, T, K, y, stream))
    return dtype == MOEDC_F32   ? MOEDC_UNSORT(float)
           : dtype == MOEDC_F16 ? MOEDC_UNSORT(__half)
                                : MOEDC_UNSORT(__nv_bfloat16);
#undef MOEDC_UNSORT
}

extern "C" int moedc_unsort_grad(const void* dy, int64_t lddy, const void* sorted, int dtype,
                                 int T, int H, int K, const int32_t* row, const int32_t* src,
                                 const float* topk_weights, int rows, void* dsorted,
                                 float* dweights, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!rows_args_ok(dtype, T, H, K, rows) || lddy < H) return MOEDC_ERR_ARG;
    const int size = lm_dtype_size(dtype);
    if (!aligned(dy, size) || !aligned(sorted, size) || !aligned(dsorted, size) ||
        !aligned(row, 4) || !aligned(src, 4) || !aligned(topk_weights, 4) || !aligned(dweights, 4))
        return MOEDC_ERR_ARG;
    if (rows > 0 && (!src || !dsorted || (dweights && !sorted))) return MOEDC_ERR_ARG;
    if (T > 0 && (!dy || !row || !topk_weights)) return MOEDC_ERR_ARG;
    if (T == 0 && rows == 0) return MOEDC_OK;
    const bool vec = rows_vec(dtype, H, lddy, dy, sorted, dsorted);
#define MOEDC_UNSORT_GRAD(T_)                                                                   \
    (vec ? launch_unsort_grad<T_, moedc::kVec<T_>>(dy, lddy, sorted, rows, H, row, src,         \
                                                   topk_weights, T, K, dsorted, dweights, stream) \
         : launch_unsort_grad<T_, 1>(dy, lddy, sorted, rows, H, row, src, topk_weights, T, K,   \
                                     dsorted, dweights, stream))
    return dtype == MOEDC_F32   ? MOEDC_UNSORT_GRAD(float)
           : dtype == MOEDC_F16 ? MOEDC_UNSORT_GRAD(__half)
                                : MOEDC_UNSORT_GRAD(__nv_bfloat16);
#undef MOEDC_UNSORT_GRAD
}
