// Token rows sorted by expert into one packed buffer, the weighted way back,
// and their gradients.
//
// With row[t][k] the packed row of entry (t, k):
//   sort         rows[row[t][k]] = x[t]
//   unsort       y[t] = sum_k w[t][k] rows[row[t][k]]   (w = 1: sort's gradient)
//   unsort_grad  drows[row[t][k]] = w[t][k] dy[t],  dw[t][k] = <dy[t], rows[row[t][k]]>
// All four move rows: HBM traffic bounds them.
#include <climits>

#include "lm_common.cuh"

namespace moedc {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / kWarp;

// Exclusive prefix over the experts of the aligned counts (s_off[0..E]) and of
// the padding before each group (s_pad[0..E]: padding rows of the groups
// before it), by the whole block.  Counts are clamped to [0, rows] and the
// sums saturate at `rows`, so that no count, whatever it holds, leads out of
// the buffer.
__device__ __forceinline__ void group_offsets(const int32_t* __restrict__ counts, int E,
                                              int align, int rows, int32_t* s_off,
                                              int32_t* s_pad, int32_t* s_cnt)
{
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        s_cnt[e] = min(max(__ldg(counts + e), 0), rows);
    __syncthreads();
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

// U: the unit of one access (16 bytes, or one element where rows are not
// 16-byte multiples); `units` of them per row.
template <typename U>
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(const U* __restrict__ x, int64_t ldx, int units, const int32_t* __restrict__ topk_idx,
            const int32_t* __restrict__ slot, const int32_t* __restrict__ counts, int T, int K,
            int E, int align, int rows, U* __restrict__ sorted, int32_t* __restrict__ row,
            int32_t* __restrict__ src, int32_t* __restrict__ offsets, int32_t* __restrict__ status)
{
    extern __shared__ int32_t s_mem[];   // off [E + 1], pad [E + 1], cnt [E]
    pdl_enter();
    int32_t *s_off = s_mem, *s_pad = s_mem + E + 1, *s_cnt = s_mem + 2 * (E + 1);
    group_offsets(counts, E, align, rows, s_off, s_pad, s_cnt);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = s_off[e];
    const int lane = threadIdx.x % kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kSortWarps;
    const int64_t warp0 = (int64_t)blockIdx.x * kSortWarps + threadIdx.x / kWarp;
    const int slices = units ? (units + 4 * kWarp - 1) / (4 * kWarp) : 1;
    bool dropped = false;
    for (int64_t it = warp0; it < (int64_t)T * slices; it += nwarps) {
        const int64_t t = it / slices;
        const int u0 = (int)(it - t * slices) * 4 * kWarp + lane;
        int r = -1;
        if (lane < K) {
            const int e = __ldg(topk_idx + t * K + lane);
            const int s = __ldg(slot + t * K + lane);
            if (e >= 0 && e < E && s >= 0) {
                const int64_t at = (int64_t)s_off[e] + s;
                if (at < rows) r = (int)at;
                else dropped = true;
            }
            if (u0 == lane) {
                row[t * K + lane] = r;
                if (r >= 0) src[r] = (int)(t * K + lane);
            }
        }
        U v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (u0 + j * kWarp < units) v[j] = __ldg(x + t * ldx + u0 + j * kWarp);
        for (int k = 0; k < K; ++k) {
            const int rk = __shfl_sync(0xffffffffu, r, k);
            if (rk < 0) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (u0 + j * kWarp < units)
                    sorted[(int64_t)rk * units + u0 + j * kWarp] = v[j];
        }
    }
    // the rows that no entry reaches: padding of each group, and the tail
    const int64_t live = (int64_t)s_off[E] - s_pad[E];
    for (int64_t p = warp0; p < rows - live; p += nwarps) {
        int lo = 0, hi = E;   // last group g with s_pad[g] <= p
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_pad[mid] <= p) lo = mid; else hi = mid - 1;
        }
        const int64_t r = (int64_t)s_off[lo] + (lo < E ? s_cnt[lo] : 0) + (p - s_pad[lo]);
        if (r < 0 || r >= rows) continue;
        if (lane == 0) src[r] = -1;
        U zero{};
        for (int u = lane; u < units; u += kWarp) sorted[r * units + u] = zero;
    }
    if (dropped) raise_status(status, MOEDC_ERR_CAPACITY);
}

template <typename T, int V>
__global__ void __launch_bounds__(kSortThreads)
unsort_kernel(const T* __restrict__ sorted, int rows, int H, const int32_t* __restrict__ row,
              const float* __restrict__ weights, int tokens, int K, T* __restrict__ y)
{
    pdl_enter();
    using P = Pack<T, V>;
    const int lane = threadIdx.x % kWarp;
    const int units = H / V;
    const int slices = (units + kWarp - 1) / kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kSortWarps;
    for (int64_t it = (int64_t)blockIdx.x * kSortWarps + threadIdx.x / kWarp;
         it < (int64_t)tokens * slices; it += nwarps) {
        const int64_t t = it / slices;
        const int u = (int)(it - t * slices) * kWarp + lane;
        int r = -1;
        float w = 1.0f;
        if (lane < K) {
            r = __ldg(row + t * K + lane);
            if (r >= rows) r = -1;
            if (weights) w = __ldg(weights + t * K + lane);
        }
        float acc[V] = {};
        for (int k = 0; k < K; ++k) {
            const int rk = __shfl_sync(0xffffffffu, r, k);
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (rk < 0 || u >= units) continue;
            const P v = reinterpret_cast<const P*>(sorted)[(int64_t)rk * units + u];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, to_f32(v.v[i]), acc[i]);
        }
        if (u < units) {
            P o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(acc[i]);
            reinterpret_cast<P*>(y)[t * units + u] = o;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kSortThreads)
unsort_grad_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ sorted, int rows,
                   int H, const int32_t* __restrict__ row, const int32_t* __restrict__ src,
                   const float* __restrict__ weights, int tokens, int K, T* __restrict__ dsorted,
                   float* __restrict__ dweights)
{
    __shared__ float s_part[kSortWarps];
    pdl_enter();
    using P = Pack<T, V>;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int units = H / V;
    const int64_t entries = (int64_t)tokens * K;
    for (int64_t i = blockIdx.x; i < entries; i += gridDim.x) {
        const int64_t t = i / K;
        const int r = row[i];
        const bool ok = r >= 0 && r < rows;
        float dot = 0.0f;
        if (ok) {
            const float w = weights[i];
            const P* g = reinterpret_cast<const P*>(dy + t * lddy);
            for (int u = threadIdx.x; u < units; u += kSortThreads) {
                const P d = g[u];
                P o;
#pragma unroll
                for (int j = 0; j < V; ++j) o.v[j] = from_f32<T>(w * to_f32(d.v[j]));
                reinterpret_cast<P*>(dsorted)[(int64_t)r * units + u] = o;
                if (dweights) {
                    const P v = reinterpret_cast<const P*>(sorted)[(int64_t)r * units + u];
#pragma unroll
                    for (int j = 0; j < V; ++j) dot = fmaf(to_f32(d.v[j]), to_f32(v.v[j]), dot);
                }
            }
        }
        if (!dweights) continue;
        dot = warp_sum(dot);
        if (lane == 0) s_part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float s = 0.0f;
            for (int j = 0; j < kSortWarps; ++j) s += s_part[j];
            dweights[i] = ok ? s : 0.0f;
        }
        __syncthreads();
    }
    const int64_t nwarps = (int64_t)gridDim.x * kSortWarps;
    for (int64_t r = (int64_t)blockIdx.x * kSortWarps + warp; r < rows; r += nwarps) {
        if (src[r] >= 0) continue;
        P zero{};
        for (int u = lane; u < units; u += kWarp) reinterpret_cast<P*>(dsorted)[r * units + u] = zero;
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
int launch_sort(const void* x, int64_t ldx, int units, const int32_t* topk_idx,
                const int32_t* slot, const int32_t* counts, int T, int K, int E, int align,
                int rows, void* sorted, int32_t* row, int32_t* src, int32_t* offsets,
                int32_t* status, cudaStream_t stream)
{
    auto* k = moedc::sort_kernel<U>;
    const size_t smem = (3 * (size_t)E + 2) * sizeof(int32_t);
    const int slices = units ? (units + 127) / 128 : 1;
    const int64_t want = ((int64_t)T * slices + moedc::kSortWarps - 1) / moedc::kSortWarps;
    const int blocks = sort_blocks((const void*)k, smem, want);
    clear_stale_error();
    launch(k, blocks, moedc::kSortThreads, smem, stream, static_cast<const U*>(x), ldx, units,
           topk_idx, slot, counts, T, K, E, align, rows, static_cast<U*>(sorted), row, src,
           offsets, status);
    return launch_status();
}

template <typename T, int V>
int launch_unsort(const void* sorted, int rows, int H, const int32_t* row, const float* w,
                  int tokens, int K, void* y, cudaStream_t stream)
{
    auto* k = moedc::unsort_kernel<T, V>;
    const int64_t items = (int64_t)tokens * ((H / V + 31) / 32);
    const int blocks = sort_blocks((const void*)k, 0, (items + moedc::kSortWarps - 1) / moedc::kSortWarps);
    clear_stale_error();
    launch(k, blocks, moedc::kSortThreads, 0, stream, static_cast<const T*>(sorted), rows, H, row,
           w, tokens, K, static_cast<T*>(y));
    return launch_status();
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
    char* base = static_cast<char*>(workspace);
    int32_t* slot = reinterpret_cast<int32_t*>(base + ws.slot);
    const int st = launch_layout(topk_idx, T, K, E, 1, INT32_MAX, counts,
                                 reinterpret_cast<int32_t*>(base + ws.per_rank),
                                 reinterpret_cast<uint8_t*>(base + ws.in_rank), slot,
                                 base + ws.layout, ws.total - ws.layout, dev_status, stream);
    if (st != MOEDC_OK) return st;
    if (!x) H = 0;
    if (rows_vec(dtype, H, x ? ldx : 0, x, sorted, nullptr))
        return launch_sort<uint4>(x, ldx * size / 16, H * size / 16, topk_idx, slot, counts, T, K,
                                  E, align, rows, sorted, row, src, offsets, dev_status, stream);
    if (size == 4)
        return launch_sort<uint32_t>(x, ldx, H, topk_idx, slot, counts, T, K, E, align, rows,
                                     sorted, row, src, offsets, dev_status, stream);
    return launch_sort<uint16_t>(x, ldx, H, topk_idx, slot, counts, T, K, E, align, rows, sorted,
                                 row, src, offsets, dev_status, stream);
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
    (vec ? launch_unsort<T_, moedc::kVec<T_>>(sorted, rows, H, row, topk_weights, T, K, y, stream) \
         : launch_unsort<T_, 1>(sorted, rows, H, row, topk_weights, T, K, y, stream))
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
