// Products of packed expert rows in e4m3 with a scale for each block of 128.
#include "matmul.cuh"

namespace moedc {

// Rows of x and their scales in packed order, a warp a row (70 us for 32768 rows of 7168); a row of
// nobody's is left alone, one that src leads outside is zeros under scales that no other row has,
// as a weight's NaN times 0 would not be 0.  (Looked up in src again by matmul_rows it costs 332 ->
// 336 us, 64 experts of 128 rows x 2 x 2048 x 7168.)
constexpr int kMmCopyRows = 8;
__global__ void __launch_bounds__(kMmCopyRows* kWarp) matmul_gather_kernel(const __grid_constant__ MmArgs a,
                                                                          const uint8_t* __restrict__ x, int groups,
                                                                          uint8_t* __restrict__ to, float* __restrict__ to_xs)
{
    extern __shared__ int32_t s_maps[];
    __shared__ int64_t s_scan[kMmCopyRows];
    int32_t *s_pre = s_maps, *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;
    pdl_enter();
    const bool over = mm_chunks<kMmCopyRows * kWarp>(a, kMmCopyRows, 1, s_scan, s_pre, s_beg, s_end);
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);
    const int lane = threadIdx.x % kWarp;
    bool bad = false;
    for (int unit = blockIdx.x; unit < s_pre[a.E]; unit += gridDim.x) {
        int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_pre[mid] <= unit) lo = mid; else hi = mid - 1;
        }
        const int in = (unit - s_pre[lo]) * kMmCopyRows + threadIdx.x / kWarp;
        if (in >= s_end[lo] - s_beg[lo]) continue;
        const int r = s_beg[lo] + in;
        const int t = mm_x_row(a, r);
        bad |= t < 0;
        const uint4* from = reinterpret_cast<const uint4*>(x + (int64_t)max(t, 0) * a.K);
        uint4* out = reinterpret_cast<uint4*>(to + (int64_t)r * a.K);
        for (int i = lane; i < a.K / 16; i += 8 * kWarp) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = t < 0 || i + k * kWarp >= a.K / 16 ? make_uint4(0, 0, 0, 0) : __ldg(from + i + k * kWarp);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k * kWarp < a.K / 16) out[i + k * kWarp] = v[k];
        }
        for (int g = lane; g < groups; g += kWarp)
            // (a scale of -0 becomes 0, which no sum shows)
            to_xs[(int64_t)r * groups + g] =
                t < 0 ? __uint_as_float(kMmLostScale) : __fadd_rn(__ldg(a.xs + t * a.xs_r + g * a.xs_g), 0.0f);
    }
    if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
}

}  // namespace moedc

namespace moedc_host {

#ifndef MOEDC_STREAM_ROWS
#define MOEDC_STREAM_ROWS 24
#endif

// By rows an expert, us of the weights on the tile's rows / of the tokens on them:
//   rows                              8         16        24        32
//   64 experts of 2 x 2048 x 7168  270 / 300 273 / 302 275 / 304 280 / 305
//   128 of 2048 x 2048                        87 / 90   90 / 91       / 92
//   8 of 7168 x 2048                          26 / 28             31 / 29
// Tiles so few that clusters share them are the exception, up to twice as many rows: one expert of
// 7168 x 7168, 16 rows 15.5 / 28, 32 rows 17.6 / 28, 48 rows 19 / 28.  (49 to 64 rows are still
// one chunk of tokens and would take 20 to 23; four experts of 2 x 2048 x 7168, 64 tiles, are
// beyond: 32 / 33 at 16 rows, 36 / 33 at 32.)
// `rows` is what the buffer holds, padding and unused slots included: the counts are on the device.
static bool weights_on_rows(int E, int N, bool gated, int rows)
{
    const int64_t active = E < rows ? E : rows;
    return rows <= MOEDC_STREAM_ROWS * active ||
           (rows <= 2 * MOEDC_STREAM_ROWS && active * ((N + (gated ? 127 : 255)) / (gated ? 128 : 256)) <= 36);
}

// Gathering the rows of a block's stage by TMA takes some 80 clocks for four of them, again
// for every tile of columns.  By rows an expert, us of rows gathered so / of rows brought into
// packed order first, with the tokens on the tile's rows:
//   rows                              8         16        24        32        48        128
//   64 experts of 2 x 2048 x 7168  284 / 307 297 / 310 321 / 312 352 / 314 407 / 317 908 / 333
//   128 of 2 x 1024 x 4096         170 / 189 179 / 191 193 / 193 213 / 196 242 / 199
static bool gathers_first(int E, int rows)
{
    const int64_t active = E < rows ? E : rows;
    return rows > MOEDC_STREAM_ROWS * active;
}

static int launch_mm_gather(moedc::MmArgs& a, const void* x, uint8_t* workspace, cudaStream_t stream)
{
    const int groups = a.xs_g == 0 ? 1 : a.K / 128;
    float* xs = reinterpret_cast<float*>(workspace + (size_t)a.rows * a.K);
    const int64_t units = (int64_t)a.rows / moedc::kMmCopyRows + a.E, most = 8 * (int64_t)sm_count();
    clear_stale_error();
    launch(moedc::matmul_gather_kernel, (int)(units < most ? units : most), moedc::kMmCopyRows * moedc::kWarp,
           (3 * (size_t)a.E + 1) * sizeof(int32_t), stream, a, static_cast<const uint8_t*>(x), groups, workspace, xs);
    a.xs = xs;
    a.xs_r = groups;
    a.packed = true;
    return launch_status();
}

}  // namespace moedc_host

extern "C" size_t moedc_matmul_e4m3_workspace_bytes(int Kd, int E, int rows)
{
    if (Kd < 128 || Kd % 128 != 0 || E < 1 || E > MOEDC_MAX_E || rows < 1) return 0;
    return moedc_host::gathers_first(E, rows) ? (size_t)rows * Kd + (size_t)rows * (Kd / 128) * sizeof(float) : 0;
}

extern "C" int moedc_matmul_e4m3(const void* x, int x_rows, int Kd, const float* xs, int scale_layout, const void* w,
                                 const float* ws, int E, int N, int flags, const int32_t* offsets,
                                 const int32_t* counts, const int32_t* src, int top_k, int rows, int out_dtype, void* out,
                                 float* out_scales, void* workspace, size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    const bool gated = (flags & MOEDC_SWIGLU) != 0, codes = out_dtype == MOEDC_FP8_E4M3;
    const bool slots = counts && !offsets;
    const int mode = scale_mode(scale_layout);
    if (Kd < 128 || Kd % 128 != 0 || N < 1 || N > INT32_MAX / 2 || E < 1 || E > MOEDC_MAX_E || x_rows < 0 || rows < 0 ||
        (flags & ~MOEDC_SWIGLU) != 0 || (out_dtype != MOEDC_BF16 && out_dtype != MOEDC_F16 && !codes))
        return MOEDC_ERR_ARG;
    if ((!counts && (offsets || E != 1)) || (slots && rows % E != 0) || mode < 0 || (mode == 1 && (!slots || src)) ||
        (src && top_k < 1) || (!src && x_rows != rows) || (codes && N % 128 != 0))
        return MOEDC_ERR_ARG;
    if (!w || !ws || !dev_status || !aligned(x, 16) || !aligned(w, 16) || !aligned(xs, 4) || !aligned(ws, 4) ||
        !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(src, 4) || !aligned(out, codes ? 16 : 2) ||
        !aligned(out_scales, 4) || !aligned(workspace, 16) || !aligned(dev_status, 4))
        return MOEDC_ERR_ARG;
    if (((int64_t)rows / 64 + E) * (N / 128 + 1) > INT32_MAX) return MOEDC_ERR_ARG;   // units are counted in 32 bits
    if (rows == 0 || x_rows == 0) return MOEDC_OK;
    if (!x || !xs || !out || (codes && !out_scales)) return MOEDC_ERR_ARG;
    moedc::MmArgs a{};
    a.E = E;
    a.N = N;
    a.K = Kd;
    a.rows = rows;
    a.x_rows = x_rows;
    a.slots = rows / E;
    a.top_k = top_k;
    a.offsets = offsets;
    a.counts = counts;
    a.src = src;
    a.status = dev_status;
    a.xs = xs;
    a.ws = ws;
    const int64_t G = Kd / 128;
    a.xs_r = mode == 0 ? G : 1;
    a.xs_g = mode == 0 ? 1 : mode == 1 ? a.slots : 0;
    a.xs_e = (mode == 2 ? 1 : G) * a.slots;
    a.out = out;
    a.extra = out_scales;
    a.gated = gated;
    a.f16 = out_dtype == MOEDC_F16;
    a.codes = codes;
    a.vec = N % 8 == 0 && aligned(out, 16);
    a.wait_extra = test_wait_extra();
    const size_t copy = src && workspace ? moedc_matmul_e4m3_workspace_bytes(Kd, E, rows) : 0;
    if (copy && workspace_bytes >= copy) {
        const int st = launch_mm_gather(a, x, static_cast<uint8_t*>(workspace), stream);
        if (st != MOEDC_OK) return st;
        x = workspace;
    }
    // Rows to gather that a workspace would have brought to the other form keep its order of
    // sums, every channel's in one block: the workspace changes no bit.
    const bool few = weights_on_rows(E, N, gated, rows);
    if ((a.src && !a.packed) || few) return launch_mm_stream(a, x, w, few, stream);
    return launch_mm_rows(a, x, w, stream);
}
