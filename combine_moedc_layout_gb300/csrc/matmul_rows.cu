// e4m3 products for many rows to an expert: the tokens on the rows of the tile.
//
// A block multiplies 128 tokens by 256 weight rows (with `gated` the gate and the up rows of
// 128 channels).  A stage is 128 channels, 48 KB, and has sums of its own in one of two
// buffers of 256 columns of tensor memory: a thread of the epilogue owns a token and half of
// the columns, gate and up of the same channels, and adds
//   xs[token] ws[block] * sum
// into 128 registers, so that the factor is one for 64 columns and the SwiGLU stays in the
// thread.
//
// A buffer goes from the products to the epilogue and back in some 1500 clocks, 512 of them
// products: that bounds a stage to 750, and reading and adding under it to some 900.
// 8192^3: 429 us, 2560 TFLOP/s; 256 experts of 128 rows x 2 x 2048 x 7168: 1182 us, 6.4 TB/s
// of weights.
//
// Warps: 0-7 epilogue (0-3 the first half of the columns, or of the channels, 4-7 the
// others), 8 TMA, 9 MMA.
#include "matmul_store.cuh"
#include "quotient.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace moedc {

constexpr int kMrThreads = 12 * kWarp;             // whole groups of four warps: they share registers out
constexpr int kMrRows = 128;
constexpr int kMrCols = 256;
constexpr int kMrGroup = 128;                      // channels, and bytes, of a stage
constexpr int kMrStage = (kMrRows + kMrCols) * kMrGroup;
constexpr int kMrStages = 4;
constexpr int kMrBuf = 8 * 2048;                   // of the epilogue's warps, for their stores
constexpr int kMrColumns = 512;

struct MrUnit {
    int e, r0, m, n0;
};

__device__ __forceinline__ MrUnit mr_unit(const MmArgs& a, const int32_t* s_pre, const int32_t* s_beg, const int32_t* s_end,
                                          int tiles, int unit)
{
    int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((int64_t)s_pre[mid] * tiles <= unit) lo = mid; else hi = mid - 1;
    }
    const int chunks = s_pre[lo + 1] - s_pre[lo];
    int t, c;
    mm_order(unit - s_pre[lo] * tiles, tiles, chunks, t, c);
    MrUnit u;
    u.e = lo;
    u.n0 = t * (a.gated ? kMrCols / 2 : kMrCols);
    u.r0 = s_beg[lo] + c * kMrRows;
    u.m = min(kMrRows, s_end[lo] - u.r0);
    return u;
}

__device__ __forceinline__ float ld_scale(const float* p)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__global__ void __launch_bounds__(kMrThreads, 1)
matmul_rows_kernel(const __grid_constant__ MmArgs a, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ BoxMaps xmaps)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMrThreads / kWarp];
    __shared__ uint64_t full[kMrStages], empty[kMrStages], d_full[2], d_empty[2], done, never;
    __shared__ float s_amax[2][kMrRows];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int tile_n = a.gated ? kMrCols / 2 : kMrCols;
    const int tiles = (a.N + tile_n - 1) / tile_n, groups = a.K / kMrGroup;
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + kMrStages * kMrStage + kMrBuf);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMrStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(d_full + b, 1);
            mbar_init(d_empty + b, 8);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "n"(kMrColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    pdl_enter();
    const bool over = mm_chunks<kMrThreads>(a, kMrRows, tiles, s_scan, s_pre, s_beg, s_end);   // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // The epilogue's threads keep 128 sums each.  The shares add up to the launch's 384 x 168
    // registers: 256 x 208 + 128 x 88.
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp < 8) {
        // ---- epilogue (without calls: with one, its registers do not compile to a share)
        if (a.wait_extra) mbar_wait_inline(&never, 0, &s_abort);
        const int half = warp >> 2, first = (warp & 3) * kWarp;
        const uint32_t d0 = tmem + ((uint32_t)first << 16);
        // the columns of the thread's four parts of 32
        const int c01 = a.gated ? half * 64 : half * 128, c23 = a.gated ? 128 + half * 64 : half * 128 + 64;
        uint8_t* buf = smem + kMrStages * kMrStage + warp * 2048;
        MvRing accs;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const MrUnit u = mr_unit(a, s_pre, s_beg, s_end, tiles, unit);
            // how many of the warp's 32 rows there are
            const int have = u.m - first;
            const bool some = have > 0, mine = lane < have;
            const int r = u.r0 + first + lane;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.0f, 0.0f);
            const int xr = mine ? r : u.r0;
            const float* xs = a.xs + (a.offsets || !a.counts || a.packed ? xr * a.xs_r : u.e * a.xs_e + (xr - u.e * a.slots) * a.xs_r);
            const int blocks = (a.N + 127) / 128;
            const int b0 = a.gated ? u.n0 / 128 : min(u.n0 / 128 + half, blocks - 1);
            const float* w0 = a.ws + ((int64_t)u.e * (a.gated ? 2 : 1) * blocks + b0) * groups;
            const float* w1 = a.gated ? w0 + (int64_t)blocks * groups : w0;
            // scales of four groups, each replaced as soon as it is used: volatile loads, as the
            // compiler would move them to their use
            float sx[4], s0[4], s1[4];
            auto load = [&](int i, int g) __attribute__((always_inline)) {
                g = min(g, groups - 1);
                sx[i] = ld_scale(xs + g * a.xs_g), s0[i] = ld_scale(w0 + g), s1[i] = ld_scale(w1 + g);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) load(i, i);
            for (int g0 = 0; g0 < groups; g0 += 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (g0 + i >= groups) break;
                    const float f0 = sx[i] * s0[i], f1 = sx[i] * s1[i];
                    load(i, g0 + i + 4);
                    mbar_wait_inline(d_full + accs.slot, accs.phase, &s_abort);
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t d = d0 + accs.slot * kMrCols;
                    auto release = [&]() __attribute__((always_inline)) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(d_empty + accs.slot);
                    };
                    if (some) {
                        // the next 32 columns are read while 32 are added up; the buffer is free
                        // once the last ones are in registers
                        float v[2][32];
                        tc_ld32(d + c01, v[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(v[c & 1][j]));
                            if (c < 3) tc_ld32(d + (c < 1 ? c01 + 32 : c23 + (c - 1) * 32), v[(c + 1) & 1]);
                            else release();
                            const float2 s = splat2(c < 2 ? f0 : f1);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                acc[c * 16 + j] = fma2_rn(make_float2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), s, acc[c * 16 + j]);
                        }
                    } else {
                        release();
                    }
                    accs.next(2);
                }
            }
            float* v = reinterpret_cast<float*>(acc);
            // a row that src led outside of x: zeros, whatever the weights hold (every sx is the last
            // group's by now)
            if (a.packed && __float_as_uint(sx[0]) == kMmLostScale) {
#pragma unroll
                for (int j = 0; j < 128; ++j) v[j] = 0.0f;
            }
            if (a.gated) {
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = mm_silu_mul(v[j], v[64 + j]);
            }
            if (!a.codes) {
                uint16_t* o = static_cast<uint16_t*>(a.out) + (int64_t)(u.r0 + first) * a.N;
                if (some) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < 2 || !a.gated)
                            mm_store32(buf, o, a.N, u.n0 + half * (a.gated ? 64 : 128) + c * 32, a.N, have, a.vec, a.f16, v + c * 32);
                }
            } else {
                // the rule of dispatch, of the binary32 values: 128 channels are this thread's,
                // or with `gated` this thread's and that of the other half's same lane
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j < 64 || !a.gated) top = fmaxf(top, fabsf(v[j]));
                if (a.gated) {
                    s_amax[half][(warp & 3) * kWarp + lane] = top;
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    top = fmaxf(top, s_amax[half ^ 1][(warp & 3) * kWarp + lane]);
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                top = fmaxf(top, 1e-4f);
                const float sc = __fdiv_rn(top, 448.0f);
                const Quotient<2> by = Quotient<2>::by(sc);
                const int n = u.n0 + half * (a.gated ? 64 : 128);
                if (some && n < a.N) {
                    uint8_t* o = static_cast<uint8_t*>(a.out) + (int64_t)(u.r0 + first) * a.N + n;
#pragma unroll
                    for (int h = 0; h < 128; h += 64) {
                        if (h >= 64 && a.gated) break;
                        uint4 q[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float* f = v + h + 16 * k + 4 * i;
                                w[i] = by.codes(f[0], f[1]) | by.codes(f[2], f[3]) << 16;
                            }
                            q[k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        mm_store_rows(buf, q, o + h, a.N, have, 64);
                    }
                    if (mine && (!a.gated || half == 0))
                        static_cast<float*>(a.extra)[(int64_t)r * (a.N / 128) + n / 128] = sc;
                }
            }
        }
    } else if (warp == 8) {
        // ---- TMA
        // (one lane waits and issues)
        MvRing ring;
        int issued = 0;
        bool stop = !tc_elect();
        for (int unit = blockIdx.x; unit < units && !stop; unit += gridDim.x) {
            const MrUnit u = mr_unit(a, s_pre, s_beg, s_end, tiles, unit);
            const int box = (u.m + 31) / 32;   // in 32 rows
            const int bytes = (kMrCols + box * 32) * kMrGroup;
            for (int g = 0; g < groups; ++g) {
                if (!mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort)) {
                    stop = true;
                    break;
                }
                uint8_t* st = smem + ring.slot * kMrStage;
                uint64_t* bar = full + ring.slot;
                mbar_arrive_expect(bar, bytes);
                // [E][1 or 2][N][K]
                tma_4d(st, &wmap, g * kMrGroup, u.n0, 0, u.e, bar);
                tma_4d(st + kMrCols / 2 * kMrGroup, &wmap, g * kMrGroup, u.n0 + (a.gated ? 0 : kMrCols / 2), a.gated ? 1 : 0, u.e, bar);
                st += kMrCols * kMrGroup;
                // rows past the chunk's are of no account
                tma_2d(st, xmaps.by + (box - 1), g * kMrGroup, u.r0, bar);
                ring.next(kMrStages);
                ++issued;
            }
        }
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - kMrStages); n < issued; ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % kMrStages, (n / kMrStages) & 1, &alone)) s_abort = 1;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- MMA: one elected lane issues; the warp stays together
        const bool leader = tc_elect();
        MvRing ring, accs;
        int k = 0;
        const uint32_t idesc = (1u << 4) | ((uint32_t)(kMrCols / 8) << 17) | ((uint32_t)(kMrRows / 16) << 24);
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            for (int g = 0; g < groups; ++g) {
                if (k++ >= 2) mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                mbar_wait_warp(full + ring.slot, ring.phase, &s_abort);
                tc_fence_after();
                const uint32_t st = smem_u32(smem + ring.slot * kMrStage);
                const uint64_t w = tc_smem_desc(st), x = tc_smem_desc(st + kMrCols * kMrGroup);
                if (leader) {
#pragma unroll
                    for (int p = 0; p < 4; ++p)   // 32 channels each; a descriptor counts in 16 bytes
                        tc_mma_e4m3(tmem + accs.slot * kMrCols, x + p * 2, w + p * 2, idesc, p != 0);
                    tc_commit(d_full + accs.slot);
                    tc_commit(empty + ring.slot);
                }
                __syncwarp();
                accs.next(2);
                ring.next(kMrStages);
            }
        }
        // tensor memory is given back only when the last product is through
        if (leader) tc_commit(&done);
        __syncwarp();
        volatile int alone = 0;
        if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kMrColumns) : "memory");
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {

int launch_mm_rows(const moedc::MmArgs& a, const void* x, const void* w, cudaStream_t stream)
{
    constexpr auto kType = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    constexpr auto kSwizzle = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap wmap;
    moedc::BoxMaps xmaps{};
    const cuuint64_t K = a.K, N = a.N, parts = a.gated ? 2 : 1;
    const cuuint64_t xsize[2] = {K, (cuuint64_t)(a.packed ? a.rows : a.x_rows)}, xstride[1] = {K};
    const cuuint64_t size[4] = {K, N, parts, (cuuint64_t)a.E}, stride[3] = {K, K * N, K * N * parts};
    const cuuint32_t box[4] = {128, moedc::kMrCols / 2, 1, 1};
    if (!tensor_map(&wmap, kType, kSwizzle, w, 4, size, stride, box)) return MOEDC_ERR_CUDA;
    for (int i = 0; i < 4; ++i) {
        const cuuint32_t xbox[2] = {128, (cuuint32_t)(32 * (i + 1))};
        if (!tensor_map(xmaps.by + i, kType, kSwizzle, x, 2, xsize, xstride, xbox)) return MOEDC_ERR_CUDA;
    }
    auto* k = moedc::matmul_rows_kernel;
    constexpr size_t kFixed = moedc::kMrStages * moedc::kMrStage + moedc::kMrBuf;
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, (int)kFixed + (3 * MOEDC_MAX_E + 1) * 4)) return MOEDC_ERR_CUDA;
    const int tile = a.gated ? moedc::kMrCols / 2 : moedc::kMrCols;
    const int64_t units = ((int64_t)a.rows / moedc::kMrRows + (a.E < a.rows ? a.E : a.rows)) * ((a.N + (int64_t)tile - 1) / tile);
    const int blocks = sm_count();
    clear_stale_error();
    launch(k, (int)(units < blocks ? units : blocks), moedc::kMrThreads, kFixed + (3 * (size_t)a.E + 1) * sizeof(int32_t), stream, a,
           wmap, xmaps);
    return launch_status();
}

}  // namespace moedc_host
