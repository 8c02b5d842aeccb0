// e4m3 products for few rows to an expert, where the stream of the weights is the bound.
//
// The weights lie on the rows of the tile and the tokens on its columns, as many (in
// sixteens) as there are: a block multiplies 256 weight rows, in two tiles of 128 (with
// `gated` the gate and the up rows of 128 channels), by up to 64 tokens.  A stage, 128
// channels, is 32 KB of weights and 2 KB for each 16 tokens; four or five stages under way
// on each SM keep HBM busy.
//
// Each stage has sums of its own, four buffers of tensor memory in turn.  A thread of the
// epilogue owns a weight row of both tiles and half of the tokens, and adds
//   xs[token] ws[block] * sum
// into 64 registers; the factors come from shared memory, where one warp puts them four
// groups ahead.
//
// Where there are too few tiles for the SMs, a cluster of blocks shares one: each block takes
// a part of the channels, in fours of groups, and sends its sums to the first one's shared
// memory, which adds them in the blocks' order.
//
// 64 experts of 8 rows x 2 x 2048 x 7168: 270 us, 7.0 TB/s of weights, HBM's rate (289 us with
// room for 128 tokens, two sums and four stages); one token x 7168 x 7168: 13 us, latency.
//
// Warps: 0-7 epilogue (0-3 the first 32 tokens, 4-7 the others), 8 TMA, 9 MMA, 10 factors.
#include "matmul.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace moedc {

constexpr int kMsThreads = 11 * kWarp;
constexpr int kMsRows = 128;                        // of a tile of weights
constexpr int kMsTokens = 64;
constexpr int kMsHalf = kMsTokens / 2;
constexpr int kMsGroup = 128;                       // channels, and bytes, of a stage
constexpr int kMsTile = kMsRows * kMsGroup;
constexpr int kMsStage = 2 * kMsTile + kMsTokens * kMsGroup;
constexpr int kMsStages = 5;
constexpr int kMsFactors = 4 * 2 * kMsTokens;       // floats of four groups
constexpr int kMsFactorBufs = 3;
constexpr int kMsColumns = 512;
constexpr int kMsAccs = kMsColumns / (2 * kMsTokens);   // sums under way

struct MsUnit {
    int e, r0, m, n0;
};

__device__ __forceinline__ MsUnit ms_unit(const MmArgs& a, const int32_t* s_pre, const int32_t* s_beg, const int32_t* s_end,
                                          int tiles, int unit)
{
    int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((int64_t)s_pre[mid] * tiles <= unit) lo = mid; else hi = mid - 1;
    }
    const int chunks = s_pre[lo + 1] - s_pre[lo];
    const int in = unit - s_pre[lo] * tiles, t = in / chunks;   // chunks of one tile are neighbours
    MsUnit u;
    u.e = lo;
    u.n0 = t * (a.gated ? kMsRows : 2 * kMsRows);
    u.r0 = s_beg[lo] + (in - t * chunks) * kMsTokens;
    u.m = min(kMsTokens, s_end[lo] - u.r0);
    return u;
}

__global__ void __launch_bounds__(kMsThreads, 1)
matmul_stream_kernel(const __grid_constant__ MmArgs a, int parts, const __grid_constant__ CUtensorMap wmap,
                     const __grid_constant__ BoxMaps xmaps)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMsThreads / kWarp];
    __shared__ uint64_t full[kMsStages], empty[kMsStages], d_full[kMsAccs], d_empty[kMsAccs], f_full[kMsFactorBufs], f_empty[kMsFactorBufs];
    __shared__ uint64_t done, never;
    __shared__ float s_top[2][2][4][kMsHalf], s_scale[2][2][kMsHalf];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int tile_n = a.gated ? kMsRows : 2 * kMsRows;
    const int tiles = (a.N + tile_n - 1) / tile_n, groups = a.K / kMsGroup;
    const int part = parts > 1 ? cluster_rank() : 0, first_unit = blockIdx.x / parts, unit_step = gridDim.x / parts;
    const int quads_all = (groups + 3) / 4;
    const int g_beg = quads_all * part / parts * 4, g_end = min(quads_all * (part + 1) / parts * 4, groups);
    float* s_factors = reinterpret_cast<float*>(smem + kMsStages * kMsStage);
    int32_t* s_pre = reinterpret_cast<int32_t*>(s_factors + kMsFactorBufs * kMsFactors);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMsStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < kMsAccs; ++b) {
            mbar_init(d_full + b, 1);
            mbar_init(d_empty + b, 8);
        }
        for (int b = 0; b < kMsFactorBufs; ++b) {
            mbar_init(f_full + b, 1);
            mbar_init(f_empty + b, 8);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "n"(kMsColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    pdl_enter();
    const bool over = mm_chunks<kMsThreads>(a, kMsTokens, tiles, s_scan, s_pre, s_beg, s_end);   // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // every warp of a cluster comes by the three barriers of a tile, those that have nothing
    // to do between them as well
    auto tile_done = [&]() __attribute__((always_inline)) {
        if (parts > 1) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
            cluster_sync();
        }
    };
    if (warp < 8) {
        // ---- epilogue
        if (a.wait_extra) mbar_wait(&never, 0, &s_abort);
        const int half = warp >> 2, quad = warp & 3, row = quad * kWarp + lane, j0 = half * kMsHalf;
        const uint32_t d0 = tmem + ((uint32_t)(quad * kWarp) << 16) + j0;
        MvRing accs, facs;
        bool bad = false;
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MsUnit u = ms_unit(a, s_pre, s_beg, s_end, tiles, unit);
            const int mine = u.m - j0;                      // tokens of this warp
            float2 acc[2][kMsHalf / 2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < kMsHalf / 2; ++j) acc[t][j] = make_float2(0.0f, 0.0f);
            for (int g = g_beg; g < g_end; ++g) {
                if (g % 4 == 0) mbar_wait_inline(f_full + facs.slot, facs.phase, &s_abort);
                mbar_wait_inline(d_full + accs.slot, accs.phase, &s_abort);
                __syncwarp();
                tc_fence_after();
                const float* f = s_factors + facs.slot * kMsFactors + (g % 4) * (2 * kMsTokens) + j0;
                const uint32_t d = d0 + accs.slot * (2 * kMsTokens);
#pragma unroll
                for (int c = 0; c < kMsHalf; c += 16) {
                    if (c < mine) {
                        float v[2][16];
                        tc_ld16(d + c, v[0]);
                        tc_ld16(d + kMsTokens + c, v[1]);
                        tc_wait_ld();
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[t][j]));
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 s = *reinterpret_cast<const float4*>(f + t * kMsTokens + c + j);
                                float2* o = acc[t] + (c + j) / 2;
                                o[0] = fma2_rn(make_float2(v[t][j], v[t][j + 1]), make_float2(s.x, s.y), o[0]);
                                o[1] = fma2_rn(make_float2(v[t][j + 2], v[t][j + 3]), make_float2(s.z, s.w), o[1]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(d_empty + accs.slot);
                    if (g % 4 == 3 || g == g_end - 1) mbar_arrive(f_empty + facs.slot);
                }
                accs.next(kMsAccs);
                if (g % 4 == 3 || g == g_end - 1) facs.next(kMsFactorBufs);
            }
            if (parts > 1) {
                cluster_sync();     // 1: no block's products read its stages any more
                float* sums = reinterpret_cast<float*>(smem);   // [part - 1][tile][token / 4][row][token % 4]
                const int cols = (u.m + 15) / 16 * 16;
                // four tokens of a row together: each store at another block costs some 40 clocks
                if (part > 0) {
                    const uint32_t to = cluster_addr(sums + ((part - 1) * 2 * cols + j0) * kMsRows + row * 4, 0);
#pragma unroll
                    for (int j = 0; j < kMsHalf; j += 4) {
                        if (j >= mine) break;       // whole fours: `cols` has room for them
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            st_cluster(to + (t * cols + j) * (kMsRows * 4), acc[t][j / 2], acc[t][j / 2 + 1]);
                    }
                }
                cluster_sync();     // 2: the sums are there
                for (int p = 1; p < parts && part == 0; ++p) {
                    const float* from = sums + ((p - 1) * 2 * cols + j0) * kMsRows + row * 4;
#pragma unroll
                    for (int j = 0; j < kMsHalf; j += 4) {
                        if (j >= mine) break;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float4 s = *reinterpret_cast<const float4*>(from + (t * cols + j) * kMsRows);
                            acc[t][j / 2].x += s.x, acc[t][j / 2].y += s.y;
                            acc[t][j / 2 + 1].x += s.z, acc[t][j / 2 + 1].y += s.w;
                        }
                    }
                }
                // (the next tile's copies come to where these were)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                cluster_sync();     // 3: the sums have been read
                if (part > 0) continue;
            }
            // tokens that src leads outside of x: zeros
            if (a.src) {
#pragma unroll
                for (int c = 0; c < kMsHalf; c += kWarp) {
                    const bool out = c + lane < mine && mm_x_row(a, u.r0 + j0 + c + lane) < 0;
                    const unsigned lost = __ballot_sync(0xffffffffu, out);
                    bad |= out;
                    if (lost) {
#pragma unroll
                        for (int j = 0; j < kWarp; j += 2)
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                float2& o = acc[t][(c + j) / 2];
                                if (lost >> j & 1) o.x = 0.0f;
                                if (lost >> (j + 1) & 1) o.y = 0.0f;
                            }
                    }
                }
            }
            if (a.gated) {
#pragma unroll
                for (int j = 0; j < kMsHalf / 2; ++j) {
                    if (2 * j >= mine) break;
                    acc[0][j].x = mm_silu_mul(acc[0][j].x, acc[1][j].x);
                    acc[0][j].y = mm_silu_mul(acc[0][j].y, acc[1][j].y);
                }
            }
            const int n = u.n0 + row;
            const int64_t at = (int64_t)(u.r0 + j0) * a.N + n;
            if (!a.codes) {
                // a warp's lanes are 32 neighbouring channels of a token
                uint16_t* o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
                for (int c = 0; c < kMsHalf; c += 8) {
                    if (c >= mine) break;
#pragma unroll
                    for (int j = c; j < c + 8; ++j)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t == 1 && a.gated) break;
                            const float v = j & 1 ? acc[t][j / 2].y : acc[t][j / 2].x;
                            if (j < mine && n + t * kMsRows < a.N)
                                o[(int64_t)j * a.N + t * kMsRows] =
                                    a.f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        }
                }
            } else {
                // the rule of dispatch, of the binary32 values: a token's 128 channels are the
                // lanes of four warps.  Magnitudes order as their bits do; NaN is left out.
#pragma unroll
                for (int j = 0; j < kMsHalf; ++j) {
                    if (j >= mine) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && a.gated) break;
                        const float v = fabsf(j & 1 ? acc[t][j / 2].y : acc[t][j / 2].x);
                        const unsigned top = __reduce_max_sync(0xffffffffu, v == v ? __float_as_uint(v) : 0u);
                        if (lane == 0) s_top[half][t][quad][j] = __uint_as_float(top);
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                {
                    const int t = row / kMsHalf, j = row % kMsHalf;   // both tiles' 32 tokens
                    if (t < (a.gated ? 1 : 2) && j < mine) {
                        const float(&p)[4][kMsHalf] = s_top[half][t];
                        const float top = fmaxf(fmaxf(p[0][j], p[1][j]), fmaxf(p[2][j], p[3][j]));
                        const float sc = __fdiv_rn(fmaxf(top, 1e-4f), 448.0f);
                        s_scale[half][t][j] = sc;
                        const int b = u.n0 / 128 + t;
                        if (b < a.N / 128) static_cast<float*>(a.extra)[(int64_t)(u.r0 + j0 + j) * (a.N / 128) + b] = sc;
                    }
                }
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                uint8_t* o = static_cast<uint8_t*>(a.out) + at;
#pragma unroll
                for (int j = 0; j < kMsHalf; ++j) {
                    if (j >= mine) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && a.gated) break;
                        const float v = j & 1 ? acc[t][j / 2].y : acc[t][j / 2].x;
                        if (n + t * kMsRows < a.N)
                            o[(int64_t)j * a.N + t * kMsRows] = (uint8_t)pack_e4m3x2(__fdiv_rn(v, s_scale[half][t][j]), 0.0f);
                    }
                }
            }
        }
        if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    } else if (warp == 8) {
        // ---- TMA: two tiles of weights; the tokens, four by four where they are gathered
        // (one lane waits and issues, but where each lane gathers four of the rows)
        MvRing ring;
        int issued = 0;
        const bool gather = a.src && !a.packed, first = gather ? lane == 0 : tc_elect();
        bool stop = !gather && !first;
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MsUnit u = ms_unit(a, s_pre, s_beg, s_end, tiles, unit);
            int t[4] = {0, 0, 0, 0};
            if (gather) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane * 4 + i < u.m) t[i] = max(mm_x_row(a, u.r0 + lane * 4 + i), 0);
            }
            const int box = u.m <= 16 ? 0 : u.m <= 32 ? 1 : 2;   // 16 << box rows
            const int bytes = 2 * kMsTile + (gather ? (u.m + 3) / 4 * 4 : 16 << box) * kMsGroup;
            for (int g = g_beg; g < g_end && !stop; ++g) {
                stop = !mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort);
                if (gather) stop = __any_sync(0xffffffffu, stop);
                if (stop) break;
                uint8_t* st = smem + ring.slot * kMsStage;
                uint64_t* bar = full + ring.slot;
                if (first) {
                    mbar_arrive_expect(bar, bytes);
                    // [E][1 or 2][N][K]
                    tma_4d(st, &wmap, g * kMsGroup, u.n0, 0, u.e, bar);
                    tma_4d(st + kMsTile, &wmap, g * kMsGroup, u.n0 + (a.gated ? 0 : kMsRows), a.gated ? 1 : 0, u.e, bar);
                    // rows past the chunk's are of no account
                    if (!gather) tma_2d(st + 2 * kMsTile, xmaps.by + box, g * kMsGroup, u.r0, bar);
                }
                if (gather) {
                    __syncwarp();
                    if (lane * 4 < u.m)
                        tma_gather4(st + 2 * kMsTile + lane * 4 * kMsGroup, xmaps.by, g * kMsGroup, t[0], t[1], t[2], t[3], bar);
                    __syncwarp();
                }
                ring.next(kMsStages);
                ++issued;
            }
            tile_done();
        }
        __syncwarp();
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - kMsStages); n < issued; ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % kMsStages, (n / kMsStages) & 1, &alone)) s_abort = 1;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- MMA: one elected lane issues; the warp stays together
        const bool leader = tc_elect();
        MvRing ring, accs;
        int k = 0;
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MsUnit u = ms_unit(a, s_pre, s_beg, s_end, tiles, unit);
            // columns: as many tokens as there are, by 16
            const uint32_t idesc = (1u << 4) | ((uint32_t)((u.m + 15) / 16 * 2) << 17) | ((uint32_t)(kMsRows / 16) << 24);
            for (int g = g_beg; g < g_end; ++g) {
                if (k++ >= kMsAccs) mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                mbar_wait_warp(full + ring.slot, ring.phase, &s_abort);
                tc_fence_after();
                const uint32_t st = smem_u32(smem + ring.slot * kMsStage);
                const uint64_t w = tc_smem_desc(st), x = tc_smem_desc(st + 2 * kMsTile);
                if (leader) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int p = 0; p < 4; ++p)   // 32 channels each; a descriptor counts in 16 bytes
                            tc_mma_e4m3(tmem + accs.slot * (2 * kMsTokens) + t * kMsTokens, w + t * (kMsTile / 16) + p * 2, x + p * 2,
                                        idesc, p != 0);
                    tc_commit(empty + ring.slot);
                    tc_commit(d_full + accs.slot);
                }
                __syncwarp();
                accs.next(kMsAccs);
                ring.next(kMsStages);
            }
            tile_done();
        }
        // tensor memory is given back only when the last product is through
        if (leader) tc_commit(&done);
        __syncwarp();
        volatile int alone = 0;
        if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        __syncwarp();
    } else {
        // ---- factors: four groups of a token are one load where they are 16 aligned bytes
        MvRing facs;
        const bool quads = a.xs_g == 1 && groups % 4 == 0 && reinterpret_cast<uintptr_t>(a.xs) % 16 == 0;
        const int blocks = (a.N + 127) / 128;
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MsUnit u = ms_unit(a, s_pre, s_beg, s_end, tiles, unit);
            const float* xs[kMsTokens / kWarp];
#pragma unroll
            for (int q = 0; q < kMsTokens / kWarp; ++q) {
                const int r = u.r0 + min(q * kWarp + lane, u.m - 1);
                xs[q] = a.xs + (a.packed                                ? r * a.xs_r
                                : a.offsets || !a.counts || a.src ? max(mm_x_row(a, r), 0) * a.xs_r
                                                                  : u.e * a.xs_e + (r - u.e * a.slots) * a.xs_r);
            }
            const int b0 = u.n0 / 128;
            const float* w0 = a.ws + ((int64_t)u.e * (a.gated ? 2 : 1) * blocks + b0) * groups;
            const float* w1 = w0 + (int64_t)(a.gated ? blocks : b0 + 1 < blocks) * groups;
            float s[kMsTokens / kWarp][4], v0[4], v1[4];
            auto load = [&](int g0) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int g = min(g0 + i, groups - 1);
                    v0[i] = __ldg(w0 + g), v1[i] = __ldg(w1 + g);
                }
#pragma unroll
                for (int q = 0; q < kMsTokens / kWarp; ++q) {
                    if (q * kWarp >= u.m) break;
                    if (quads) {
                        const float4 v = __ldg(reinterpret_cast<const float4*>(xs[q] + min(g0, groups - 4)));
                        s[q][0] = v.x, s[q][1] = v.y, s[q][2] = v.z, s[q][3] = v.w;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[q][i] = __ldg(xs[q] + min(g0 + i, groups - 1) * a.xs_g);
                    }
                }
            };
            load(g_beg);
            for (int g0 = g_beg; g0 < g_end; g0 += 4) {
                mbar_wait_warp(f_empty + facs.slot, facs.phase ^ 1, &s_abort);
                float* f = s_factors + facs.slot * kMsFactors + lane;
#pragma unroll
                for (int q = 0; q < kMsTokens / kWarp; ++q) {
                    if (q * kWarp >= u.m) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[i * (2 * kMsTokens) + q * kWarp] = s[q][i] * v0[i];
                        f[i * (2 * kMsTokens) + kMsTokens + q * kWarp] = s[q][i] * v1[i];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(f_full + facs.slot);
                facs.next(kMsFactorBufs);
                load(min(g0 + 4, groups - 1));
            }
            tile_done();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kMsColumns) : "memory");
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {

// most tiles that are split into as many parts
#ifndef MOEDC_PARTS_8
#define MOEDC_PARTS_8 14
#define MOEDC_PARTS_4 36
#define MOEDC_PARTS_2 72
#endif

int launch_mm_stream(const moedc::MmArgs& a, const void* x, const void* w, bool share, cudaStream_t stream)
{
    constexpr auto kType = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    constexpr auto kSwizzle = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap wmap;
    moedc::BoxMaps xmaps{};
    const cuuint64_t K = a.K, N = a.N, both = a.gated ? 2 : 1;
    const cuuint64_t xsize[2] = {K, (cuuint64_t)(a.packed ? a.rows : a.x_rows)}, xstride[1] = {K};
    const cuuint64_t size[4] = {K, N, both, (cuuint64_t)a.E}, stride[3] = {K, K * N, K * N * both};
    const cuuint32_t box[4] = {128, moedc::kMsRows, 1, 1};
    if (!tensor_map(&wmap, kType, kSwizzle, w, 4, size, stride, box)) return MOEDC_ERR_CUDA;
    // gathered rows: one map, a row high; else as many as the rows can need
    const bool gather = a.src && !a.packed;
    for (int i = 0; i < 3 && (i == 0 || (!gather && a.rows > 8 << i)); ++i) {
        const cuuint32_t xbox[2] = {128, gather ? 1u : 16u << i};
        if (!tensor_map(xmaps.by + i, kType, kSwizzle, x, 2, xsize, xstride, xbox)) return MOEDC_ERR_CUDA;
    }
    auto* k = moedc::matmul_stream_kernel;
    constexpr size_t kFixed = moedc::kMsStages * moedc::kMsStage + moedc::kMsFactorBufs * moedc::kMsFactors * sizeof(float);
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, (int)kFixed + (3 * MOEDC_MAX_E + 1) * 4)) return MOEDC_ERR_CUDA;
    const int tile = a.gated ? moedc::kMsRows : 2 * moedc::kMsRows;
    const int64_t units = ((int64_t)a.rows / moedc::kMsTokens + (a.E < a.rows ? a.E : a.rows)) * ((a.N + (int64_t)tile - 1) / tile);
    const int blocks = sm_count();
    // parts of the channels: a cluster of four or eight needs its SMs in one of the GPU's
    // groups of them, which holds two or three of the former.  One token x 7168 channels,
    // 28 tiles: 29.1 us in one part, 18.1 in two, 14.1 in four, 19.8 in eight (a second wave);
    // 14 tiles: 28.8, 17.8, 13.0, 10.7; 56 tiles: 29.8, 22.7, 26.8.
    const int64_t most = a.rows < moedc::kMsTokens ? a.rows : moedc::kMsTokens;
    const int64_t sums = (most + 15) / 16 * 16 * 2 * moedc::kMsRows * sizeof(float);
    auto fits = [&](int p, int64_t tiles) {
        return share && units <= tiles && a.K / moedc::kMsGroup >= 4 * p && (p - 1) * sums <= moedc::kMsStages * moedc::kMsStage;
    };
    const int parts = fits(8, MOEDC_PARTS_8) ? 8 : fits(4, MOEDC_PARTS_4) ? 4 : fits(2, MOEDC_PARTS_2) ? 2 : 1;
    clear_stale_error();
    launch_cluster(k, parts, (int)(units * parts < blocks ? units * parts : blocks), moedc::kMsThreads,
                   kFixed + (3 * (size_t)a.E + 1) * sizeof(int32_t), stream, a, parts, wmap, xmaps);
    return launch_status();
}

}  // namespace moedc_host
