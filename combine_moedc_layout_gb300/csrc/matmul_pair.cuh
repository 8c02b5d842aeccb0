// Products of packed expert rows on the 5th-generation tensor cores, by pairs of SMs.
//
// A pair (a cluster of two blocks) computes a tile of 256 x 256 with one instruction
// stream: block r of the pair brings rows 128 r .. of the left operand and half of the
// right one into its shared memory, and holds rows 128 r .. of the sums in its tensor
// memory.  So each operand byte is fetched once for a tile, and each SM's share is
// 32 KB for 512 clocks of products (a stage: 128 bytes of the contracted axis, that is
// 64 16-bit or 128 8-bit elements).
//
//   kMmForward   left x (tokens), right W; both K-major
//   kMmDx        left dout (tokens), K-major; right W, whose contracted axis is its rows
//   kMmDw        left dout, right x: the contracted axis is the tokens of one expert
//   kMmE4m3      as kMmForward in e4m3, a sum of its own for each 128 channels: the
//                epilogue's threads, a token each, add them with their two scales
//
// With `gated`, the right operand's first half are gate rows, its second half the up rows
// of the same channels, so that a thread finds both products of a channel in its own lane
// of tensor memory.
//
// Warps: 0-7 epilogue (0-3 the first half of the columns, or of the channels, 4-7 the
// rest), 8 TMA, 9 MMA (of the pair's first block, for both), 10 (kMmDw) clears what a stage
// of tokens holds of the next expert and tells the first block that it has arrived; in the
// other forms the copies of both blocks count at the first one's barrier.
// Tensor memory: two sums of 256 columns.
#pragma once

#include "matmul.cuh"
#include "tcgen05.cuh"

namespace moedc {

constexpr int kMmThreads = 12 * kWarp;
constexpr int kMmEpilogue = 8 * kWarp;
constexpr int kMmTile = 256;                    // of the pair, both ways
constexpr int kMmHalf = kMmTile / 2;
constexpr int kMmBytes = 128;                   // of the contracted axis in a stage
constexpr int kMmOperand = kMmHalf * kMmBytes;  // a block's share of one operand
constexpr int kMmStage = 2 * kMmOperand;
constexpr int kMmStages = 6;
constexpr int kMmBuf = 8 * 2048;                 // of the epilogue's warps, for their stores
constexpr int kMmColumns = 512;

struct MmUnit {
    int e, r0, m;       // expert, first row and rows (kMmDw: all of the expert's)
    int n0;             // first column of the output
    int m0;             // kMmDw: first row of the output
    int ksteps;
};

template <int MODE>
__device__ __forceinline__ MmUnit mm_unit(const MmArgs& a, const int32_t* s_pre, const int32_t* s_beg,
                                          const int32_t* s_end, int tiles, int unit)
{
    constexpr int kElems = MODE == kMmE4m3 ? kMmBytes : kMmBytes / 2;
    MmUnit u;
    if constexpr (MODE == kMmDw) {
        const int mtiles = (a.M + kMmTile - 1) / kMmTile;
        u.e = unit / (tiles * mtiles);
        const int in = unit - u.e * tiles * mtiles, t = in / mtiles;
        u.n0 = t * kMmTile;
        u.m0 = (in - t * mtiles) * kMmTile;
        u.r0 = s_beg[u.e];
        u.m = s_end[u.e] - u.r0;
        u.ksteps = (u.m + kElems - 1) / kElems;
    } else {
        int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if ((int64_t)s_pre[mid] * tiles <= unit) lo = mid; else hi = mid - 1;
        }
        const int chunks = s_pre[lo + 1] - s_pre[lo];
        const int in = unit - s_pre[lo] * tiles;
        const int t = in / chunks;
        u.e = lo;
        u.n0 = t * (a.gated ? kMmHalf : kMmTile);
        u.r0 = s_beg[lo] + (in - t * chunks) * kMmTile;
        u.m = min(kMmTile, s_end[lo] - u.r0);
        u.m0 = 0;
        u.ksteps = (a.K + kElems - 1) / kElems;
    }
    return u;
}

// Row of x of packed row r; -1 where there is none.
__device__ __forceinline__ int mm_x_row(const MmArgs& a, int r)
{
    if (!a.src) return r;
    const int i = __ldg(a.src + r);
    const int t = i < 0 ? -1 : i / a.top_k;
    return t < a.x_rows ? t : -1;
}

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
        mm_store_rows(buf, q, reinterpret_cast<uint8_t*>(out + n), 2 * ld, rows, 2 * (N - n));
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
        mm_store_rows(buf, q, reinterpret_cast<uint8_t*>(out + n + h), 4 * ld, rows, 4 * (N - n - h));
    }
}

__device__ __forceinline__ float mm_silu_mul(float g, float u)
{
    float s, rest;
    sigmoid_both(g, s, rest);
    return g * s * u;
}

__device__ __forceinline__ float ld_scale(const float* p)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
matmul_pair_kernel(const __grid_constant__ MmArgs a, const __grid_constant__ CUtensorMap lmap,
                   const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap allmap)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMmThreads / kWarp];
    __shared__ uint64_t full[kMmStages], ready[kMmStages], empty[kMmStages], d_full[2], d_empty[2], done, never;
    __shared__ float s_amax[2][kMmHalf];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    constexpr int kElems = MODE == kMmE4m3 ? kMmBytes : kMmBytes / 2;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int tiles = (a.N + (a.gated ? kMmHalf : kMmTile) - 1) / (a.gated ? kMmHalf : kMmTile);
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + kMmStages * kMmStage + kMmBuf);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMmStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(ready + s, 2);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(d_full + b, 1);
            mbar_init(d_empty + b, 2 * kMmEpilogue / kWarp);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        tc_alloc_pair(&s_tmem, kMmColumns);
        tc_fence_before();
    }
    pdl_enter();
    const bool over = mm_chunks<kMmThreads>(a, kMmTile, tiles, s_scan, s_pre, s_beg, s_end);
    cluster_sync();   // the other block's barriers stand
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = MODE == kMmDw ? a.E * tiles * ((a.M + kMmTile - 1) / kMmTile) : s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // kMmE4m3: the epilogue's threads keep 128 sums each.  The shares add up to the launch's
    // 384 x 168 registers: 256 x 232 + 128 x 40.
    if constexpr (MODE == kMmE4m3) {
        if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    }
    if (warp < 8) {
        // ---- epilogue
        // (no calls in kMmE4m3's epilogue: with one the registers do not compile to a share)
        if (a.wait_extra) mbar_wait_inline(&never, 0, &s_abort);
        const int half = warp >> 2;
        const uint32_t d0 = tmem + ((uint32_t)((warp & 3) * kWarp) << 16);
        // the columns of the thread's four parts of 32
        const int c01 = a.gated ? half * 64 : half * 128, c23 = a.gated ? 128 + half * 64 : half * 128 + 64;
        uint8_t* buf = smem + kMmStages * kMmStage + warp * 2048;
        MvRing accs;
        bool bad = false;
        for (int unit = pair; unit < units; unit += pairs) {
            const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
            // the warp's first row, and how many of its 32 there are
            const int first = rank * kMmHalf + (warp & 3) * kWarp;
            const int have = MODE == kMmDw ? a.M - u.m0 - first : u.m - first;
            const bool some = have > 0, mine = lane < have;
            const int r = u.r0 + first + lane;             // MODE != kMmDw
            if constexpr (MODE == kMmE4m3) {
                float2 acc[64];
#pragma unroll
                for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.0f, 0.0f);
                int xr = mine ? mm_x_row(a, r) : 0;
                const bool lost = xr < 0;
                bad |= lost;
                if (lost) xr = 0;
                const float* xs = a.xs + (a.offsets || !a.counts || a.src ? xr * a.xs_r
                                              : u.e * a.xs_e + (mine ? r - u.e * a.slots : 0) * a.xs_r);
                const int groups = u.ksteps, blocks = (a.N + 127) / 128;
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
                        const uint32_t d = d0 + accs.slot * kMmTile;
                        auto release = [&]() __attribute__((always_inline)) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, 0);
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
                if (lost) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.0f, 0.0f);
                }
                float* v = reinterpret_cast<float*>(acc);
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
                                    w[i] = pack_e4m3x2(__fdiv_rn(f[0], sc), __fdiv_rn(f[1], sc)) |
                                           pack_e4m3x2(__fdiv_rn(f[2], sc), __fdiv_rn(f[3], sc)) << 16;
                                }
                                q[k] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            mm_store_rows(buf, q, o + h, a.N, have, 64);
                        }
                        if (mine && (!a.gated || half == 0))
                            static_cast<float*>(a.extra)[(int64_t)r * (a.N / 128) + n / 128] = sc;
                    }
                }
            } else {
                const bool any = u.ksteps > 0;
                if (any) {
                    mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                    tc_fence_after();
                }
                const uint32_t d = d0 + accs.slot * kMmTile;
                const int64_t at = MODE == kMmDw ? (int64_t)u.e * a.M + u.m0 + first : u.r0 + first;
                uint16_t* o = static_cast<uint16_t*>(a.out) + at * a.N;
                if (MODE == kMmForward && a.gated) {
                    if (some) {
                        uint16_t* keep = static_cast<uint16_t*>(a.extra) + at * 2 * a.N;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float g[32], v[32];
                            tc_ld32(d + c01 + c * 32, g);
                            tc_ld32(d + c23 + c * 32, v);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                asm volatile("" : "+f"(g[j]));
                                asm volatile("" : "+f"(v[j]));
                            }
                            const int n = u.n0 + half * 64 + c * 32;
                            if (a.extra) {
                                mm_store32(buf, keep, 2 * (int64_t)a.N, n, a.N, have, true, a.f16, g);
                                mm_store32(buf, keep + a.N, 2 * (int64_t)a.N, n, a.N, have, true, a.f16, v);
                            }
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = mm_silu_mul(g[j], v[j]);
                            mm_store32(buf, o, a.N, n, a.N, have, true, a.f16, v);
                        }
                    }
                } else if (some) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float v[32];
                        if (any) {
                            tc_ld32(d + half * 128 + c * 32, v);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(v[j]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = 0.0f;   // an expert without rows
                        }
                        const int n = u.n0 + half * 128 + c * 32;
                        if (MODE == kMmDw && a.f32) mm_store32(buf, static_cast<float*>(a.out) + at * a.N, a.N, n, a.N, have, v);
                        else mm_store32(buf, o, a.N, n, a.N, have, true, a.f16, v);
                    }
                }
                if (any) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, 0);
                    accs.next(2);
                }
            }
        }
        if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    } else if (warp == 8) {
        // ---- TMA: this block's rows of the left operand, its half of the right one
        MvRing ring;
        int issued = 0;
        bool stop = false;
        for (int unit = pair; unit < units && !stop; unit += pairs) {
            const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
            const int m = MODE == kMmDw ? kMmHalf : min(max(u.m - rank * kMmHalf, 0), kMmHalf);   // rows of this block
            const int r0 = u.r0 + rank * kMmHalf;
            const bool gather = MODE == kMmE4m3 && a.src;
            int t[4] = {0, 0, 0, 0};
            if (gather) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane * 4 + i < m) t[i] = max(mm_x_row(a, r0 + lane * 4 + i), 0);
            }
            auto left_bytes = [&](int rows) { return (gather ? (rows + 3) / 4 * 4 : (rows + 31) / 32 * 32) * kMmBytes; };
            // kMmDw: what this block brings, counted here; else that of both, at the first block
            const int bytes = MODE == kMmDw ? kMmStage
                                            : 2 * kMmOperand + left_bytes(min(u.m, kMmHalf)) + left_bytes(max(u.m - kMmHalf, 0));
            for (int s = 0; s < u.ksteps; ++s) {
                const bool ok = mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort);
                if (__any_sync(0xffffffffu, !ok)) {
                    stop = true;
                    break;
                }
                uint8_t* left = smem + ring.slot * kMmStage;
                uint8_t* right = left + kMmOperand;
                uint64_t* bar = full + ring.slot;
                if constexpr (MODE == kMmDw) {
                    if (lane == 0) {
                        mbar_arrive_expect(bar, bytes);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            tma_2d(left + h * (kMmOperand / 2), &lmap, u.m0 + rank * kMmHalf + h * 64, u.r0 + s * kElems, bar);
                            tma_2d(right + h * (kMmOperand / 2), &rmap, u.n0 + rank * kMmHalf + h * 64, u.r0 + s * kElems, bar);
                        }
                    }
                } else {
                    const uint32_t at = cluster_addr(bar, 0);
                    if (lane == 0 && rank == 0) mbar_arrive_expect(bar, bytes);
                    __syncwarp();
                    if (gather && lane * 4 < m)
                        tma_gather4_pair(left + lane * 4 * kMmBytes, &lmap, s * kElems, t[0], t[1], t[2], t[3], at);
                    if (lane == 0) {
                        if (!gather) {
                            if (m == kMmHalf) tma_2d_pair(left, &allmap, s * kElems, r0, at);
                            else
                                for (int i = 0; i < m; i += 32) tma_2d_pair(left + i * kMmBytes, &lmap, s * kElems, r0 + i, at);
                        }
                        if constexpr (MODE == kMmDx) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                tma_3d_pair(right + h * (kMmOperand / 2), &rmap, u.n0 + rank * kMmHalf + h * 64, s * kElems, u.e, at);
                        } else {
                            // [E][1 or 2][N][K]
                            tma_4d_pair(right, &rmap, s * kElems, u.n0 + (a.gated ? 0 : rank * kMmHalf), a.gated ? rank : 0, u.e, at);
                        }
                    }
                }
                __syncwarp();
                ring.next(kMmStages);
                ++issued;
            }
        }
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - kMmStages); n < issued && (MODE == kMmDw || rank == 0); ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % kMmStages, (n / kMmStages) & 1, &alone)) s_abort = 1;
        }
        // a second block that gave up sees no barrier of its copies: they have a millisecond
        if (s_abort)
            for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < 1000000ull;) {}
        __syncwarp();
    } else if (warp == 9) {
        // ---- MMA, for both blocks: one elected lane issues; the warp stays together
        if (rank == 0) {
            const bool leader = tc_elect();
            MvRing ring, accs;
            int k = 0;
            const uint32_t type = MODE == kMmE4m3 || a.f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t major = (MODE == kMmDw ? 1u << 15 : 0u) | (MODE == kMmDw || MODE == kMmDx ? 1u << 16 : 0u);
            const uint32_t idesc = (1u << 4) | type | major | ((uint32_t)(kMmTile / 8) << 17) | ((uint32_t)(kMmTile / 16) << 24);
            for (int unit = pair; unit < units; unit += pairs) {
                const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
                for (int s = 0; s < u.ksteps; ++s) {
                    if ((MODE == kMmE4m3 || s == 0) && k++ >= 2) {
                        mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                    }
                    mbar_wait_warp((MODE == kMmDw ? ready : full) + ring.slot, ring.phase, &s_abort);
                    tc_fence_after();
                    const uint32_t left = smem_u32(smem + ring.slot * kMmStage);
                    const uint64_t l = MODE == kMmDw ? tc_smem_desc_mn(left, kMmOperand / 2) : tc_smem_desc(left);
                    const uint64_t r = MODE == kMmDw || MODE == kMmDx ? tc_smem_desc_mn(left + kMmOperand, kMmOperand / 2)
                                                                     : tc_smem_desc(left + kMmOperand);
                    // 32 bytes of the contracted axis each; rows of tokens only as far as there are some
                    const int steps = MODE == kMmDw ? min(4, (u.m - s * kElems + 15) / 16) : 4;
                    if (leader) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            if (p >= steps) break;
                            // a descriptor counts in 16 bytes: 32 of a row, or 16 rows of 128
                            tc_mma_pair<MODE == kMmE4m3>(tmem + accs.slot * kMmTile, l + p * (MODE == kMmDw ? 128 : 2),
                                                         r + p * (MODE == kMmDw || MODE == kMmDx ? 128 : 2), idesc,
                                                         p != 0 || (MODE != kMmE4m3 && s != 0));
                        }
                        tc_commit_pair(empty + ring.slot);
                        if (MODE == kMmE4m3 || s == u.ksteps - 1) tc_commit_pair(d_full + accs.slot);
                    }
                    __syncwarp();
                    if (MODE == kMmE4m3 || s == u.ksteps - 1) accs.next(2);
                    ring.next(kMmStages);
                }
            }
            // tensor memory is given back only when the last product is through
            if (leader) tc_commit_pair(&done);
            __syncwarp();
        }
        volatile int alone = 0;
        if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        __syncwarp();
    } else if (MODE == kMmDw && warp == 10) {
        // ---- stages that have arrived in this block
        MvRing ring;
        for (int unit = pair; unit < units; unit += pairs) {
            const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
            for (int s = 0; s < u.ksteps; ++s) {
                mbar_wait_warp(full + ring.slot, ring.phase, &s_abort);
                bool cleared = false;
                if constexpr (MODE == kMmDw) {
                    // rows behind the expert's last one, up to the end of their 16: a row is 128
                    // bytes of each of the four boxes, in whatever order
                    const int have = u.m - s * kElems, to = min((have + 15) / 16 * 16, kElems);
                    cleared = have < to;
                    if (cleared) {
                        for (int i = lane; i < (to - have) * 32; i += kWarp) {
                            const int box = i & 3, chunk = (i >> 2) & 7, row = have + (i >> 5);
                            *reinterpret_cast<uint4*>(smem + ring.slot * kMmStage + box * (kMmOperand / 2) + row * kMmBytes +
                                                      chunk * 16) = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    if (cleared) mbar_arrive_pair_release(ready + ring.slot, 0);
                    else mbar_arrive_pair(ready + ring.slot, 0);
                }
                ring.next(kMmStages);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (warp == 9) tc_free_pair(tmem, kMmColumns);
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {

template <int MODE>
int launch_mm_pair(const moedc::MmArgs& a, int64_t units, const CUtensorMap& lmap, const CUtensorMap& rmap,
                   const CUtensorMap& allmap, cudaStream_t stream)
{
    auto* k = moedc::matmul_pair_kernel<MODE>;
    const size_t smem = (size_t)moedc::kMmStages * moedc::kMmStage + moedc::kMmBuf + (3 * (size_t)a.E + 1) * sizeof(int32_t);
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, moedc::kMmStages * moedc::kMmStage + moedc::kMmBuf + (3 * MOEDC_MAX_E + 1) * 4))
        return MOEDC_ERR_CUDA;
    const int pairs = sm_count() / 2;
    clear_stale_error();
    launch(k, 2 * (int)(units < pairs ? units : pairs), moedc::kMmThreads, smem, stream, a, lmap, rmap, allmap);
    return launch_status();
}

}  // namespace moedc_host
