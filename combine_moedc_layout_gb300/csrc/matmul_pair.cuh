// Products of packed expert rows on the 5th-generation tensor cores, by pairs of SMs.
//
// A pair (a cluster of two blocks) computes a tile of 256 x 256 with one instruction
// stream: block r of the pair brings rows 128 r .. of the left operand and half of the
// right one into its shared memory, and holds rows 128 r .. of the sums in its tensor
// memory.  So each operand byte is fetched once for a tile, and each SM's share is
// 32 KB for 512 clocks of products (a stage: 64 elements of the contracted axis).
//
//   kMmForward   left x (tokens), right W; both K-major
//   kMmDx        left dout (tokens), K-major; right W, whose contracted axis is its rows
//   kMmDw        left dout, right x: the contracted axis is the tokens of one expert
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

#include "matmul_store.cuh"
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
    constexpr int kElems = kMmBytes / 2;
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

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
matmul_pair_kernel(const __grid_constant__ MmArgs a, const __grid_constant__ CUtensorMap lmap,
                   const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap allmap)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMmThreads / kWarp];
    __shared__ uint64_t full[kMmStages], ready[kMmStages], empty[kMmStages], d_full[2], d_empty[2], done, never;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    constexpr int kElems = kMmBytes / 2;

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

    if (warp < 8) {
        // ---- epilogue
        if (a.wait_extra) mbar_wait(&never, 0, &s_abort);
        const int half = warp >> 2;
        const uint32_t d0 = tmem + ((uint32_t)((warp & 3) * kWarp) << 16);
        // the columns of the thread's four parts of 32
        const int c01 = a.gated ? half * 64 : half * 128, c23 = a.gated ? 128 + half * 64 : half * 128 + 64;
        uint8_t* buf = smem + kMmStages * kMmStage + warp * 2048;
        MvRing accs;
        for (int unit = pair; unit < units; unit += pairs) {
            const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
            // the warp's first row, and how many of its 32 there are
            const int first = rank * kMmHalf + (warp & 3) * kWarp;
            const int have = MODE == kMmDw ? a.M - u.m0 - first : u.m - first;
            const bool some = have > 0;
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
    } else if (warp == 8) {
        // ---- TMA: this block's rows of the left operand, its half of the right one
        MvRing ring;
        int issued = 0;
        bool stop = false;
        for (int unit = pair; unit < units && !stop; unit += pairs) {
            const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
            const int m = MODE == kMmDw ? kMmHalf : min(max(u.m - rank * kMmHalf, 0), kMmHalf);   // rows of this block
            const int r0 = u.r0 + rank * kMmHalf;
            auto left_bytes = [&](int rows) { return (rows + 31) / 32 * 32 * kMmBytes; };
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
                    if (lane == 0) {
                        if (m == kMmHalf) tma_2d_pair(left, &allmap, s * kElems, r0, at);
                        else
                            for (int i = 0; i < m; i += 32) tma_2d_pair(left + i * kMmBytes, &lmap, s * kElems, r0 + i, at);
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
            const uint32_t type = a.f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t major = (MODE == kMmDw ? 1u << 15 : 0u) | (MODE == kMmDw || MODE == kMmDx ? 1u << 16 : 0u);
            const uint32_t idesc = (1u << 4) | type | major | ((uint32_t)(kMmTile / 8) << 17) | ((uint32_t)(kMmTile / 16) << 24);
            for (int unit = pair; unit < units; unit += pairs) {
                const MmUnit u = mm_unit<MODE>(a, s_pre, s_beg, s_end, tiles, unit);
                for (int s = 0; s < u.ksteps; ++s) {
                    if (s == 0 && k++ >= 2) {
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
                            tc_mma_pair(tmem + accs.slot * kMmTile, l + p * (MODE == kMmDw ? 128 : 2),
                                                         r + p * (MODE == kMmDw || MODE == kMmDx ? 128 : 2), idesc,
                                                         p != 0 || s != 0);
                        }
                        tc_commit_pair(empty + ring.slot);
                        if (s == u.ksteps - 1) tc_commit_pair(d_full + accs.slot);
                    }
                    __syncwarp();
                    if (s == u.ksteps - 1) accs.next(2);
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
