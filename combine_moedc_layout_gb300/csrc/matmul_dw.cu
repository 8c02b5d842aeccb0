// Gradient of 16-bit weights: dW = dout^T x for each expert, on the 5th-generation tensor
// cores, by pairs of SMs.
//
// A pair (a cluster of two blocks) computes a tile of 256 x 256 of one expert's dW with one
// instruction stream: block r brings columns 128 r .. of dout's 256 and of x's 256 into its
// shared memory, and holds rows 128 r .. of the sums in its tensor memory.  So each operand
// byte is fetched once for a tile, and each SM's share is 32 KB for 512 clocks of products
// (a stage: 64 tokens).  The contracted axis is the rows of both operands as they lie in
// memory.  An expert's tokens end anywhere: the rows behind them, which are another
// expert's, are cleared in shared memory as far as the products reach, by copies of boxes that
// lie behind the tensor's end and so are zeros.  They count at the barrier of the first block's
// thread that issues the products.  Stores by threads of the second block would need a release of
// the cluster's scope: 64 experts of 517 tokens x 2048 x 2048 240 us, 208 so, 200 with stores in
// no order that the memory model knows.
//
// A sum in tensor memory loses up to an ulp, always towards zero, with each product of 16
// tokens: some 4e-8 of it a step for values of random signs, 1e-7 for those of one sign, 5e-5
// over 8192 tokens, which binary32 gradients would show, and half a step of f16 over 80000.  So
// tokens are summed in pieces, of 768 for binary32 and of 8192 for 16 bits, which the epilogue
// adds up, rounding to nearest.
// (A piece is also what the epilogue's bounded wait waits for.)
//
// 32 experts of 512 tokens x 4096 x 4096: 357 us, 1540 TFLOP/s, stores and products together;
// 60 of 64 x 1024 x 1024: 34 us, the stores (4.4 TB/s); binary32, 64 of 512 x 7168 x 2048: 850 us
// (815 to 890).
//
// Warps: 0-7 epilogue (0-3 the first half of the columns, 4-7 the others), 8 TMA, 9 MMA (of
// the pair's first block, for both), 10 tells the first block that a stage has arrived, and
// clears.  Tensor memory: two sums of 256 columns.
#include "matmul_store.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace moedc {

constexpr int kMmThreads = 11 * kWarp;
constexpr int kMmEpilogue = 8 * kWarp;
constexpr int kMmTile = 256;                    // of the pair, both ways
constexpr int kMmHalf = kMmTile / 2;
constexpr int kMmElems = 64;                    // tokens of a stage
constexpr int kMmPiece = 12;                    // stages of one sum, of binary32 gradients
constexpr int kMmPiece16 = 128;                 // of 16-bit ones
constexpr int kMmBytes = 128;                   // of a row of a box
constexpr int kMmOperand = kMmHalf * kMmBytes;  // a block's share of one operand
constexpr int kMmStage = 2 * kMmOperand;
constexpr int kMmStages = 6;
constexpr int kMmBuf = 8 * 2048;                 // of the epilogue's warps, for their stores
constexpr int kMmColumns = 512;

struct DwUnit {
    int e, r0, m;       // expert, its first row and rows
    int m0, n0;         // first row and column of the output
    int ksteps, piece;  // stages, and those of one sum
};

__device__ __forceinline__ DwUnit dw_unit(const MmArgs& a, const int32_t* s_beg, const int32_t* s_end, int tiles, int mtiles, int unit)
{
    DwUnit u;
    u.e = unit / (tiles * mtiles);
    int t, c;
    mm_order(unit - u.e * tiles * mtiles, tiles, mtiles, t, c);
    u.n0 = t * kMmTile;
    u.m0 = c * kMmTile;
    u.r0 = s_beg[u.e];
    u.m = s_end[u.e] - u.r0;
    u.ksteps = u.m / kMmElems + (u.m % kMmElems != 0);   // (sizes go up to INT_MAX)
    u.piece = a.f32 ? kMmPiece : kMmPiece16;
    return u;
}

// Rows behind the expert's last one that the products of stage s reach: up to the end of their 16.
__device__ __forceinline__ int dw_clears(const DwUnit& u, int s) { return s == u.ksteps - 1 ? (16 - u.m % 16) % 16 : 0; }

// Whether a 16-bit sum has several pieces.  By a whole warp.
__device__ __forceinline__ bool dw_pieces(const MmArgs& a, const int32_t* s_beg, const int32_t* s_end)
{
    int most = 0;
    if (a.rows > kMmPiece16 * kMmElems)
        for (int e = threadIdx.x % kWarp; e < a.E; e += kWarp) most = max(most, s_end[e] - s_beg[e]);
    return __reduce_max_sync(0xffffffffu, most) > kMmPiece16 * kMmElems;
}

template <bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
matmul_dw_kernel(const __grid_constant__ MmArgs a, const __grid_constant__ CUtensorMap lmap,
                 const __grid_constant__ CUtensorMap rmap, const __grid_constant__ BoxMaps zeros)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMmThreads / kWarp];
    __shared__ uint64_t full[kMmStages], ready[kMmStages], empty[kMmStages], d_full[2], d_empty[2], done, never;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int tiles = (a.N - 1) / kMmTile + 1, mtiles = (a.M - 1) / kMmTile + 1;
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
    const bool over = mm_chunks<kMmThreads>(a, kMmTile, 1, s_scan, s_pre, s_beg, s_end);
    cluster_sync();   // the other block's barriers stand
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = a.E * tiles * mtiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    if (warp < 8) {
        // ---- epilogue
        if (a.wait_extra) mbar_wait(&never, 0, &s_abort);
        const int half = warp >> 2;
        const uint32_t d0 = tmem + ((uint32_t)((warp & 3) * kWarp) << 16);
        uint8_t* buf = smem + kMmStages * kMmStage + warp * 2048;
        // 16 bits: a loop of its own for calls in which an expert has several pieces.  In one with
        // the other it made that slower (60 x 64 x 1024 x 1024: 33.4 -> 35.1 us).
        auto tiles_of = [&](auto pieces) __attribute__((always_inline)) {
            constexpr bool kPieces = decltype(pieces)::value;
            MvRing accs;
            for (int unit = pair; unit < units; unit += pairs) {
                const DwUnit u = dw_unit(a, s_beg, s_end, tiles, mtiles, unit);
                // the warp's first row, and how many of its 32 there are
                const int first = rank * kMmHalf + (warp & 3) * kWarp;
                const int have = a.M - u.m0 - first;
                const bool some = have > 0;
                if (kPieces && u.ksteps > u.piece) {
                    float acc[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[c][j] = 0.0f;
                    for (int s = 0; s < u.ksteps; s += u.piece) {
                        mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                        tc_fence_after();
                        if (some) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                float v[16];
                                tc_ld16(d0 + accs.slot * kMmTile + half * 128 + c * 16, v);
                                tc_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[j]));
#pragma unroll
                                for (int j = 0; j < 16; ++j) acc[c / 2][c % 2 * 16 + j] += v[j];
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, 0);
                        accs.next(2);
                    }
                    const int64_t at = ((int64_t)u.e * a.M + u.m0 + first) * a.N;
                    if (some) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int n = u.n0 + half * 128 + c * 32;
                            if (n >= a.N) break;
                            if constexpr (kF32) mm_store32(buf, static_cast<float*>(a.out) + at, a.N, n, a.N, have, acc[c]);
                            else mm_store32(buf, static_cast<uint16_t*>(a.out) + at, a.N, n, a.N, have, true, a.f16, acc[c]);
                        }
                    }
                    continue;
                }
                const bool any = u.ksteps > 0;
                if (any) {
                    mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                    tc_fence_after();
                }
                const uint32_t d = d0 + accs.slot * kMmTile;
                const int64_t at = ((int64_t)u.e * a.M + u.m0 + first) * a.N;
                if (some) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int n = u.n0 + half * 128 + c * 32;
                        if (n >= a.N) break;
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
                        if constexpr (kF32) mm_store32(buf, static_cast<float*>(a.out) + at, a.N, n, a.N, have, v);
                        else mm_store32(buf, static_cast<uint16_t*>(a.out) + at, a.N, n, a.N, have, true, a.f16, v);
                    }
                }
                if (any) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, 0);
                    accs.next(2);
                }
            }
        };
        if (kF32 || dw_pieces(a, s_beg, s_end)) tiles_of(std::true_type());
        else tiles_of(std::false_type());
    } else if (warp == 8) {
        // ---- TMA: this block's rows of the left operand, its half of the right one
        // (one lane waits and issues)
        MvRing ring;
        int issued = 0;
        bool stop = !tc_elect();
        for (int unit = pair; unit < units && !stop; unit += pairs) {
            const DwUnit u = dw_unit(a, s_beg, s_end, tiles, mtiles, unit);
            for (int s = 0; s < u.ksteps; ++s) {
                if (!mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort)) {
                    stop = true;
                    break;
                }
                uint8_t* left = smem + ring.slot * kMmStage;
                uint8_t* right = left + kMmOperand;
                uint64_t* bar = full + ring.slot;
                mbar_arrive_expect(bar, kMmStage);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tma_2d(left + h * (kMmOperand / 2), &lmap, u.m0 + rank * kMmHalf + h * 64, u.r0 + s * kMmElems, bar);
                    tma_2d(right + h * (kMmOperand / 2), &rmap, u.n0 + rank * kMmHalf + h * 64, u.r0 + s * kMmElems, bar);
                }
                ring.next(kMmStages);
                ++issued;
            }
        }
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - kMmStages); n < issued; ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % kMmStages, (n / kMmStages) & 1, &alone)) s_abort = 1;
        }
        __syncwarp();
        // the last product's arrival at the second block; the wait begins behind the block's last
        // copy, as its bound is one of a step and not of the call
        if (rank == 1) {
            volatile int alone = 0;
            if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- MMA, for both blocks: one elected lane issues; the warp stays together
        if (rank == 0) {
            const bool leader = tc_elect();
            MvRing ring, accs;
            int k = 0;
            const uint32_t type = a.f16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t major = (1u << 15) | (1u << 16);
            const uint32_t idesc = (1u << 4) | type | major | ((uint32_t)(kMmTile / 8) << 17) | ((uint32_t)(kMmTile / 16) << 24);
            for (int unit = pair; unit < units; unit += pairs) {
                const DwUnit u = dw_unit(a, s_beg, s_end, tiles, mtiles, unit);
                int in = 0;     // stage of the sum
                for (int s = 0; s < u.ksteps; ++s) {
                    if (in == 0 && k++ >= 2) mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                    const bool last = in == u.piece - 1 || s == u.ksteps - 1;
                    mbar_wait_warp(ready + ring.slot, ring.phase, &s_abort);
                    tc_fence_after();
                    const uint32_t left = smem_u32(smem + ring.slot * kMmStage);
                    const uint64_t l = tc_smem_desc_mn(left, kMmOperand / 2), r = tc_smem_desc_mn(left + kMmOperand, kMmOperand / 2);
                    // 16 tokens each, as far as there are some
                    const int steps = min(4, (u.m - s * kMmElems + 15) / 16);
                    if (leader) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            if (p >= steps) break;
                            // a descriptor counts in 16 bytes: 16 rows of 128
                            tc_mma_pair(tmem + accs.slot * kMmTile, l + p * 128, r + p * 128, idesc, p != 0 || in != 0);
                        }
                        tc_commit_pair(empty + ring.slot);
                        if (last) tc_commit_pair(d_full + accs.slot);
                    }
                    __syncwarp();
                    if (last) accs.next(2);
                    in = last ? 0 : in + 1;
                    ring.next(kMmStages);
                }
            }
            // tensor memory is given back only when the last product is through
            if (leader) tc_commit_pair(&done);
            __syncwarp();
            volatile int alone = 0;
            if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        }
        __syncwarp();
    } else {
        // ---- stages that have arrived in this block
        MvRing ring;
        for (int unit = pair; unit < units; unit += pairs) {
            const DwUnit u = dw_unit(a, s_beg, s_end, tiles, mtiles, unit);
            for (int s = 0; s < u.ksteps; ++s) {
                mbar_wait_warp(full + ring.slot, ring.phase, &s_abort);
                const int n = dw_clears(u, s);
                if (n > 0) {
                    // two boxes of 1, 2, 4 or 8 rows, which may overlap, in each of the four boxes of data
                    const int log = 31 - __clz(n), rows = 1 << log, have = u.m - s * kMmElems;
                    if (lane < 8) {
                        const int row = lane & 1 ? have : have + n - rows;
                        tma_2d_pair(smem + ring.slot * kMmStage + lane / 2 * (kMmOperand / 2) + row * kMmBytes, zeros.by + log, 0,
                                    a.rows, cluster_addr(ready + ring.slot, 0));
                    }
                    __syncwarp();
                    // (those of both blocks)
                    if (lane == 0 && rank == 0) mbar_arrive_expect(ready + ring.slot, 2 * 8 * rows * kMmBytes);
                }
                if (lane == 0 && (rank == 1 || n == 0)) mbar_arrive_pair(ready + ring.slot, 0);
                ring.next(kMmStages);
            }
        }
        // zeros on their way that nobody waits for any more have a millisecond
        if (s_abort)
            for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < 1000000ull;) {}
        __syncwarp();
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

namespace {

template <bool kF32>
int launch_dw(const moedc::MmArgs& a, const CUtensorMap& l, const CUtensorMap& r, const moedc::BoxMaps& zeros, cudaStream_t stream)
{
    auto* k = moedc::matmul_dw_kernel<kF32>;
    constexpr size_t kFixed = moedc::kMmStages * moedc::kMmStage + moedc::kMmBuf;
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, (int)kFixed + (3 * MOEDC_MAX_E + 1) * 4)) return MOEDC_ERR_CUDA;
    const int64_t units = a.E * ((a.N + (int64_t)moedc::kMmTile - 1) / moedc::kMmTile) * ((a.M + (int64_t)moedc::kMmTile - 1) / moedc::kMmTile);
    const int pairs = sm_count() / 2;
    clear_stale_error();
    launch(k, 2 * (int)(units < pairs ? units : pairs), moedc::kMmThreads, kFixed + (3 * (size_t)a.E + 1) * sizeof(int32_t), stream, a, l,
           r, zeros);
    return launch_status();
}

}  // namespace

int launch_mm_dw(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* x, int64_t ldx, cudaStream_t stream)
{
    CUtensorMap l, r;
    moedc::BoxMaps zeros{};
    if (!map_rows16(&l, dout, a.M, a.rows, ldd, moedc::kMmElems) || !map_rows16(&r, x, a.N, a.rows, ldx, moedc::kMmElems))
        return MOEDC_ERR_CUDA;
    for (int i = 0; i < 4; ++i) {
        const cuuint64_t size[2] = {(cuuint64_t)a.M, (cuuint64_t)a.rows}, stride[1] = {(cuuint64_t)ldd * 2};
        const cuuint32_t box[2] = {moedc::kMmBytes / 2, 1u << i};
        if (!tensor_map(zeros.by + i, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_NONE, dout, 2, size, stride, box))
            return MOEDC_ERR_CUDA;
    }
    return a.f32 ? launch_dw<true>(a, l, r, zeros, stream) : launch_dw<false>(a, l, r, zeros, stream);
}

}  // namespace moedc_host
