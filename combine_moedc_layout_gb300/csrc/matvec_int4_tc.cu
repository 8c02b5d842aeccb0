// The 4-bit expert products on the 5th-generation tensor cores, for calls whose
// experts have many rows: there the products bound the call, not the weights' stream.
//
// Tile: 128 weight rows (with SwiGLU 64 gate and 64 up rows) x up to 64 rows of x; a
// stage is 256 channels of it.  The weights are the operand that tcgen05 takes from
// tensor memory: a thread of an unpacking warp owns one weight row, reads its 128
// bytes of the stage from shared memory (where TMA put them) and stores the nibbles,
// as f16 subnormals less their zero point, into the row's lane of tensor memory: nine
// operations for eight weights.  x is the shared-memory operand, K-major in the
// 128-byte swizzle, in the channel order that the unpacking leaves.  Its records lie by
// packed row, so that a unit's are a box of a tensor map: four instructions a stage,
// where gathers of four rows took 80 clocks each and made the stream of x the bound.
//
// Each group has an accumulator of its own (64 columns of binary32, four of them in
// turn), so that the scale stays outside the sum: a thread of an epilogue warp owns
// one weight row and half of the rows of x, reads the group's sums and adds
//   scale sum (q - z) x
// in binary32 into registers that live until the unit's end.
//
// Warps: 0-7 epilogue (0-3 the first 32 rows of x, 4-7 the others), 8-11 and 12-15
// unpacking (alternate stages, one buffer of tensor memory each), 16 TMA, 17 MMA.
// Tensor memory: columns 0-255 two buffers of weights, 256-511 four accumulators.
//
// A stage takes some 2300 clocks with groups of 128, which unpacking, products and
// epilogue share evenly; with groups of 64 the hand-overs of accumulators (some 600
// clocks each) are the longest.  128 rows x 7168 x 7168, groups of 128: 39.2 us, 335
// TFLOP/s, against 69 us of the warp tiles.
#include "matvec_int4_ring.cuh"

namespace moedc {

constexpr int kTcThreads = 18 * kWarp;
constexpr int kTcRows = 128;
constexpr int kTcN = 64;              // rows of x in a unit
constexpr int kTcHalf = kTcN / 2;     // of an epilogue warp
constexpr int kTcAccs = 256 / kTcN;
constexpr int kTcW = kTcRows * kMvChunk / 2;
constexpr int kTcX = kTcN * kMvChunk * 2;
constexpr int kTcFactors = kTcN * 16;  // 16 bytes of a record, the first four its factor
constexpr int kTcStage = kTcW + kTcX + kTcFactors;
// Warps that take alternate stages rely on the ring being that deep: one that skipped
// over a whole round of it could take the phase before last for the one it waits for.
constexpr int kTcStages = 4;
constexpr int kTcUp = 2 * 8 * 64 * 4; // SwiGLU's up rows, eight rows of x at a time
constexpr int kTcColumns = 512;

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b),
                 "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t at, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(at));
}

__device__ __forceinline__ void tma_2d(void* to, const CUtensorMap* map, int x, int y, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_u32(to)), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_3d(void* to, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_u32(to)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

// The same lane every time.
__device__ __forceinline__ bool tc_elect()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// K-major operand in the 128-byte swizzle: atoms of 8 rows x 128 bytes, 1024 bytes apart
__device__ __forceinline__ uint64_t tc_smem_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3fffu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// By a whole warp.  Its lanes may come out of a wait apart, and the loads and stores of
// tensor memory want them together.
__device__ __forceinline__ void mbar_wait_warp(uint64_t* b, int parity, volatile int* abort)
{
    mbar_wait(b, parity, abort);
    __syncwarp();
}

// One group's accumulator, times its scale, into the stage's sums of a thread's weight
// row.
template <int ROWS>
__device__ __forceinline__ void tc_accumulate(uint32_t d, float s, float (&part)[kTcHalf])
{
    float v[ROWS / 16][16];
#pragma unroll
    for (int h = 0; h < ROWS / 16; ++h) tc_ld16(d + h * 16, v[h]);
    tc_wait_ld();
#pragma unroll
    for (int h = 0; h < ROWS / 16; ++h) {
        // the values count from here: no use of them may be moved above the wait
#pragma unroll
        for (int j = 0; j < 16; ++j) asm volatile("" : "+f"(v[h][j]));
#pragma unroll
        for (int j = 0; j < 16; ++j) part[h * 16 + j] = fmaf(s, v[h][j], part[h * 16 + j]);
    }
}

template <int GROUP, typename S>
__global__ void __launch_bounds__(kTcThreads, 1)
matvec_int4_tc_kernel(const __grid_constant__ MatvecArgs a, const __grid_constant__ CUtensorMap wmap,
                      const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap fmap,
                      uint16_t* __restrict__ out)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kTcThreads / kWarp];
    __shared__ uint64_t full_w[kTcStages], empty_w[kTcStages], full_x[kTcStages], empty_x[kTcStages];
    __shared__ uint64_t a_full[2], a_empty[2], d_full[kTcAccs], d_empty[kTcAccs], done, never;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    constexpr int kGroups = kMvChunk / GROUP;
    using Scales = MvScales<GROUP, S, 1>;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int tile_n = a.swiglu ? kTcRows / 2 : kTcRows;
    const int tiles = (a.N + tile_n - 1) / tile_n;
    const int groups = a.Kd / GROUP;
    const int wrows = a.swiglu ? 2 * a.N : a.N;
    const int ksteps = (a.Kd + kMvChunk - 1) / kMvChunk;
    float* s_up = reinterpret_cast<float*>(smem + kTcStages * kTcStage);
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + kTcStages * kTcStage + kTcUp);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kTcStages; ++s) {
            mbar_init(full_w + s, 1);
            mbar_init(empty_w + s, 4);
            mbar_init(full_x + s, 1);
            mbar_init(empty_x + s, 9);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(a_full + b, 4);
            mbar_init(a_empty + b, 1);
        }
        for (int b = 0; b < kTcAccs; ++b) {
            mbar_init(d_full + b, 1);
            mbar_init(d_empty + b, 8);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "n"(kTcColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    pdl_enter();
    const bool over = mv_chunks<kTcThreads>(a, tiles, s_scan, s_pre, s_beg, s_end);   // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // stage i of the block: slot i % stages of the ring, weights' buffer i & 1; group k of
    // the block: accumulator k % kTcAccs
    if (warp < 8) {
        // ---- epilogue: weight row `row` of the tile, rows j0 .. j0 + 31 of x
        if (a.wait_extra) mbar_wait(&never, 0, &s_abort);
        const int row = (warp & 3) * kWarp + lane, j0 = (warp >> 2) * kTcHalf;
        const uint32_t d0 = tmem + ((uint32_t)((warp & 3) * kWarp) << 16) + 256 + j0;
        const bool whole = Scales::aligned_groups(a, groups);
        const int last = whole ? groups - kGroups : groups - 1;
        auto rows_of = [&](const MvUnit& u, typename Scales::Rows& r) __attribute__((always_inline)) {
            const int n = a.swiglu ? min(u.n0 + (row & 63), a.N - 1) + (row & 64 ? a.N : 0) : min(u.n0 + row, a.N - 1);
            const int64_t at = ((int64_t)u.e * wrows + n) * groups;
            r.s[0] = static_cast<const S*>(a.scales) + at;
        };
        MvRing ring, accs;
        int unit = blockIdx.x;
        if (unit < units) {
            MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            typename Scales::Rows rows;
            rows_of(u, rows);
            Scales now;
            now.load(rows, 0, groups, whole, false);
            while (unit < units) {
                unit += gridDim.x;
                MvUnit un = u;
                if (unit < units) un = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
                const int mine = u.m - j0;             // rows of x of this warp
                float acc[kTcHalf];
#pragma unroll
                for (int j = 0; j < kTcHalf; ++j) acc[j] = 0.0f;
                for (int s = 1; s <= ksteps; ++s) {
                    // the next stage's scales, those of the next unit's first stage at the end
                    Scales next = now;
                    if (s == ksteps) rows_of(un, rows);
                    const int q0 = s == ksteps ? 0 : min(s * kGroups, last);
                    next.load(rows, q0, groups - q0, whole, false);
                    mbar_wait_warp(full_x + ring.slot, ring.phase, &s_abort);
                    const float* f = reinterpret_cast<const float*>(smem + ring.slot * kTcStage + kTcW + kTcX) + j0 * 4;
                    float part[kTcHalf];
#pragma unroll
                    for (int j = 0; j < kTcHalf; ++j) part[j] = 0.0f;
                    const int have = min(kGroups, groups - (s - 1) * kGroups);
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        if (q >= have) break;
                        mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                        tc_fence_after();
                        if (mine > 16) tc_accumulate<32>(d0 + accs.slot * kTcN, now.scale(0, q), part);
                        else if (mine > 0) tc_accumulate<16>(d0 + accs.slot * kTcN, now.scale(0, q), part);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(d_empty + accs.slot);
                        accs.next(kTcAccs);
                    }
#pragma unroll
                    for (int j = 0; j < kTcHalf; ++j) acc[j] = fmaf(part[j], f[j * 4], acc[j]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty_x + ring.slot);
                    ring.next(kTcStages);
                    now = next;
                }
                // outputs: a warp's lanes are 32 neighbouring channels; 2^12 is the rest of the
                // records' scaling
#pragma unroll
                for (int j = 0; j < kTcHalf; ++j) acc[j] *= 4096.0f;
                const int n = u.n0 + (a.swiglu ? row & 63 : row);
                uint16_t* o = out + (int64_t)(u.r0 + j0) * a.N + n;
                if (!a.swiglu) {
#pragma unroll
                    for (int j = 0; j < kTcHalf; ++j)
                        if (j < mine && n < a.N) store16(o + (int64_t)j * a.N, acc[j], a.f16);
                } else {
                    // the up rows' warps hand theirs to the gate rows', eight rows of x at a time
                    float* up = s_up + (warp >> 2) * 8 * 64;
#pragma unroll
                    for (int j8 = 0; j8 < kTcHalf; j8 += 8) {
                        if (j8 >= mine) break;         // the same for the four warps of a barrier
                        asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory");
                        if (row >= 64) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) up[j * 64 + row - 64] = acc[j8 + j];
                        }
                        asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory");
                        if (row < 64 && n < a.N) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float v = acc[j8 + j];
                                if (j8 + j < mine)
                                    store16(o + (int64_t)(j8 + j) * a.N, v / (1.0f + expf(-v)) * up[j * 64 + row], a.f16);
                            }
                        }
                    }
                }
                u = un;
            }
        }
    } else if (warp < 16) {
        // ---- unpacking: set b of four warps takes the stages of buffer b
        const int b = (warp - 8) >> 2, quad = warp & 3;
        const int row = quad * kWarp + lane;
        const uint32_t to = tmem + ((uint32_t)(quad * kWarp) << 16) + b * 128;
        MvRing ring;
        int i = 0;
        const bool whole = Scales::aligned_groups(a, groups);
        uint32_t zero[Scales::zwords];
#pragma unroll
        for (int k = 0; k < Scales::zwords; ++k) zero[k] = 0x08080808u;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            const int n = a.swiglu ? min(u.n0 + (row & 63), a.N - 1) + (row & 64 ? a.N : 0) : min(u.n0 + row, a.N - 1);
            const uint8_t* z = a.zeros + ((int64_t)u.e * wrows + n) * groups;
            for (int s = 0; s < ksteps; ++s, ++i, ring.next(kTcStages)) {
                if ((i & 1) != b) continue;
                if (a.zeros) Scales::load_zeros(zero, z + s * kGroups, whole, groups - s * kGroups);
                mbar_wait_warp(full_w + ring.slot, ring.phase, &s_abort);
                const uint8_t* w = smem + ring.slot * kTcStage + row * 128;
                uint4 v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(w + ((c ^ (row & 7)) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_w + ring.slot);
                // the products of two stages ago have read this buffer
                if (i >= 2) mbar_wait_warp(a_empty + b, ((i >> 1) - 1) & 1, &s_abort);
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
                    uint32_t o[16];
                    const int g = c * 32 / GROUP;
                    const uint32_t z0 = ((zero[g / 4] >> (8 * (g % 4))) & 0xffu) * 0x00010001u;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // exact: subnormals of one exponent
                        o[4 * k] = sub_f16x2(q[k] & 0x000f000fu, z0);
                        o[4 * k + 1] = sub_f16x2(q[k] & 0x00f000f0u, z0 << 4);
                        o[4 * k + 2] = sub_f16x2((q[k] >> 8) & 0x000f000fu, z0);
                        o[4 * k + 3] = sub_f16x2((q[k] >> 8) & 0x00f000f0u, z0 << 4);
                    }
                    tc_st16(to + c * 16, o);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full + b);
            }
        }
    } else if (warp == 16) {
        // ---- TMA: the two halves of the tile's weight rows; x, 64 channels at a time, and
        // its factors.  Packed rows are neighbours: those past the unit's are of no account.
        int issued = 0;
        bool bad = false, lone = false;   // lone: weights under way without their x
        MvRing ring;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            if (__any_sync(0xffffffffu, s_abort != 0)) break;
            const MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            for (int r = lane; r < u.m; r += kWarp) x_row(a, u.r0 + r, bad);
            if (lane == 0) {   // the waits are of this one lane
                const int wrow = u.e * wrows + u.n0;
                for (int s = 0; s < ksteps; ++s) {
                    if (!mbar_wait(empty_w + ring.slot, ring.phase ^ 1, &s_abort)) break;
                    uint8_t* st = smem + ring.slot * kTcStage;
                    mbar_arrive_expect(full_w + ring.slot, kTcW);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        tma_2d(st + h * (kTcW / 2), &wmap, s * (kMvChunk / 2),
                               wrow + h * (a.swiglu ? a.N : kTcRows / 2), full_w + ring.slot);
                    if (!mbar_wait(empty_x + ring.slot, ring.phase ^ 1, &s_abort)) {
                        lone = true;
                        break;
                    }
                    mbar_arrive_expect(full_x + ring.slot, kTcX + kTcFactors);
                    st += kTcW;
                    // a record's rows in the maps are [row][stage]
#pragma unroll
                    for (int c = 0; c < kMvChunk / 64; ++c)
                        tma_3d(st + c * (kTcN * 128), &xmap, c * 64, s, u.r0, full_x + ring.slot);
                    tma_3d(st + kTcX, &fmap, kMvFactor / 2, s, u.r0, full_x + ring.slot);
                    ring.next(kTcStages);
                    ++issued;
                }
            }
            __syncwarp();
        }
        // no copy may land after the block has gone, whatever else gave up
        if (lane == 0) {
            for (int n = max(0, issued - kTcStages); n < issued + lone; ++n) {
                volatile int alone = 0;
                if (!mbar_wait(full_w + n % kTcStages, (n / kTcStages) & 1, &alone)) s_abort = 1;
                if (n < issued && !mbar_wait(full_x + n % kTcStages, (n / kTcStages) & 1, &alone)) s_abort = 1;
            }
        }
        __syncwarp();
        if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    } else {
        // ---- MMA: one elected lane issues; the warp stays together, so that the compiler
        // sees operands that are the same in all of it
        const bool leader = tc_elect();
        MvRing ring, accs;
        int i = 0, k = 0;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            // columns: as many rows of x as there are, by 16
            const uint32_t idesc = (1u << 4) | ((uint32_t)((u.m + 15) / 16 * 2) << 17) | ((uint32_t)(kTcRows / 16) << 24);
            for (int s = 0; s < ksteps; ++s, ++i) {
                const int b = i & 1;
                mbar_wait_warp(full_x + ring.slot, ring.phase, &s_abort);
                mbar_wait_warp(a_full + b, (i >> 1) & 1, &s_abort);
                tc_fence_after();
                const uint64_t x = tc_smem_desc(smem_u32(smem + ring.slot * kTcStage + kTcW));
                const uint32_t w = tmem + b * 128;
                const int have = min(kGroups, groups - s * kGroups);
#pragma unroll
                for (int q = 0; q < kGroups; ++q) {
                    if (q >= have) break;
                    if (k++ >= kTcAccs) {
                        mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                        tc_fence_after();
                    }
                    if (leader) {
#pragma unroll
                        for (int p = 0; p < GROUP / 16; ++p) {
                            const int st = q * (GROUP / 16) + p;
                            // a descriptor counts in 16 bytes
                            tc_mma(tmem + 256 + accs.slot * kTcN, w + st * 8,
                                   x + (((st >> 2) * (kTcN * 128) + (st & 3) * 32) >> 4), idesc, p != 0);
                        }
                        tc_commit(d_full + accs.slot);
                    }
                    __syncwarp();
                    accs.next(kTcAccs);
                }
                if (leader) {
                    tc_commit(a_empty + b);
                    tc_commit(empty_x + ring.slot);
                }
                __syncwarp();
                ring.next(kTcStages);
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
    if (warp == 17)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTcColumns) : "memory");
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {
namespace {

size_t tc_smem(int E)
{
    return (size_t)moedc::kTcStages * moedc::kTcStage + moedc::kTcUp + (3 * (size_t)E + 1) * sizeof(int32_t);
}
constexpr size_t kTcSmem = kMvSmem - 2048;

template <int GROUP, typename S>
int launch_tc(const moedc::MatvecArgs& a, void* out, cudaStream_t stream)
{
    auto* k = moedc::matvec_int4_tc_kernel<GROUP, S>;
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, (int)kTcSmem)) return MOEDC_ERR_CUDA;
    CUtensorMap map;
    if (!matvec_weight_map(&map, a.wq, a.Kd, (int64_t)a.E * (a.swiglu ? 2 : 1) * a.N, moedc::kTcRows / 2))
        return MOEDC_ERR_CUDA;
    CUtensorMap xmap, fmap;
    if (!matvec_x_maps(&xmap, &fmap, a.records, (a.Kd + moedc::kMvChunk - 1) / moedc::kMvChunk, a.rows, moedc::kTcN))
        return MOEDC_ERR_CUDA;
    const int tile_n = a.swiglu ? moedc::kTcRows / 2 : moedc::kTcRows;
    const int64_t most = ((int64_t)a.rows / moedc::kTcN + (a.E < a.rows ? a.E : a.rows)) * ((a.N + tile_n - 1) / tile_n);
    const int blocks = sm_count();
    clear_stale_error();
    launch(k, (int)(most < blocks ? most : blocks), moedc::kTcThreads, tc_smem(a.E), stream, a, map, xmap, fmap,
           static_cast<uint16_t*>(out));
    return launch_status();
}

template <typename S>
int launch_tc_group(const moedc::MatvecArgs& a, int group, void* out, cudaStream_t stream)
{
    return group == 64 ? launch_tc<64, S>(a, out, stream) : launch_tc<128, S>(a, out, stream);
}

}  // namespace

#ifndef MOEDC_TC_ROWS
#define MOEDC_TC_ROWS 20
#endif

// By rows an expert, as many as there can be: us of the warp tiles / of this kernel, with
// 8 experts of 2048 x 7168 and with 64 of them (rows not quite equal among experts):
//   rows             12         16         20         24         32         48
//   group 128, 8   36 / 37    45 / 37    46 / 39    47 / 39    70 / 39    70 / 41
//   group 128, 64 184 / 211  231 / 215  252 / 217  273 / 219  316 / 224  440 / 233
//   group 64, 8    39 / 48    49 / 49    49 / 49    49 / 49    79 / 51    80 / 51
//   group 64, 64  223 / 282  273 / 289  296 / 294  298 / 296  369 / 303  511 / 315
// and 32 experts of 1024 x 2048: group 128 26 / 25 at 16, 27 / 27 at 20, 45 / 27 at 32,
// group 64 29 / 32 at 20, 33 / 33 at 24, 51 / 33 at 32.  Many experts of few channels are
// the exception: 128 of 2 x 768 x 2048 with SwiGLU, group 128, 122 / 172 at 20, 174 / 200
// at 32.  Groups of 32 (eight accumulators a stage) 82 / 104 at 32 rows and
// 105 / 211 at 20: never.
bool matvec_tc_takes(int E, int rows, int group)
{
    const int64_t active = E < rows ? E : rows;
    return group >= 64 && tc_smem(E) <= kTcSmem && rows >= (group == 64 ? MOEDC_TC_ROWS + 4 : MOEDC_TC_ROWS) * active;
}

int launch_matvec_tc(const moedc::MatvecArgs& b, int group, void* out, cudaStream_t stream)
{
    moedc::MatvecArgs a = b;
    a.chunk_rows = moedc::kTcN;
    return a.scale_dtype == MOEDC_F32   ? launch_tc_group<float>(a, group, out, stream)
           : a.scale_dtype == MOEDC_F16 ? launch_tc_group<__half>(a, group, out, stream)
                                        : launch_tc_group<__nv_bfloat16>(a, group, out, stream);
}

}  // namespace moedc_host
