// Products of packed expert rows with 16-bit weights, and the rows' gradient, on the
// 5th-generation tensor cores, by pairs of SMs.
//
// The weights lie on the rows of the tile and the tokens on its columns, as many (in
// 32s, up to 256) as there are, so that experts of uneven sizes cost what they hold.  A
// pair (a cluster of two blocks) computes a tile of 256 weight rows with one instruction
// stream: block r of the pair brings rows 128 r .. of the weights and half of the tokens into
// its shared memory, and holds its rows' sums in its tensor memory.  So each operand byte is
// fetched once for a tile, and each SM's share is at most 32 KB for 512 clocks of products (a
// stage: 64 elements of the contracted axis).
//
//   kMmForward   out = x W^T: the rows are those of W, K-major.  With `gated` they are gate and
//                up rows of the same channels in turn, so that a thread finds the other product
//                of its channel in the neighbouring lane
//   kMmDx        dx = dout W: the rows are W's columns; the contracted axis is its rows
//
// A sum in tensor memory rounds towards zero with each product of 16 elements: 1e-7 of it a step
// for values of one sign, 5e-5 over 8192 elements (half a step of f16 is 4.9e-4).  Longer axes are
// summed in pieces of 8192, which the epilogue adds up, rounding to nearest; a piece is also what
// its bounded wait waits for.  8192 x 4096 x 16384, two pieces: 562 us, 560 without them.
//
// Where there are too few tiles for the SMs, two or four pairs share one: each takes a part of
// the contracted axis and sends its sums to the first pair's shared memory, which adds them in
// the pairs' order.
//
// 8192^3: 573 us, 1917 TFLOP/s, the tensor pipe busy in 97% of the clocks; 32 experts of 512
// rows x 2 x 2048 x 4096 with both products kept 345 us, 1590 TFLOP/s, of 300 rows 279 us, 1150:
// with fewer than 256 columns the weights' way from L2 is the bound.
//
// Warps: 0-7 epilogue (0-3 every other 32 tokens, 4-7 the others), 8 TMA, 9 MMA (of the
// pair's first block, for both; the copies of both count at its barrier).  Tensor memory: two
// sums of 256 columns.
#include "matmul.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace moedc {

constexpr int kMpThreads = 10 * kWarp;
constexpr int kMpTile = 256;                    // weight rows of the pair; tokens
constexpr int kMpHalf = kMpTile / 2;
constexpr int kMpElems = 64;                    // of the contracted axis in a stage
constexpr int kMpBytes = 128;
constexpr int kMpOperand = kMpHalf * kMpBytes;  // a block's share of one operand
constexpr int kMpStage = 2 * kMpOperand;
constexpr int kMpStages = 6;
constexpr int kMpPiece = 128;                   // stages of one sum
constexpr int kMpColumns = 512;

struct MpUnit {
    int e, r0, m, n0;
    int cols;           // of the product: m in 32s, as a pair's products go
};

__device__ __forceinline__ MpUnit mp_unit(const MmArgs& a, const int32_t* s_pre, const int32_t* s_beg, const int32_t* s_end,
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
    // an expert's chunks are equal ones: chunks - 1 of them are fewer rows than it has, as a
    // chunk is at most 256 and all of its rows more than chunks - 1 times that
    const int rows = s_end[lo] - s_beg[lo];
    const int size = ((rows - 1) / chunks + 32) / 32 * 32;
    MpUnit u;
    u.e = lo;
    u.n0 = t * (a.gated ? kMpHalf : kMpTile);
    u.r0 = s_beg[lo] + c * size;
    u.m = min(size, s_end[lo] - u.r0);
    u.cols = (u.m + 31) / 32 * 32;
    return u;
}

__device__ __forceinline__ uint16_t mp_round(float v, bool f16)
{
    return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ uint32_t mp_round2(float lo, float hi, bool f16)
{
    return (uint32_t)mp_round(lo, f16) | (uint32_t)mp_round(hi, f16) << 16;
}

// kPieces: the sums of a block's part have several pieces
template <int MODE, bool kPieces>
__global__ void __launch_bounds__(kMpThreads, 1)
matmul_pair_kernel(const __grid_constant__ MmArgs a, int parts, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ BoxMaps xmaps)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMpThreads / kWarp];
    __shared__ uint64_t full[kMpStages], empty[kMpStages], d_full[2], d_empty[2], done, never;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    // of the block in its pair; of the pair's first block, and the pair's part of a tile
    const int rank = cluster_rank() & 1, leader_rank = cluster_rank() & ~1, part = cluster_rank() / 2;
    const int first_unit = blockIdx.x / (2 * parts), unit_step = gridDim.x / (2 * parts);
    const int tile_n = a.gated ? kMpHalf : kMpTile;
    const int tiles = (a.N - 1) / tile_n + 1, ksteps = (a.K - 1) / kMpElems + 1;   // (sizes go up to INT_MAX)
    const int s_first = ksteps * part / parts, s_last = ksteps * (part + 1) / parts - 1;
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + kMpStages * kMpStage);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMpStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(d_full + b, 1);
            mbar_init(d_empty + b, 16);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        tc_alloc_pair(&s_tmem, kMpColumns);
        tc_fence_before();
    }
    pdl_enter();
    const bool over = mm_chunks<kMpThreads>(a, kMpTile, tiles, s_scan, s_pre, s_beg, s_end);
    cluster_sync();   // the other block's barriers stand
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // every warp of a cluster of several pairs comes by the three barriers of a tile, those that
    // have nothing to do between them as well
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
        const int half = warp >> 2, row = rank * kMpHalf + (warp & 3) * kWarp + lane, odd = lane & 1;
        const uint32_t d0 = tmem + ((uint32_t)((warp & 3) * kWarp) << 16);
        MvRing accs;
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MpUnit u = mp_unit(a, s_pre, s_beg, s_end, tiles, unit);
            if constexpr (kPieces) {
                // the pieces but the last one, then all of them to the last one's place
                float acc[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[i][j] = 0.0f;
                for (int s = s_first;; s += kMpPiece) {
                    mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                    tc_fence_after();
                    const uint32_t at = d0 + accs.slot * kMpTile + half * 32;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (half * 32 + i / 2 * 64 >= u.m) break;
                        float v[16];
                        tc_ld16(at + i / 2 * 64 + i % 2 * 16, v);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+f"(v[j]));
                            acc[i / 2][i % 2 * 16 + j] += v[j];
                        }
                    }
                    if (s + kMpPiece > s_last) break;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, leader_rank);
                    accs.next(2);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (half * 32 + i / 2 * 64 >= u.m) break;
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(acc[i / 2][i % 2 * 16 + j]);
                    tc_st16(d0 + accs.slot * kMpTile + half * 32 + i / 2 * 64 + i % 2 * 16, v);
                }
                tc_wait_st();
            } else {
                mbar_wait_warp(d_full + accs.slot, accs.phase, &s_abort);
                tc_fence_after();
            }
            const uint32_t d = d0 + accs.slot * kMpTile;
            // The thread's channel; neighbouring lanes trade a token for a token, so that each has
            // two channels of one (with `gated`: gate and up of one), the even lane of the first
            const int n = u.n0 + (a.gated ? row / 2 : row - odd);
            const bool in = n < a.N;
            uint16_t* o = static_cast<uint16_t*>(a.out) + (int64_t)u.r0 * a.N + n;
            uint16_t* keep = static_cast<uint16_t*>(a.extra);
            if (keep) keep += (int64_t)u.r0 * 2 * a.N + odd * a.N + n;
            // [part - 1][token / 4][row][token % 4] of the other pairs' sums
            float* sums = reinterpret_cast<float*>(smem) + (row & (kMpHalf - 1)) * 4;
            if (parts > 1) {
                cluster_sync();     // 1: no block's products read its stages any more
                if (part > 0) {
                    const uint32_t to = cluster_addr(sums + (part - 1) * u.cols * kMpHalf, rank);
                    for (int c = half * 32; c < u.m; c += 64) {
                        float v[32];
                        tc_ld32(d + c, v);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(v[j]));
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            if (c + j >= u.m) break;
                            st_cluster(to + (c + j) * (kMpHalf * 4), make_float2(v[j], v[j + 1]), make_float2(v[j + 2], v[j + 3]));
                        }
                    }
                }
                cluster_sync();     // 2: the sums are there
            }
            for (int c = half * 32; c < u.m && part == 0; c += 64) {
                float v[32];
                tc_ld32(d + c, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(v[j]));
                for (int p = 1; p < parts; ++p) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        if (c + j >= u.m) break;
                        const float4 s = *reinterpret_cast<const float4*>(sums + ((p - 1) * u.cols + c + j) * kMpHalf);
                        v[j] += s.x, v[j + 1] += s.y, v[j + 2] += s.z, v[j + 3] += s.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                    const int t = c + j + odd;
                    if (a.gated) {
                        const float g = odd ? got : v[j], up = odd ? v[j + 1] : got;
                        if (keep && in) {
                            if (c + j < u.m) keep[(int64_t)(c + j) * 2 * a.N] = mp_round(v[j], a.f16);
                            if (c + j + 1 < u.m) keep[(int64_t)(c + j + 1) * 2 * a.N] = mp_round(v[j + 1], a.f16);
                        }
                        if (t < u.m && in) o[(int64_t)t * a.N] = mp_round(mm_silu_mul(g, up), a.f16);
                    } else if (t < u.m && in) {
                        *reinterpret_cast<uint32_t*>(o + (int64_t)t * a.N) =
                            odd ? mp_round2(got, v[j + 1], a.f16) : mp_round2(v[j], got, a.f16);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (parts > 1) {
                // (the next tile's copies come to where these were)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                cluster_sync();     // 3: the sums have been read
            }
            if (lane == 0) mbar_arrive_pair(d_empty + accs.slot, leader_rank);
            accs.next(2);
        }
    } else if (warp == 8) {
        // ---- TMA: this block's weight rows, its half of the tokens
        // (one lane waits and issues: with the warp together 161 us against 150 for 8192 x 4096 x 4096)
        MvRing ring;
        int issued = 0;
        bool stop = !tc_elect();
        for (int unit = first_unit; unit < units; unit += unit_step) {
            const MpUnit u = mp_unit(a, s_pre, s_beg, s_end, tiles, unit);
            const int mine = u.cols / 2, r0 = u.r0 + rank * mine;
            const int box = (mine + 31) / 32;                             // in 32 rows
            const int bytes = 2 * (kMpOperand + box * 32 * kMpBytes);     // of both blocks
            for (int s = s_first; s <= s_last && !stop; ++s) {
                stop = !mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort);
                if (stop) break;
                uint8_t* w = smem + ring.slot * kMpStage;
                uint8_t* x = w + kMpOperand;
                const uint32_t at = cluster_addr(full + ring.slot, leader_rank);
                if (rank == 0) mbar_arrive_expect(full + ring.slot, bytes);
                if constexpr (MODE == kMmDx) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        tma_3d_pair(w + h * (kMpOperand / 2), &wmap, u.n0 + rank * kMpHalf + h * 64, s * kMpElems, u.e, at);
                } else if (a.gated) {
                    // [E][N][gate or up][K]
                    tma_4d_pair(w, &wmap, s * kMpElems, 0, u.n0 + rank * (kMpHalf / 2), u.e, at);
                } else {
                    tma_4d_pair(w, &wmap, s * kMpElems, 0, u.n0 + rank * kMpHalf, u.e, at);
                }
                // rows past the chunk's are of no account
                tma_2d_pair(x, xmaps.by + (box - 1), s * kMpElems, r0, at);
                ring.next(kMpStages);
                ++issued;
            }
            tile_done();
        }
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - kMpStages); n < issued && rank == 0; ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % kMpStages, (n / kMpStages) & 1, &alone)) s_abort = 1;
        }
        __syncwarp();
        // the last product's arrival at the second block; the wait begins behind the block's last
        // copy, as its bound is one of a step and not of the call
        if (rank == 1) {
            volatile int alone = 0;
            if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        }
        // a second block that gave up sees no barrier of its copies: they have a millisecond
        if (s_abort)
            for (const unsigned long long t0 = globaltimer(); globaltimer() - t0 < 1000000ull;) {}
        __syncwarp();
    } else {
        // ---- MMA, for both blocks: one elected lane issues; the warp stays together
        if (rank == 0) {
            const bool leader = tc_elect();
            MvRing ring, accs;
            int k = 0;
            const uint32_t type = (a.f16 ? 0u : (1u << 7) | (1u << 10)) | (MODE == kMmDx ? 1u << 15 : 0u);
            for (int unit = first_unit; unit < units; unit += unit_step) {
                const MpUnit u = mp_unit(a, s_pre, s_beg, s_end, tiles, unit);
                const uint32_t idesc = (1u << 4) | type | ((uint32_t)(u.cols / 8) << 17) | ((uint32_t)(kMpTile / 16) << 24);
                for (int s = s_first; s <= s_last; ++s) {
                    const bool first = kPieces ? (s - s_first) % kMpPiece == 0 : s == s_first;
                    const bool last = s == s_last || (kPieces && (s - s_first) % kMpPiece == kMpPiece - 1);
                    if (first && k++ >= 2) mbar_wait_warp(d_empty + accs.slot, accs.phase ^ 1, &s_abort);
                    mbar_wait_warp(full + ring.slot, ring.phase, &s_abort);
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + ring.slot * kMpStage);
                    const uint64_t w = MODE == kMmDx ? tc_smem_desc_mn(st, kMpOperand / 2) : tc_smem_desc(st);
                    const uint64_t x = tc_smem_desc(st + kMpOperand);
                    if (leader) {
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            // a descriptor counts in 16 bytes: 32 of a row, or 16 rows of 128
                            tc_mma_pair(tmem + accs.slot * kMpTile, w + p * (MODE == kMmDx ? 128 : 2), x + p * 2, idesc, p != 0 || !first);
                        tc_commit_pair(empty + ring.slot, leader_rank);
                        if (last) tc_commit_pair(d_full + accs.slot, leader_rank);
                    }
                    __syncwarp();
                    if (last) accs.next(2);
                    ring.next(kMpStages);
                }
                tile_done();
            }
            // tensor memory is given back only when the last product is through
            if (leader) tc_commit_pair(&done, leader_rank);
            __syncwarp();
            volatile int alone = 0;
            if (!mbar_wait(&done, 0, &alone)) s_abort = 1;
        } else {
            for (int unit = first_unit; unit < units; unit += unit_step) tile_done();
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (warp == 9) tc_free_pair(tmem, kMpColumns);
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {

bool map_rows16(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t ld, int box_rows)
{
    const cuuint64_t size[2] = {(cuuint64_t)width, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_128B, base, 2, size, stride, box);
}

namespace {

// most tiles that are split into as many parts
#ifndef MOEDC_PAIR_PARTS_4
#define MOEDC_PAIR_PARTS_4 14
#define MOEDC_PAIR_PARTS_2 36
#endif

// x: the rows
template <int MODE>
int launch_mm_pair(const moedc::MmArgs& a, const CUtensorMap& w, const void* x, int64_t ldx, cudaStream_t stream)
{
    moedc::BoxMaps rows{};
    // a block's half of a chunk, in 32s
    for (int i = 0; i < 4 && (i == 0 || a.rows > 64 * i); ++i)
        if (!map_rows16(rows.by + i, x, a.K, a.rows, ldx, 32 * (i + 1))) return MOEDC_ERR_CUDA;
    constexpr size_t kFixed = moedc::kMpStages * moedc::kMpStage;
    const int tile = a.gated ? moedc::kMpHalf : moedc::kMpTile;
    const int64_t units = ((int64_t)a.rows / moedc::kMpTile + (a.E < a.rows ? a.E : a.rows)) * ((a.N + (int64_t)tile - 1) / tile);
    const int pairs = sm_count() / 2;
    // parts of the contracted axis, as in matmul_stream.cu: clusters of four or eight blocks.  One
    // token x 4096 channels: 14 tiles 21.4 us in one part, 16.1 in two, 12.7 in four; 36 tiles 22.0
    // and 18.3; 512 channels 9.5 and 10.6.
    const int64_t most = a.rows < moedc::kMpTile ? a.rows : moedc::kMpTile;
    const int64_t sums = (most + 31) / 32 * 32 * moedc::kMpHalf * sizeof(float);
    const int ksteps = (a.K - 1) / moedc::kMpElems + 1;
    auto fits = [&](int p, int64_t tiles) { return units <= tiles && ksteps >= 16 * p && (p - 1) * sums <= (int64_t)kFixed; };
    const int parts = fits(4, MOEDC_PAIR_PARTS_4) ? 4 : fits(2, MOEDC_PAIR_PARTS_2) ? 2 : 1;
    // the longest part (of parts that differ by a stage)
    const bool pieces = (ksteps + parts - 1) / parts > moedc::kMpPiece;
    auto* k = pieces ? moedc::matmul_pair_kernel<MODE, true> : moedc::matmul_pair_kernel<MODE, false>;
    static PerDevice raised[2];
    if (!raise_smem_limit(raised[pieces], (const void*)k, (int)kFixed + (3 * MOEDC_MAX_E + 1) * 4)) return MOEDC_ERR_CUDA;
    clear_stale_error();
    launch_cluster(k, 2 * parts, 2 * parts * (int)(units < pairs ? units : pairs), moedc::kMpThreads,
                   kFixed + (3 * (size_t)a.E + 1) * sizeof(int32_t), stream, a, parts, w, rows);
    return launch_status();
}

}  // namespace

int launch_mm_forward(const moedc::MmArgs& a, const void* x, int64_t ldx, const void* w, cudaStream_t stream)
{
    CUtensorMap map;
    const cuuint64_t K = a.K, N = a.N, parts = a.gated ? 2 : 1;
    const cuuint64_t size[4] = {K, parts, N, (cuuint64_t)a.E}, stride[3] = {2 * K * N, 2 * K, 2 * K * N * parts};
    const cuuint32_t box[4] = {64, (cuuint32_t)parts, (cuuint32_t)(moedc::kMpHalf / parts), 1};
    if (!tensor_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_128B, w, 4, size, stride, box)) return MOEDC_ERR_CUDA;
    return launch_mm_pair<moedc::kMmForward>(a, map, x, ldx, stream);
}

int launch_mm_dx(const moedc::MmArgs& a, const void* dout, int64_t ldd, const void* w, cudaStream_t stream)
{
    CUtensorMap map;
    const cuuint64_t size[3] = {(cuuint64_t)a.N, (cuuint64_t)a.K, (cuuint64_t)a.E};
    const cuuint64_t stride[2] = {2 * (cuuint64_t)a.N, 2 * (cuuint64_t)a.N * a.K};
    const cuuint32_t box[3] = {64, 64, 1};
    if (!tensor_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_128B, w, 3, size, stride, box)) return MOEDC_ERR_CUDA;
    return launch_mm_pair<moedc::kMmDx>(a, map, dout, ldd, stream);
}

}  // namespace moedc_host
