// Products of packed expert rows with 4-bit weights and group scales:
//   out[r][n] = sum_k x[r'][k] (q[e][n][k] - z[e][n][k/g]) s[e][n][k/g]
// for the expert e whose rows hold r.
//
// A decode step gives each expert a handful of rows, so the stream of weights
// from HBM bounds it (half a byte per weight, each read once), and what the
// SMs do per weight has to fit under that stream: 46 weights per SM and clock.
//
// Work is cut into units of (expert, tile of output channels, chunk of rows).
// One persistent block per SM takes units in turn.  Its 16 consumer warps own
// 16 weight rows each and, when there are few tiles, one of `wk` interleaved
// parts of K (the parts are added in shared memory at the unit's end).  One
// more warp fills a ring of stages by TMA that runs on across units, so the
// stream never drains between them.  x is prepared once per call by a kernel of
// its own (records of 256 channels in the order the products read them): doing
// that in the ring, for every block again, took as long as the stream.
//
// The products run on the tensor cores with the weights as the 16-row operand
// and eight rows of x as the other, both in f16 with binary32 sums.  The ALU,
// which masks and shifts, issues every other clock and is the pipe that fills
// first, so a weight costs it one mask and a quarter of a shift:
// a nibble in the low bits of an f16 is the subnormal q * 2^-24 (one nibble
// higher q * 2^-20, with x scaled by 2^-4 to match), exact as it stands, and the
// zero point a subtraction of two such numbers, exact as well.  (Taken out of the
// group's sum instead, sum q x - z sum x, it would cost less, 104 against 111 us and
// 502 against 528 in the shapes below, but a large value of x whose weight is at the
// zero point would then cancel in binary32 and take the small ones' bits along.)
// x is brought into f16 per row and stage by a power of two that puts its largest
// value into [2^14, 2^15), the high nibbles' channels by another 2^-4: bf16 stays exact
// down to 2^-27 of that value, f16, which has three bits more, to 2^-24, and what lies
// below is off by at most 2^-35 of it.  The group's sum is then scaled in binary32, so
// neither weights nor scales are ever rounded.  An infinity or a NaN stays one in f16.
//
// 16 tokens, top 8 of 128 experts, 2 x 1024 x 6144 with SwiGLU, groups of 128: 111
// us (535 MB, 4.8 TB/s); 128 tokens, top 8 of 288 experts, 2048 x 7168, groups of 64:
// with zero points 528 us (2255 MB, 4.3 TB/s).  The stream alone would take 93 and 335
// us: unpacking and the latencies of shared memory and of the matrix instructions bound
// it.
//
// For few rows tcgen05 is the slower form: a product with 16 columns of x takes it
// 120 clocks for 16 channels of 128 weight rows, and every stage four hand-overs (16
// tokens 241 us, 128 tokens 930 us in the shapes below); where experts have many rows
// it is taken (matvec_int4_tc.cu).
#include <climits>
#include <cmath>

#include "matvec_int4_ring.cuh"

namespace moedc {

constexpr int kMvConsumers = 16;                       // warps
constexpr int kMvThreads = (kMvConsumers + 1) * kWarp;
constexpr int kMvRows = kMvConsumers * 16;             // weight rows x parts of K in a stage
constexpr int kMvW = kMvRows * kMvChunk / 2;           // a stage's weights
constexpr int kMvTokens = 32;                          // rows of x x parts of K, at most
constexpr int kMvMaxStages = 6;
constexpr int kMvRed = kMvConsumers * 8 * kWarp * (int)sizeof(float);
// ---------------------------------------------------------- tensor products

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// plain loads, so that the compiler may order them between the waits as it likes
template <typename V> __device__ __forceinline__ V lds(const uint8_t* at) { return *reinterpret_cast<const V*>(at); }

// One stage of one warp: its 16 weight rows x 256 channels with 8 NT rows of x.
//   w    place of row g at word t (128 bytes a row, 16-byte pieces permuted by the
//        row's low three bits); the warp's other eight rows lie kMvW / 2 further
//   x    place of row g's record at its words t
//   c    place of the factor of x row 2t
template <int GROUP, int NT, bool FULL, typename S>
__device__ __forceinline__ void mv_stage(const uint8_t* st, uint32_t w, uint32_t x, uint32_t c,
                                         const MvScales<GROUP, S, 2>& sz, int steps, float (&acc)[NT][4])
{
    constexpr int kPer = GROUP / 32;       // 32-channel steps of a group
    constexpr int kGroups = kMvChunk / GROUP;
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float sum[NT][4];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
        if (!FULL && q * kPer >= steps) break;
        float tmp[NT][4];
        const uint32_t za = sz.zero_f16(0, q), zb = sz.zero_f16(1, q);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int k = q * kPer + p;
            const uint32_t at = w ^ (k << 4);
            const uint32_t a = lds<uint32_t>(st + at), b = lds<uint32_t>(st + at + kMvW / 2);
            constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
            uint32_t m[8] = {a & lo, b & lo, a & hi, b & hi, (a >> 8) & lo, (b >> 8) & lo, (a >> 8) & hi, (b >> 8) & hi};
            // exact: subnormals of one exponent
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = sub_f16x2(m[j], (j % 2 ? zb : za) << (j & 2 ? 4 : 0));
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 r = lds<uint4>(st + x + k * 64 + i * 8 * kMvRecord);
                if (p == 0) mma_f16(tmp[i], m[0], m[1], m[2], m[3], r.x, r.y, none);
                else mma_f16(tmp[i], m[0], m[1], m[2], m[3], r.x, r.y, tmp[i]);
                mma_f16(tmp[i], m[4], m[5], m[6], m[7], r.z, r.w, tmp[i]);
            }
        }
        const float s0 = sz.scale(0, q), s1 = sz.scale(1, q);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const float (&d)[4] = tmp[i];
            sum[i][0] = q ? fmaf(s0, d[0], sum[i][0]) : s0 * d[0];
            sum[i][1] = q ? fmaf(s0, d[1], sum[i][1]) : s0 * d[1];
            sum[i][2] = q ? fmaf(s1, d[2], sum[i][2]) : s1 * d[2];
            sum[i][3] = q ? fmaf(s1, d[3], sum[i][3]) : s1 * d[3];
        }
    }
    // the stage's factor of x, and the rest of the weights' 2^24
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const float fu = lds<float>(st + c + i * 8 * kMvRecord);
        const float fv = lds<float>(st + c + i * 8 * kMvRecord + kMvRecord);
        acc[i][0] = fmaf(fu, 4096.0f * sum[i][0], acc[i][0]);
        acc[i][1] = fmaf(fv, 4096.0f * sum[i][1], acc[i][1]);
        acc[i][2] = fmaf(fu, 4096.0f * sum[i][2], acc[i][2]);
        acc[i][3] = fmaf(fv, 4096.0f * sum[i][3], acc[i][3]);
    }
}

// The unit's end: the parts of K added, the epilogue, the outputs.
template <int NT>
__device__ __forceinline__ void mv_store(const MatvecArgs& a, const MvUnit& u, float* s_red,
                                         float (&acc)[NT][4], uint16_t* __restrict__ out)
{
    const int lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x / kWarp;
    const int wk = 1 << a.lk, part = warp & (wk - 1), tile = warp >> a.lk;
    if (wk > 1) {
        // consumers only: the first barrier ends the reads of the unit before
        asm volatile("bar.sync 1, %0;" ::"n"(kMvConsumers * kWarp) : "memory");
        if (part != 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s_red[(warp * NT * 4 + i * 4 + j) * kWarp + lane] = acc[i][j];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kMvConsumers * kWarp) : "memory");
        if (part != 0) return;
        for (int p = 1; p < wk; ++p)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += s_red[((warp + p) * NT * 4 + i * 4 + j) * kWarp + lane];
    }
    const int n = u.n0 + tile * 8 + g, n2 = n + (kMvRows >> a.lk) / 2;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = i * 8 + t * 2 + c;
            if (r >= u.m) continue;
            uint16_t* o = out + (int64_t)(u.r0 + r) * a.N;
            if (a.swiglu) {
                const float v = acc[i][c];
                if (n < a.N) store16(o + n, v / (1.0f + expf(-v)) * acc[i][2 + c], a.f16);
            } else {
                if (n < a.N) store16(o + n, acc[i][c], a.f16);
                if (n2 < a.N) store16(o + n2, acc[i][2 + c], a.f16);
            }
        }
}

// Records of x, by row of x (then one of zeros) or by packed row, a warp each: eight
// channels a lane, brought into f16 range and stored in the order of the weights'
// registers, channels (0,4), (1,5) 2^-4, (2,6), (3,7) 2^-4.
template <typename T>
__global__ void __launch_bounds__(256)
matvec_x_kernel(const __grid_constant__ MatvecArgs a, bool packed, uint8_t* __restrict__ records)
{
    pdl_enter();
    const int lane = threadIdx.x % kWarp;
    const int chunks = (a.Kd + kMvChunk - 1) / kMvChunk;
    const int64_t n = (packed ? (int64_t)a.rows : (int64_t)a.x_rows + 1) * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / kWarp; i < n; i += (int64_t)gridDim.x * 8) {
        int64_t r = i / chunks;
        const int k = (int)(i - r * chunks) * kMvChunk + lane * 8;
        bool bad = false;   // told by the kernel that knows which rows count
        if (packed) r = x_row(a, (int)r, bad);
        Pack<T, 8> h;
        float f[8] = {};
        if (r < a.x_rows && k < a.Kd) {
            h = *reinterpret_cast<const Pack<T, 8>*>(static_cast<const T*>(a.x) + r * a.ldx + k);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = to_f32(h.v[j]);
        }
        unsigned top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        // scale = 2^sc: the record's largest exponent goes to 14
        const int sc = min(127, 141 - (int)(__reduce_max_sync(0xffffffffu, top) >> 23));
        const float scale = __uint_as_float((unsigned)(sc + 127) << 23);
        Pack<__half2, 4> o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __half2 b = __floats2half2_rn(f[j] * scale, f[j + 4] * scale);
            if (j & 1) b = __hmul2(b, __float2half2_rn(0.0625f));   // the odd nibble
            o.v[j] = b;
        }
        uint8_t* to = records + i * kMvRecord;
        reinterpret_cast<Pack<__half2, 4>*>(to)[lane] = o;
        if (lane == 0) *reinterpret_cast<float*>(to + kMvFactor) = __uint_as_float((unsigned)(139 - sc) << 23);
    }
}

// What a consumer warp carries through its units.
struct MvWarp {
    uint32_t ow, ox, oc;           // offsets in a stage: weights, x, factors of x
    int part, row, half;
    bool whole;                    // a row's groups of a stage are one aligned load
};

// Where the scales of the warp's two rows of a unit begin; rows past the last read the
// last one's, and nothing uses them.
template <int GROUP, typename S>
__device__ __forceinline__ void mv_rows(const MatvecArgs& a, const MvWarp& w, const MvUnit& u, int groups,
                                        typename MvScales<GROUP, S, 2>::Rows& rows)
{
    const int n0 = min(u.n0 + w.row, a.N - 1);
    const int n1 = a.swiglu ? n0 + a.N : min(u.n0 + w.half + w.row, a.N - 1);
    const int64_t first = (int64_t)u.e * (a.swiglu ? 2 * a.N : a.N);
    rows.s[0] = static_cast<const S*>(a.scales) + (first + n0) * groups;
    rows.s[1] = static_cast<const S*>(a.scales) + (first + n1) * groups;
    rows.z[0] = a.zeros + (first + n0) * groups;
    rows.z[1] = a.zeros + (first + n1) * groups;
}

// All stages of one unit with 8 NT rows of x.  `now` holds the first stage's
// scales and is left with those of the next unit's (`un`, when there is one).
template <int GROUP, int NT, typename S>
__device__ __forceinline__ void mv_consume(const MatvecArgs& a, const MvWarp& w, const uint8_t* smem, MvRing& ring, uint64_t* full,
                                           uint64_t* empty, volatile int* abort, int ksteps, int groups,
                                           bool more, const MvUnit& un, MvScales<GROUP, S, 2>& now,
                                           typename MvScales<GROUP, S, 2>::Rows& rows, float (&acc)[NT][4])
{
    constexpr int kGroups = kMvChunk / GROUP;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const bool zeros = a.zeros != nullptr;
    const int last = w.whole ? groups - kGroups : groups - 1;    // the last group to begin a load at
    int left = a.Kd - w.part * kMvChunk, q = w.part * kGroups;
    for (int s = ksteps; s > 0; --s, left -= kMvChunk << a.lk) {
        MvScales<GROUP, S, 2> next = now;
        q = min(q + (kGroups << a.lk), last);
        if (s == 1) {
            q = min(w.part * kGroups, last);
            if (more) mv_rows<GROUP, S>(a, w, un, groups, rows);
        }
        next.load(rows, q, groups - q, w.whole, zeros);
        mbar_wait(full + ring.slot, ring.phase, abort);
        __syncwarp();   // the products want the warp's lanes together, a wait may part them
        const uint8_t* st = smem + ring.slot * a.stage_bytes;
        // a part without channels left in the last stage has no records of x there either
        if (left >= kMvChunk) mv_stage<GROUP, NT, true>(st, w.ow, w.ox, w.oc, now, 8, acc);
        else if (left > 0) mv_stage<GROUP, NT, false>(st, w.ow, w.ox, w.oc, now, left / 32, acc);
        __syncwarp();
        if (threadIdx.x % kWarp == 0) mbar_arrive(empty + ring.slot);
        ring.next(a.stages);
        now = next;
    }
}

// NTMAX: eights of rows in a unit, at most
template <int GROUP, typename S, int NTMAX>
__global__ void __launch_bounds__(kMvThreads, 1)
matvec_int4_kernel(const __grid_constant__ MatvecArgs a, const __grid_constant__ CUtensorMap wmap,
                   uint16_t* __restrict__ out)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[kMvThreads / kWarp];
    __shared__ uint64_t full[kMvMaxStages], empty[kMvMaxStages], never;
    __shared__ volatile int s_abort;
    constexpr int kGroups = kMvChunk / GROUP;      // of a row in a stage

    const int lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x / kWarp;
    const int wk = 1 << a.lk, part = warp & (wk - 1), tile = warp >> a.lk;
    const int half = (kMvRows >> a.lk) / 2;                // weight rows of half a tile
    const int tile_n = a.swiglu ? half : 2 * half;
    const int tiles = (a.N + tile_n - 1) / tile_n;
    const int groups = a.Kd / GROUP;
    const int wrows = a.swiglu ? 2 * a.N : a.N;
    const int ksteps = (a.Kd + (kMvChunk << a.lk) - 1) / (kMvChunk << a.lk);
    // a stage: weights [half of the tile][part][row][128 bytes] (with SwiGLU the halves
    // are gate and up rows), x [part][row] as records
    float* s_red = reinterpret_cast<float*>(smem + a.stages * a.stage_bytes);
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + a.stages * a.stage_bytes + kMvRed);
    int32_t *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kMvConsumers);
        }
        mbar_init(&never, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_enter();

    const bool over = mv_chunks<kMvThreads>(a, tiles, s_scan, s_pre, s_beg, s_end);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);

    MvRing ring;
    if (warp < kMvConsumers) {
        if (a.wait_extra) mbar_wait(&never, 0, &s_abort);
        MvWarp w;
        w.part = part;
        w.row = tile * 8 + g;                              // in each half of the tile
        w.half = half;
        w.ow = part * half * 128 + w.row * 128 + (g << 4) + t * 4;
        w.ox = kMvW + (part * a.chunk_rows + g) * kMvRecord + t * 16;
        w.oc = kMvW + (part * a.chunk_rows + 2 * t) * kMvRecord + kMvFactor;
        w.whole = MvScales<GROUP, S, 2>::aligned_groups(a, groups);
        int unit = blockIdx.x;
        if (unit < units) {
            MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            MvScales<GROUP, S, 2> now;
            typename MvScales<GROUP, S, 2>::Rows rows;
            now.clear();
            mv_rows<GROUP, S>(a, w, u, groups, rows);
            const int q0 = min(part * kGroups, w.whole ? groups - kGroups : groups - 1);
            now.load(rows, q0, groups - q0, w.whole, a.zeros != nullptr);
            while (unit < units) {
                unit += gridDim.x;
                const bool more = unit < units;
                MvUnit un = u;
                if (more) un = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
                if (NTMAX == 1 || u.m <= 8) {
                    float acc[1][4];
                    mv_consume<GROUP, 1, S>(a, w, smem, ring, full, empty, &s_abort, ksteps, groups, more, un, now, rows, acc);
                    mv_store<1>(a, u, s_red, acc, out);
                } else if (NTMAX == 2 || u.m <= 16) {
                    float acc[2][4];
                    mv_consume<GROUP, 2, S>(a, w, smem, ring, full, empty, &s_abort, ksteps, groups, more, un, now, rows, acc);
                    mv_store<2>(a, u, s_red, acc, out);
                } else if constexpr (NTMAX == 4) {
                    float acc[4][4];
                    mv_consume<GROUP, 4, S>(a, w, smem, ring, full, empty, &s_abort, ksteps, groups, more, un, now, rows, acc);
                    mv_store<4>(a, u, s_red, acc, out);
                }
                u = un;
            }
        }
    } else {
        // the producer warp: two TMA boxes of weights per part, one for each half of the
        // tile's rows, and a bulk copy for each record of x, by lane
        int issued = 0;
        bool bad = false;
        const int chunks = (a.Kd + kMvChunk - 1) / kMvChunk;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            // one answer for the warp: a consumer may set the flag while its lanes are apart, and
            // the votes below want all of them
            if (__any_sync(0xffffffffu, s_abort != 0)) break;
            const MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
            const int wrow = u.e * wrows + u.n0;
            const int r = lane >> a.lk, p = lane & (wk - 1);       // this lane's record
            const bool mine = r < u.m;
            const uint8_t* xr = mine ? a.records + (int64_t)x_row(a, u.r0 + r, bad) * chunks * kMvRecord : nullptr;
            for (int s = 0; s < ksteps; ++s) {
                const bool go = mbar_wait(empty + ring.slot, ring.phase ^ 1, &s_abort);
                if (!__all_sync(0xffffffffu, go)) break;
                uint8_t* st = smem + ring.slot * a.stage_bytes;
                const uint32_t bar = smem_u32(full + ring.slot);
                const int c0 = s << a.lk;
                const int live = min(wk, chunks - c0);             // parts that have channels left
                if (lane == 0) mbar_arrive_expect(full + ring.slot, live * (2 * half * 128 + u.m * kMvRecord));
                __syncwarp();
                if (lane < 2 * live)
                    asm volatile(
                        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                        "[%0], [%1, {%2, %3}], [%4];" ::"r"(
                            smem_u32(st + (lane & 1) * (kMvW / 2) + (lane >> 1) * half * 128)), "l"(&wmap),
                        "r"((c0 + (lane >> 1)) * (kMvChunk / 2)),
                        "r"(wrow + (lane & 1) * (a.swiglu ? a.N : half)), "r"(bar) : "memory");
                if (mine && p < live)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            smem_u32(st + kMvW + (p * a.chunk_rows + r) * kMvRecord)),
                        "l"(xr + (int64_t)(c0 + p) * kMvRecord), "n"(kMvRecord), "r"(bar) : "memory");
                ring.next(a.stages);
                ++issued;
            }
        }
        // no copy may land after the block has gone, whatever else gave up
        for (int n = max(0, issued - a.stages); n < issued; ++n) {
            volatile int alone = 0;
            if (!mbar_wait(full + n % a.stages, (n / a.stages) & 1, &alone)) s_abort = 1;
        }
        if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_abort) raise_status(a.status, MOEDC_ERR_TIMEOUT);
}

}  // namespace moedc

namespace moedc_host {

namespace {

bool tensor_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int dims,
                const cuuint64_t* size, const cuuint64_t* stride, const cuuint32_t* box)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess || found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!encode) return false;
    const cuuint32_t elem[3] = {1, 1, 1};
    return encode(map, type, dims, const_cast<void*>(base), size, stride, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool matvec_weight_map(CUtensorMap* map, const void* wq, int Kd, int64_t rows, int box_rows)
{
    const cuuint64_t size[2] = {(cuuint64_t)Kd / 2, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)Kd / 2};
    const cuuint32_t box[2] = {moedc::kMvChunk / 2, (cuuint32_t)box_rows};
    return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, wq, 2, size, stride, box);
}

bool matvec_x_maps(CUtensorMap* channels, CUtensorMap* factors, const uint8_t* records, int chunks, int rows, int box_rows)
{
    const cuuint64_t size[3] = {moedc::kMvRecord / 2, (cuuint64_t)chunks, (cuuint64_t)rows};
    const cuuint64_t stride[2] = {moedc::kMvRecord, (cuuint64_t)moedc::kMvRecord * chunks};
    const cuuint32_t many[3] = {64, 1, (cuuint32_t)box_rows}, one[3] = {8, 1, (cuuint32_t)box_rows};
    return tensor_map(channels, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_128B, records, 3, size, stride, many) &&
           tensor_map(factors, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_NONE, records, 3, size, stride, one);
}

namespace {

// Parts of K and rows of a unit: the pair with the least of
//   rounds of units * (stages of a unit * cost of a stage + cost of a unit)
// where the costs are the fit of a sweep over every pair at four shapes, and name the
// fastest pair of each or one within 4% of it (16 tokens 2 x 1024 x 6144 with SwiGLU
// 118 / 116 / 132 us at 1 / 2 / 4 parts and 8 rows; 128 tokens 2048 x 7168 with zero
// points 554 / 518 / 619 us; 255 tokens 2050 x 2048 at 1 part 99 / 81 / 84 us with 8 /
// 16 / 32 rows, at 4 parts 146 us; one token 14336 x 7168 34 / 22 / 23 us).  A stage
// takes longer with more rows; one part with zero points holds more lines of scales open
// than L1 keeps.  How many experts have rows, and how many each, is the guess of a
// uniform choice.
void mv_shape(moedc::MatvecArgs& a, int blocks)
{
    const double active = a.E * (1.0 - exp(-(double)a.rows / a.E));
    const double per = a.rows / active;
    double best = 0.0;
    for (int lk = 0; lk <= 2; ++lk)
        for (int chunk = 8; chunk <= moedc::kMvTokens >> lk; chunk *= 2) {
            const int tile_n = (moedc::kMvRows >> lk) / (a.swiglu ? 2 : 1);
            const double tiles = (a.N + tile_n - 1) / tile_n;
            const double chunks = per / chunk > 0.5 ? per / chunk + 0.5 : 1.0;
            const double rounds = ceil(active * tiles * chunks / blocks);
            const double stages = (a.Kd + (moedc::kMvChunk << lk) - 1) / (moedc::kMvChunk << lk);
            double stage = chunk == 8 || per <= 8 ? 44.0 : chunk == 16 || per <= 16 ? 56.0 : 80.0;
            if (lk == 0 && a.zeros) stage *= 1.25;
            const double cost = rounds * (stages * stage + 90.0);
            if (best == 0.0 || cost < best) {
                best = cost;
                a.lk = lk;
                a.chunk_rows = chunk;
            }
        }
}

template <int GROUP, typename S, int NTMAX>
int launch_matvec(moedc::MatvecArgs a, void* out, cudaStream_t stream)
{
    auto* k = moedc::matvec_int4_kernel<GROUP, S, NTMAX>;
    static PerDevice raised;
    if (!raise_smem_limit(raised, (const void*)k, kMvSmem - 1024)) return MOEDC_ERR_CUDA;
    const int blocks = sm_count();
    a.stage_bytes = (moedc::kMvW + (a.chunk_rows << a.lk) * moedc::kMvRecord + 1023) / 1024 * 1024;
    const size_t fixed = moedc::kMvRed + (3 * (size_t)a.E + 1) * sizeof(int32_t);
    a.stages = (int)((kMvSmem - 1024 - fixed) / a.stage_bytes);
    if (a.stages > moedc::kMvMaxStages) a.stages = moedc::kMvMaxStages;
    const size_t smem = (size_t)a.stages * a.stage_bytes + fixed;

    const int part_rows = moedc::kMvRows >> a.lk;
    CUtensorMap map;
    if (!matvec_weight_map(&map, a.wq, a.Kd, (int64_t)a.E * (a.swiglu ? 2 : 1) * a.N, part_rows / 2))
        return MOEDC_ERR_CUDA;

    const int tile_n = part_rows / (a.swiglu ? 2 : 1);
    const int64_t most = ((int64_t)a.rows / a.chunk_rows + (a.E < a.rows ? a.E : a.rows)) *
                         ((a.N + tile_n - 1) / tile_n);
    clear_stale_error();
    launch(k, (int)(most < blocks ? most : blocks), moedc::kMvThreads, smem, stream, a, map,
           static_cast<uint16_t*>(out));
    return launch_status();
}

template <int GROUP, typename S>
int launch_matvec_rows(const moedc::MatvecArgs& a, void* out, cudaStream_t stream)
{
    return a.chunk_rows == 8    ? launch_matvec<GROUP, S, 1>(a, out, stream)
           : a.chunk_rows == 16 ? launch_matvec<GROUP, S, 2>(a, out, stream)
                                : launch_matvec<GROUP, S, 4>(a, out, stream);
}

template <typename S>
int launch_matvec_group(const moedc::MatvecArgs& a, int group, void* out, cudaStream_t stream)
{
    return group == 32   ? launch_matvec_rows<32, S>(a, out, stream)
           : group == 64 ? launch_matvec_rows<64, S>(a, out, stream)
                         : launch_matvec_rows<128, S>(a, out, stream);
}

template <typename T>
int launch_matvec_x(const moedc::MatvecArgs& a, bool packed, uint8_t* records, cudaStream_t stream)
{
    const int64_t n = (packed ? (int64_t)a.rows : (int64_t)a.x_rows + 1) * ((a.Kd + moedc::kMvChunk - 1) / moedc::kMvChunk);
    const int64_t want = (n + 7) / 8, most = 8 * (int64_t)sm_count();
    clear_stale_error();
    launch(moedc::matvec_x_kernel<T>, (int)(want < most ? want : most), 256, 0, stream, a, packed, records);
    return launch_status();
}

}  // namespace
}  // namespace moedc_host

extern "C" size_t moedc_matvec_int4_workspace_bytes(int x_rows, int Kd, int E, int N, int flags, int rows)
{
    if (x_rows < 0 || Kd < 1 || E < 1 || N < 1 || rows < 1 || (flags & ~MOEDC_SWIGLU) != 0) return 0;
    if (moedc_host::matvec_small_takes(Kd, E, N, flags != 0, rows)) return 0;
    // by row of x or, where experts have many rows, by packed row
    size_t records = (size_t)x_rows + 1;
    if (moedc_host::matvec_tc_takes(E, rows, 128) && (size_t)rows > records) records = (size_t)rows;
    return records * ((Kd + (size_t)moedc::kMvChunk - 1) / moedc::kMvChunk) * moedc::kMvRecord;
}

extern "C" int moedc_matvec_int4(const void* x, int64_t ldx, int dtype, int x_rows, int Kd,
                                 const void* wq, const void* scales, int scale_dtype,
                                 const uint8_t* zeros, int group, int E, int N, int flags,
                                 const int32_t* offsets, const int32_t* counts,
                                 const int32_t* src, int top_k, int rows, void* out,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 cudaStream_t stream)
{
    using namespace moedc_host;
    if ((dtype != MOEDC_BF16 && dtype != MOEDC_F16) || !lm_dtype_ok(scale_dtype)) return MOEDC_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return MOEDC_ERR_ARG;
    if (Kd < group || Kd % group != 0 || E < 1 || E > MOEDC_MAX_E || N < 1 || x_rows < 0 ||
        x_rows == INT32_MAX || rows < 0 || (flags & ~MOEDC_SWIGLU) != 0)
        return MOEDC_ERR_ARG;
    if ((offsets == nullptr) != (counts == nullptr) || (!offsets && E != 1)) return MOEDC_ERR_ARG;
    if (src && top_k < 1) return MOEDC_ERR_ARG;
    if (!wq || !scales || !dev_status || ldx < Kd || ldx % 8 != 0) return MOEDC_ERR_ARG;
    if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(scales, lm_dtype_size(scale_dtype)) ||
        !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(src, 4) || !aligned(out, 2) ||
        !aligned(dev_status, 4))
        return MOEDC_ERR_ARG;
    // weight rows and units (expert, tile, chunk of at least 8 rows) are counted in 32 bits
    if ((int64_t)E * N * (flags ? 2 : 1) > INT32_MAX - moedc::kMvRows ||
        ((int64_t)rows / 8 + E) * ((int64_t)N / 32 + 1) > INT32_MAX)
        return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!out || (x_rows > 0 && !x)) return MOEDC_ERR_ARG;   // an empty x has no address
    const bool small = matvec_small_takes(Kd, E, N, flags != 0, rows);
    if (!small && (!workspace || !aligned(workspace, 16) ||
                   workspace_bytes < moedc_matvec_int4_workspace_bytes(x_rows, Kd, E, N, flags, rows)))
        return MOEDC_ERR_ARG;
    moedc::MatvecArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.wq = static_cast<const uint8_t*>(wq);
    a.scale_dtype = scale_dtype;
    a.x_rows = x_rows;
    a.Kd = Kd;
    a.scales = scales;
    a.zeros = zeros;
    a.E = E;
    a.N = N;
    a.offsets = offsets;
    a.counts = counts;
    a.src = src;
    a.top_k = top_k;
    a.rows = rows;
    a.status = dev_status;
    a.swiglu = (flags & MOEDC_SWIGLU) != 0;
    a.wait_extra = test_wait_extra();
    a.f16 = dtype == MOEDC_F16;
    if (small) return launch_matvec_small(a, group, out, stream);
    uint8_t* records = static_cast<uint8_t*>(workspace);
    a.records = records;
    // rows that can be filled: `rows` counts what alignment leaves empty as well
    const int64_t filled = src ? (int64_t)x_rows * top_k : rows;
    const bool tc = matvec_tc_takes(E, rows, 128) && matvec_tc_takes(E, (int)(filled < rows ? filled : rows), group);
    if (!tc) mv_shape(a, sm_count());
    const int st = dtype == MOEDC_F16
                       ? launch_matvec_x<__half>(a, tc, records, stream)
                       : launch_matvec_x<__nv_bfloat16>(a, tc, records, stream);
    if (st != MOEDC_OK) return st;
    if (tc) return launch_matvec_tc(a, group, out, stream);
    return scale_dtype == MOEDC_F32   ? launch_matvec_group<float>(a, group, out, stream)
           : scale_dtype == MOEDC_F16 ? launch_matvec_group<__half>(a, group, out, stream)
                                      : launch_matvec_group<__nv_bfloat16>(a, group, out, stream);
}
