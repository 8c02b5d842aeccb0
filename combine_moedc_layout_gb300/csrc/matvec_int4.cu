// Products of packed expert rows with 4-bit weights and group scales:
//   out[r][n] = sum_k x[r'][k] (q[e][n][k] - z[e][n][k/g]) s[e][n][k/g]
// for the expert e whose rows hold r.
//
// A decode step gives each expert a handful of rows, so the stream of weights
// from HBM bounds it (half a byte per weight, each read once), and what the
// SMs do per weight has to fit under that stream: 46 weights per SM and clock.
//
// Work is cut into units of (expert, tile of output channels, chunk of rows).
// A block of eight warps takes units in turn; each warp owns 16 weight rows of
// the tile and, when there are few tiles, one of `wk` interleaved parts of K
// (the parts are added in shared memory at the unit's end).  Weights, scales
// and the rows of x travel through a ring of cp.async stages that runs on
// across units, so the stream never drains between them.
//
// The products run on the tensor cores with the weights as the 16-row operand
// and eight rows of x as the other.  A weight never leaves registers between
// its unpacking and its product: q | 0x4300 is the bf16 number 128 + q (f16:
// 0x6400, 1024 + q), and subtracting 128 + z leaves q - z, exact in either
// type.  The group's sum is formed in binary32 from these integers and only
// then multiplied by the group's scale, so neither weights nor scales are ever
// rounded.  tcgen05 reads its operands from shared or tensor memory, which
// would cost every weight a 2-byte store and a 2-byte read on the way: at the
// HBM rate 93 + 93 bytes per SM and clock, more than shared memory moves (128).
#include <climits>

#include "lm_common.cuh"

namespace moedc {

constexpr int kMvThreads = 256;
constexpr int kMvWarps = kMvThreads / kWarp;
constexpr int kMvChunk = 128;              // channels of one warp's part of a stage
constexpr int kMvTokens = 32;              // rows x parts of K staged together: 32 / wk rows
// one stage: weights (16 rows x 64 bytes per warp), x, scales and zero points
// (a 4-byte word for each weight row and group); as many stages as let two
// blocks share an SM
constexpr int kMvW = kMvWarps * 16 * 64;
constexpr int kMvX = kMvTokens * kMvChunk * 2;
constexpr int kMvRed = kMvWarps * 8 * kWarp * (int)sizeof(float);
template <int GROUP> struct MvRing {
    static constexpr int per_warp = 16 * 4 * (kMvChunk / GROUP);   // scale words
    static constexpr int words = kMvWarps * per_warp;
    static constexpr int stage = kMvW + kMvX + 2 * words;
    static constexpr int stages = GROUP == 128 ? 6 : 5;
};

struct MatvecArgs {
    const void* x;
    int64_t ldx;
    int x_rows, Kd;
    const uint8_t* wq;
    const void* scales;
    int scale_dtype;
    const uint8_t* zeros;
    int E, N;
    const int32_t *offsets, *counts, *src;
    int top_k, rows;
    int32_t* status;
    int lk;          // log2 of the parts of K
    bool swiglu;
};

// `bytes` of the 16 (or 4) are read, the rest is written as zeros
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                     (unsigned)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T> struct Int4Of;       // q | magic = base + q, exactly
template <> struct Int4Of<__nv_bfloat16> {
    static constexpr uint32_t magic = 0x43004300u;      // 128
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Int4Of<__half> {
    static constexpr uint32_t magic = 0x64006400u;      // 1024
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// A unit: rows [r0, r0 + m) of expert e and the tile's first output channel.
struct MvUnit {
    int e, n0, r0, m;
};

// First and last row of an expert, inside [0, rows].
__device__ __forceinline__ void expert_rows(const MatvecArgs& a, int e, int& beg, int& end,
                                            bool& over)
{
    int64_t b = a.offsets ? __ldg(a.offsets + e) : 0;
    int64_t n = b + (a.counts ? __ldg(a.counts + e) : a.rows);
    if (b < 0) b = 0;
    if (n > a.rows) {
        n = a.rows;
        over = true;
    }
    beg = (int)(b < n ? b : 0);
    end = (int)(b < n ? n : 0);
}

// s_pre[e]: chunks of the experts before e
__device__ __forceinline__ MvUnit mv_unit(const MatvecArgs& a, const int32_t* s_pre, int tiles,
                                          int tile_n, int chunk_rows, int unit)
{
    int lo = 0, hi = a.E - 1;   // last expert whose units begin at or before `unit`
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (s_pre[mid] * tiles <= unit) lo = mid; else hi = mid - 1;
    }
    const int chunks = s_pre[lo + 1] - s_pre[lo];
    const int in = unit - s_pre[lo] * tiles;
    const int tile = in / chunks, chunk = in - tile * chunks;   // chunks of one tile are neighbours
    int beg, end;
    bool over = false;
    expert_rows(a, lo, beg, end, over);
    MvUnit u;
    u.e = lo;
    u.n0 = tile * tile_n;
    u.r0 = beg + chunk * chunk_rows;
    u.m = min(chunk_rows, end - u.r0);
    return u;
}

// Weight row that row i (0..15) of a warp's tile holds, -1 past the end: with
// SwiGLU rows 0..7 are gate rows and rows 8..15 the up rows of the same outputs,
// so that a thread holds both.
__device__ __forceinline__ int mv_weight_row(const MatvecArgs& a, int n0, int i)
{
    const int n = a.swiglu ? n0 + (i & 7) : n0 + i;
    if (n >= a.N) return -1;
    return a.swiglu && i >= 8 ? a.N + n : n;
}

// One stage of one warp: 16 weight rows x 128 channels with 8 NT rows of x.
// at0, at1: index (modulo 4) of the first scale and zero point of rows g and
// g + 8, which tells their place in the words.
template <typename T, int GROUP, int NT>
__device__ __forceinline__ void mv_stage(const uint8_t* sw, const uint8_t* sx, const uint8_t* ss,
                                         int scale_dtype, bool zeros, int at0, int at1, int steps,
                                         float (&acc)[NT][4])
{
    const int lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    constexpr int kPer = GROUP / 32;       // 32-channel steps of a group
    float tmp[NT][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w >= steps) break;
        if (w % kPer == 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) tmp[i][j] = 0.0f;
        }
        const int q = w / kPer;            // the stage's group
        const uint8_t* sq = ss + q * 64;   // its words: [16 rows]
        uint32_t za, zb;
        if (zeros) {
            const uint8_t* sz = sq + MvRing<GROUP>::words;
            const uint32_t a = sz[g * 4 + ((at0 + q) & 3)];
            const uint32_t b = sz[(g + 8) * 4 + ((at1 + q) & 3)];
            za = Int4Of<T>::magic | a | a << 16;
            zb = Int4Of<T>::magic | b | b << 16;
        } else {
            za = zb = Int4Of<T>::magic | 0x00080008u;
        }
        const uint8_t* row = sw + g * 64 + ((w ^ ((g >> 1) & 3)) << 4) + t * 4;
        const uint32_t wa = *reinterpret_cast<const uint32_t*>(row);
        const uint32_t wb = *reinterpret_cast<const uint32_t*>(row + 8 * 64);
        // register p holds weights p and p + 4 of the word
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            lo[p] = Int4Of<T>::minus(((wa >> (4 * p)) & 0x000f000fu) | Int4Of<T>::magic, za);
            hi[p] = Int4Of<T>::minus(((wb >> (4 * p)) & 0x000f000fu) | Int4Of<T>::magic, zb);
        }
        const uint32_t a01[4] = {lo[0], hi[0], lo[1], hi[1]};
        const uint32_t a23[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(
                sx + (i * 8 + g) * 256 + (((w * 4 + t) ^ ((g & 1) << 2)) << 4));
            Int4Of<T>::mma(tmp[i], a01, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
            Int4Of<T>::mma(tmp[i], a23, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
        if (w % kPer == kPer - 1) {
            float s0, s1;
            if (scale_dtype == MOEDC_F32) {
                s0 = *reinterpret_cast<const float*>(sq + g * 4);
                s1 = *reinterpret_cast<const float*>(sq + (g + 8) * 4);
            } else {
                const uint32_t h0 = *reinterpret_cast<const uint16_t*>(sq + g * 4 + ((at0 + q) & 1) * 2);
                const uint32_t h1 = *reinterpret_cast<const uint16_t*>(sq + (g + 8) * 4 + ((at1 + q) & 1) * 2);
                if (scale_dtype == MOEDC_BF16) {
                    s0 = __uint_as_float(h0 << 16);
                    s1 = __uint_as_float(h1 << 16);
                } else {
                    s0 = __half2float(__ushort_as_half((unsigned short)h0));
                    s1 = __half2float(__ushort_as_half((unsigned short)h1));
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                acc[i][0] = fmaf(s0, tmp[i][0], acc[i][0]);
                acc[i][1] = fmaf(s0, tmp[i][1], acc[i][1]);
                acc[i][2] = fmaf(s1, tmp[i][2], acc[i][2]);
                acc[i][3] = fmaf(s1, tmp[i][3], acc[i][3]);
            }
        }
    }
}

// The unit's end: the parts of K added, the epilogue, the outputs.
template <typename T, int NT>
__device__ __forceinline__ void mv_store(const MatvecArgs& a, const MvUnit& u, float* s_red,
                                         float (&acc)[NT][4], T* __restrict__ out)
{
    const int lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x / kWarp;
    const int wk = 1 << a.lk, part = warp & (wk - 1), tile = warp >> a.lk;
    if (wk > 1) {
        // [warp][value][lane]: conflict-free
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s_red[(warp * NT * 4 + i * 4 + j) * kWarp + lane] = acc[i][j];
        __syncthreads();
        if (part != 0) return;
        for (int p = 1; p < wk; ++p)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += s_red[((warp + p) * NT * 4 + i * 4 + j) * kWarp + lane];
    }
    const int n0 = u.n0 + tile * (a.swiglu ? 8 : 16);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = i * 8 + t * 2 + c;
            if (r >= u.m) continue;
            T* o = out + (int64_t)(u.r0 + r) * a.N;
            if (a.swiglu) {
                const float v = acc[i][c];
                if (n0 + g < a.N) o[n0 + g] = from_f32<T>(v / (1.0f + expf(-v)) * acc[i][2 + c]);
            } else {
                if (n0 + g < a.N) o[n0 + g] = from_f32<T>(acc[i][c]);
                if (n0 + g + 8 < a.N) o[n0 + g + 8] = from_f32<T>(acc[i][2 + c]);
            }
        }
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(kMvThreads, 2)
matvec_int4_kernel(const __grid_constant__ MatvecArgs a, T* __restrict__ out)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kMvWarps];
    pdl_enter();
    using Ring = MvRing<GROUP>;
    constexpr int kStage = Ring::stage, kStages = Ring::stages;
    uint8_t* ring = smem;
    float* s_red = reinterpret_cast<float*>(smem + kStages * kStage);
    int32_t* s_pre = reinterpret_cast<int32_t*>(smem + kStages * kStage + kMvRed);

    const int lane = threadIdx.x % kWarp, g = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x / kWarp;
    const int wk = 1 << a.lk, part = warp & (wk - 1), tile = warp >> a.lk;
    const int chunk_rows = kMvTokens >> a.lk;
    const int tile_n = (kMvWarps >> a.lk) * (a.swiglu ? 8 : 16);
    const int tiles = (a.N + tile_n - 1) / tile_n;
    const int groups = a.Kd / GROUP;
    const int wrows = a.swiglu ? 2 * a.N : a.N;
    const int ksteps = (a.Kd + (kMvChunk << a.lk) - 1) / (kMvChunk << a.lk);

    // chunks of the experts before each one
    bool bad = false, over = false;
    {
        const int per = (a.E + kMvThreads - 1) / kMvThreads;
        const int e0 = threadIdx.x * per;
        int64_t sum = 0;
        for (int e = e0; e < min(a.E, e0 + per); ++e) {
            int beg, end;
            expert_rows(a, e, beg, end, over);
            const int c = (end - beg) / chunk_rows + ((end - beg) % chunk_rows != 0);
            s_pre[e] = c;
            sum += c;
        }
        int64_t incl = sum;
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == kWarp - 1) s_scan[warp] = incl;
        __syncthreads();
        int64_t base = incl - sum;
        for (int w = 0; w < warp; ++w) base += s_scan[w];
        for (int e = e0; e < min(a.E, e0 + per); ++e) {
            const int c = s_pre[e];
            s_pre[e] = (int)base;
            base += c;
        }
        // experts that overlap could claim more units than there are numbers: none then
        if (e0 < a.E && e0 + per >= a.E) {
            const bool fits = base * tiles <= INT_MAX;
            s_pre[a.E] = fits ? (int)base : 0;
            over |= !fits;
        }
        __syncthreads();
    }
    const int units = s_pre[a.E] * tiles;
    if (over) raise_status(a.status, MOEDC_ERR_CAPACITY);

    // ---- what this thread copies, for the unit the ring's head is in
    int p_unit = blockIdx.x, p_step = 0;
    const uint8_t* p_w[2];      // rows g and g + 8, 16 bytes t of 64
    int64_t p_s[2];             // their first scale's index
    const uint8_t* p_x[2];      // two pieces of x: token (and part) by thread, null: zeros
    auto open = [&]() {
        const MvUnit u = mv_unit(a, s_pre, tiles, tile_n, chunk_rows, p_unit);
        const int n0 = u.n0 + tile * (a.swiglu ? 8 : 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = mv_weight_row(a, n0, g + 8 * i);
            const int64_t row = (int64_t)u.e * wrows + n;
            p_w[i] = n < 0 ? nullptr : a.wq + row * (a.Kd / 2) + t * 16;
            p_s[i] = n < 0 ? -1 : row * groups;
            // pieces of x: thread i * 256 + tid of [32 / wk rows][wk parts][16 pieces]
            const int id = i * kMvThreads + threadIdx.x;
            const int r = id >> (4 + a.lk);
            int64_t xr = -1;
            if (r < u.m) {
                xr = u.r0 + r;
                if (a.src) {
                    const int at = __ldg(a.src + u.r0 + r);
                    xr = at < 0 ? -1 : at / a.top_k;
                }
                if (xr < 0 || xr >= a.x_rows) {
                    xr = -1;
                    bad = true;
                }
            }
            p_x[i] = xr < 0 ? nullptr : static_cast<const uint8_t*>(a.x) + xr * a.ldx * 2;
        }
    };
    auto issue = [&](int slot) {
        if (p_unit < units) {
            if (p_step == 0) open();
            uint8_t* st = ring + slot * kStage;
            const int k0 = (p_step << a.lk) * kMvChunk;            // of the stage
            const int kw = k0 + part * kMvChunk;                   // of this warp
            uint8_t* w = st + warp * 1024 + g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool ok = p_w[i] && kw + t * 32 < a.Kd;
                cp_async16(w + i * 512, ok ? p_w[i] + kw / 2 : a.wq, ok ? 16 : 0);
                const int id = i * kMvThreads + threadIdx.x;
                const int c = id & 15, xp = (id >> 4) & (wk - 1), r = id >> (4 + a.lk);
                const int kx = k0 + xp * kMvChunk + c * 8;
                const bool okx = p_x[i] && kx < a.Kd;
                cp_async16(st + kMvW + (xp * chunk_rows + r) * 256 + ((c ^ ((r & 1) << 2)) << 4),
                           okx ? p_x[i] + (int64_t)kx * 2 : a.x, okx ? 16 : 0);
            }
            // scales and zero points of (row, group): the aligned 4-byte word that holds each.
            // Lane t of row g takes groups t of its two rows.
            constexpr int kGroups = kMvChunk / GROUP;
            const int gi = kw / GROUP + t;
            if (t < kGroups && gi < groups) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (p_s[i] < 0) continue;
                    const int64_t at = p_s[i] + gi;
                    const int64_t total = (int64_t)a.E * wrows * groups;
                    uint8_t* s = st + kMvW + kMvX + warp * Ring::per_warp + t * 64 + (g + 8 * i) * 4;
                    if (a.scale_dtype == MOEDC_F32) {
                        cp_async4(s, static_cast<const float*>(a.scales) + at, 4);
                    } else {
                        const int64_t w2 = at & ~(int64_t)1;
                        cp_async4(s, static_cast<const uint16_t*>(a.scales) + w2, w2 + 1 < total ? 4 : 2);
                    }
                    if (a.zeros) {
                        const int64_t w4 = at & ~(int64_t)3;
                        cp_async4(s + Ring::words, a.zeros + w4, (int)min((int64_t)4, total - w4));
                    }
                }
            }
            if (++p_step == ksteps) {
                p_step = 0;
                p_unit += gridDim.x;
            }
        }
        cp_async_commit();   // an empty group past the end keeps the count
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s);

    int slot = 0;
    // one unit with 8 NT rows of x
    auto run = [&](auto nt, const MvUnit& u) {
        constexpr int NT = decltype(nt)::value;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        const int n0 = u.n0 + tile * (a.swiglu ? 8 : 16);
        const int64_t base = (int64_t)u.e * wrows;
        const int i0 = (int)(((base + mv_weight_row(a, n0, g)) * groups) & 3);
        const int i1 = (int)(((base + mv_weight_row(a, n0, g + 8)) * groups) & 3);
        for (int s = 0; s < ksteps; ++s) {
            cp_async_wait<kStages - 2>();
            __syncthreads();
            issue(slot == 0 ? kStages - 1 : slot - 1);
            const uint8_t* st = ring + slot * kStage;
            const int kw = ((s << a.lk) + part) * kMvChunk;
            const int g0 = kw / GROUP;
            mv_stage<T, GROUP, NT>(st + warp * 1024, st + kMvW + part * chunk_rows * 256,
                                   st + kMvW + kMvX + warp * Ring::per_warp, a.scale_dtype,
                                   a.zeros != nullptr, i0 + g0, i1 + g0,
                                   min(4, (a.Kd - kw) / 32), acc);
            slot = slot + 1 == kStages ? 0 : slot + 1;
        }
        mv_store<T, NT>(a, u, s_red, acc, out);
    };
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const MvUnit u = mv_unit(a, s_pre, tiles, tile_n, chunk_rows, unit);
        if (u.m <= 8) run(std::integral_constant<int, 1>{}, u);
        else if (u.m <= 16) run(std::integral_constant<int, 2>{}, u);
        else run(std::integral_constant<int, 4>{}, u);
    }
    cp_async_wait<0>();
    if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
}

}  // namespace moedc

namespace moedc_host {
namespace {

template <int GROUP> size_t mv_smem(int E)
{
    using Ring = moedc::MvRing<GROUP>;
    return (size_t)Ring::stages * Ring::stage + moedc::kMvRed + (size_t)(E + 1) * sizeof(int32_t);
}

template <typename T, int GROUP>
int launch_matvec(moedc::MatvecArgs a, void* out, cudaStream_t stream)
{
    auto* k = moedc::matvec_int4_kernel<T, GROUP>;
    const size_t smem = mv_smem<GROUP>(a.E);
    if (cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)mv_smem<GROUP>(MOEDC_MAX_E)) != cudaSuccess)
        return MOEDC_ERR_CUDA;
    const int resident = resident_blocks((const void*)k, moedc::kMvThreads, smem);
    // parts of K: as few as give every block some eight units (the last round of
    // units is then at most an eighth of the work), counting every expert that
    // can have rows
    const int64_t active = a.E < a.rows ? a.E : a.rows;
    const int64_t per = (a.rows + active - 1) / active;
    int64_t units = 0;
    for (a.lk = 0;; ++a.lk) {
        const int tile_n = (moedc::kMvWarps >> a.lk) * (a.swiglu ? 8 : 16);
        const int chunk = moedc::kMvTokens >> a.lk;
        units = active * ((a.N + tile_n - 1) / tile_n) * ((per + chunk - 1) / chunk);
        if (a.lk == 2 || units >= 8 * (int64_t)resident) break;
    }
    clear_stale_error();
    launch(k, (int)(units < resident ? units : resident), moedc::kMvThreads, smem, stream, a,
           static_cast<T*>(out));
    return launch_status();
}

template <typename T>
int launch_matvec_group(const moedc::MatvecArgs& a, int group, void* out, cudaStream_t stream)
{
    return group == 32   ? launch_matvec<T, 32>(a, out, stream)
           : group == 64 ? launch_matvec<T, 64>(a, out, stream)
                         : launch_matvec<T, 128>(a, out, stream);
}

}  // namespace
}  // namespace moedc_host

extern "C" int moedc_matvec_int4(const void* x, int64_t ldx, int dtype, int x_rows, int Kd,
                                 const void* wq, const void* scales, int scale_dtype,
                                 const uint8_t* zeros, int group, int E, int N, int flags,
                                 const int32_t* offsets, const int32_t* counts,
                                 const int32_t* src, int top_k, int rows, void* out,
                                 int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    if ((dtype != MOEDC_BF16 && dtype != MOEDC_F16) || !lm_dtype_ok(scale_dtype)) return MOEDC_ERR_ARG;
    if (group != 32 && group != 64 && group != 128) return MOEDC_ERR_ARG;
    if (Kd < group || Kd % group != 0 || E < 1 || E > MOEDC_MAX_E || N < 1 || x_rows < 0 ||
        rows < 0 || (flags & ~MOEDC_SWIGLU) != 0 || (flags && N > INT32_MAX / 2))
        return MOEDC_ERR_ARG;
    if ((offsets == nullptr) != (counts == nullptr) || (!offsets && E != 1)) return MOEDC_ERR_ARG;
    if (src && top_k < 1) return MOEDC_ERR_ARG;
    if (!wq || !scales || !dev_status || ldx < Kd || ldx % 8 != 0) return MOEDC_ERR_ARG;
    if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(scales, 4) || !aligned(zeros, 4) ||
        !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(src, 4) || !aligned(out, 2) ||
        !aligned(dev_status, 4))
        return MOEDC_ERR_ARG;
    // units (expert, tile, chunk of at least 8 rows) are counted in 32 bits
    if (((int64_t)rows / 8 + E) * ((int64_t)N / 16 + 1) > INT32_MAX) return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!out || !x) return MOEDC_ERR_ARG;
    const moedc::MatvecArgs a{x, ldx, x_rows, Kd, static_cast<const uint8_t*>(wq), scales,
                              scale_dtype, zeros, E, N, offsets, counts, src, top_k, rows,
                              dev_status, 0, (flags & MOEDC_SWIGLU) != 0};
    return dtype == MOEDC_F16 ? launch_matvec_group<__half>(a, group, out, stream)
                              : launch_matvec_group<__nv_bfloat16>(a, group, out, stream);
}
