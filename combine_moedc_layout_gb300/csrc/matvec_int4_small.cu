// The 4-bit expert products for calls with few weights to read, where launches
// and latency count: one launch, x read as it is, no workspace, no tensor map.
//
// A block takes a tile of 16 weight rows (with SwiGLU 8 gate and 8 up rows) and up
// to eight rows of x; its four warps take 128-channel chunks of K in turn, each
// with the weights of several chunks in flight straight to registers (16 bytes a
// thread and row, turned round within four threads), and add their sums
// in shared memory.  q | 0x4300 is the bf16 number 128 + q (f16: 0x6400, 1024 + q);
// less 128 + z it is q - z, exact in either type (a widely published conversion), so
// the products need no preparation of x beyond its order.  The group's sum is scaled in
// binary32.
#include "matvec_int4.cuh"

namespace moedc {

// Four warps and four blocks an SM: 25 MB 16.5 us; eight warps and two blocks 20.5,
// two warps and eight blocks 20.5 us.
constexpr int kSmThreads = 128;
constexpr int kSmWarps = kSmThreads / kWarp;

template <typename T> struct Int4Of;       // q | magic = base + q, exactly
template <> struct Int4Of<__nv_bfloat16> {
    static constexpr uint32_t magic = 0x43004300u;
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Int4Of<__half> {
    static constexpr uint32_t magic = 0x64006400u;
    static __device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// A scale as it comes from memory: widened only where it is used, since widening
// waits for the load.
template <typename S> using SmRaw = typename std::conditional<sizeof(S) == 4, float, uint16_t>::type;
template <typename S> __device__ __forceinline__ float sm_scale(SmRaw<S> v)
{
    if constexpr (sizeof(S) == 4) return v;
    else if constexpr (std::is_same<S, __half>::value) return __half2float(__ushort_as_half(v));
    else return __uint_as_float((uint32_t)v << 16);
}

// Chunks whose weights are in flight together: as many as registers hold beside
// their scales.
template <int GROUP> constexpr int kSmBatch = GROUP == 128 ? 4 : 2;

// The weights of one chunk of 128 channels: two rows, scales and zero points by
// group.
template <int GROUP, typename S> struct SmChunk {
    static constexpr int groups = 128 / GROUP;
    uint4 w[2];
    SmRaw<S> s[2][groups];
    uint32_t z[2][groups];
};

// Four threads hold four words each, thread t the words of 32 neighbouring channels
// 32 t on; afterwards word j of thread t is word t of thread j, so that the same
// word of the four threads is 32 neighbouring channels.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t)
{
    uint32_t a = t & 1 ? w[0] : w[1], b = t & 1 ? w[2] : w[3];
    a = __shfl_xor_sync(0xffffffffu, a, 1);
    b = __shfl_xor_sync(0xffffffffu, b, 1);
    if (t & 1) w[0] = a, w[2] = b;
    else w[1] = a, w[3] = b;
    a = t & 2 ? w[0] : w[2], b = t & 2 ? w[1] : w[3];
    a = __shfl_xor_sync(0xffffffffu, a, 2);
    b = __shfl_xor_sync(0xffffffffu, b, 2);
    if (t & 2) w[0] = a, w[1] = b;
    else w[2] = a, w[3] = b;
}

template <typename T, int GROUP, typename S>
__global__ void __launch_bounds__(kSmThreads, 4)
matvec_int4_small_kernel(const __grid_constant__ MatvecArgs a, uint16_t* __restrict__ out)
{
    extern __shared__ int32_t s_mem[];       // pre [E + 1], beg [E], end [E]
    __shared__ int64_t s_scan[kSmWarps];
    __shared__ float s_red[kSmWarps][4][kWarp];
    pdl_enter();
    int32_t *s_pre = s_mem, *s_beg = s_pre + a.E + 1, *s_end = s_beg + a.E;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane >> 2, t = lane & 3;
    const int tile_n = a.swiglu ? 8 : 16;
    const int tiles = (a.N + tile_n - 1) / tile_n;
    const int groups = a.Kd / GROUP;
    const int wrows = a.swiglu ? 2 * a.N : a.N;
    const int chunks = (a.Kd + 127) / 128;
    const bool over = mv_chunks<kSmThreads>(a, tiles, s_scan, s_pre, s_beg, s_end);
    const int units = s_pre[a.E] * tiles;
    if (over && blockIdx.x == 0) raise_status(a.status, MOEDC_ERR_CAPACITY);
    bool bad = false;

    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const MvUnit u = mv_unit(a, s_pre, s_beg, s_end, tiles, tile_n, unit);
        // rows past the last read the last one, and nothing uses them
        const int n0 = min(u.n0 + g, a.N - 1), n1 = a.swiglu ? n0 + a.N : min(u.n0 + g + 8, a.N - 1);
        const int64_t row[2] = {(int64_t)u.e * wrows + n0, (int64_t)u.e * wrows + n1};
        const int xr = g < u.m ? x_row(a, u.r0 + g, bad) : a.x_rows;
        const T* x = xr < a.x_rows ? static_cast<const T*>(a.x) + (int64_t)xr * a.ldx + t * 8 : nullptr;
        auto load = [&](int c, SmChunk<GROUP, S>& k) __attribute__((always_inline)) {
            const bool in = c * 128 + t * 32 < a.Kd;
#pragma unroll
            for (int r = 0; r < 2; ++r)
                k.w[r] = in ? ld_global_nc(reinterpret_cast<const uint4*>(a.wq + row[r] * (a.Kd / 2) + c * 64 + t * 16))
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < SmChunk<GROUP, S>::groups; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int64_t at = row[r] * groups + min(c * SmChunk<GROUP, S>::groups + q, groups - 1);
                    k.s[r][q] = __ldg(static_cast<const SmRaw<S>*>(a.scales) + at);
                    k.z[r][q] = a.zeros ? __ldg(a.zeros + at) : 8u;
                }
        };
        auto load_x = [&](int c, uint4 (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = x && c * 128 + j * 32 < a.Kd ? __ldg(reinterpret_cast<const uint4*>(x + c * 128 + j * 32))
                                                    : make_uint4(0, 0, 0, 0);
        };
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        auto add = [&](int c, const SmChunk<GROUP, S>& k, const uint4 (&xv)[4]) __attribute__((always_inline)) {
            uint32_t wa[4] = {k.w[0].x, k.w[0].y, k.w[0].z, k.w[0].w};
            uint32_t wb[4] = {k.w[1].x, k.w[1].y, k.w[1].z, k.w[1].w};
            quad_transpose(wa, t);
            quad_transpose(wb, t);
#pragma unroll
            for (int q = 0; q < SmChunk<GROUP, S>::groups; ++q) {
                if (c * 128 + q * GROUP >= a.Kd) break;
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const uint32_t za = Int4Of<T>::magic | k.z[0][q] * 0x00010001u;
                const uint32_t zb = Int4Of<T>::magic | k.z[1][q] * 0x00010001u;
#pragma unroll
                for (int j = q * GROUP / 32; j < (q + 1) * GROUP / 32; ++j) {
                    uint32_t m[8];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        m[2 * p] = Int4Of<T>::minus(((wa[j] >> (4 * p)) & 0x000f000fu) | Int4Of<T>::magic, za);
                        m[2 * p + 1] = Int4Of<T>::minus(((wb[j] >> (4 * p)) & 0x000f000fu) | Int4Of<T>::magic, zb);
                    }
                    // registers of weights p and p + 4 of a word, x in the same pairs
                    const uint4 v = xv[j];
                    Int4Of<T>::mma(d, m, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
                    Int4Of<T>::mma(d, m + 4, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                }
                const float s0 = sm_scale<S>(k.s[0][q]), s1 = sm_scale<S>(k.s[1][q]);
                acc[0] = fmaf(s0, d[0], acc[0]);
                acc[1] = fmaf(s0, d[1], acc[1]);
                acc[2] = fmaf(s1, d[2], acc[2]);
                acc[3] = fmaf(s1, d[3], acc[3]);
            }
        };
        // a part past the last chunk loads zeros and the last scale, and adds nothing
        constexpr int kB = kSmBatch<GROUP>;
        for (int c = warp; c < chunks; c += kB * kSmWarps) {
            SmChunk<GROUP, S> k[kB];
#pragma unroll
            for (int b = 0; b < kB; ++b) load(c + b * kSmWarps, k[b]);
            uint4 now[4], next[4];
            load_x(c, now);
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                if (b + 1 < kB) load_x(c + (b + 1) * kSmWarps, next);
                add(c + b * kSmWarps, k[b], now);
#pragma unroll
                for (int j = 0; j < 4; ++j) now[j] = next[j];
            }
        }
        __syncthreads();                       // the unit before has been read
#pragma unroll
        for (int j = 0; j < 4; ++j) s_red[warp][j][lane] = acc[j];
        __syncthreads();
        if (warp != 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = 0.0f;
#pragma unroll
            for (int w = 0; w < kSmWarps; ++w) acc[j] += s_red[w][j][lane];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = t * 2 + c;
            if (r >= u.m) continue;
            uint16_t* o = out + (int64_t)(u.r0 + r) * a.N;
            const int n = u.n0 + g;
            if (a.swiglu) {
                const float v = acc[c];
                if (n < a.N) store16(o + n, v / (1.0f + expf(-v)) * acc[2 + c], a.f16);
            } else {
                if (n < a.N) store16(o + n, acc[c], a.f16);
                if (n + 8 < a.N) store16(o + n + 8, acc[2 + c], a.f16);
            }
        }
    }
    if (bad) raise_status(a.status, MOEDC_ERR_EXPERT_RANGE);
}

}  // namespace moedc

namespace moedc_host {
namespace {

template <typename T, int GROUP, typename S>
int launch_small(const moedc::MatvecArgs& a, void* out, cudaStream_t stream)
{
    auto* k = moedc::matvec_int4_small_kernel<T, GROUP, S>;
    const size_t smem = (3 * (size_t)a.E + 1) * sizeof(int32_t);
    const int tile_n = a.swiglu ? 8 : 16;
    const int64_t want = ((int64_t)a.rows / 8 + (a.E < a.rows ? a.E : a.rows)) * ((a.N + tile_n - 1) / tile_n);
    const int64_t most = resident_blocks((const void*)k, moedc::kSmThreads, smem);
    clear_stale_error();
    launch(k, (int)(want < most ? want : most), moedc::kSmThreads, smem, stream, a, static_cast<uint16_t*>(out));
    return launch_status();
}

template <typename T, int GROUP>
int launch_small_scale(const moedc::MatvecArgs& a, void* out, cudaStream_t stream)
{
    return a.scale_dtype == MOEDC_F32   ? launch_small<T, GROUP, float>(a, out, stream)
           : a.scale_dtype == MOEDC_F16 ? launch_small<T, GROUP, __half>(a, out, stream)
                                        : launch_small<T, GROUP, __nv_bfloat16>(a, out, stream);
}

}  // namespace

#ifndef MOEDC_SMALL_BYTES
#define MOEDC_SMALL_BYTES (25ll << 20)
#endif

// Few weights to read, each expert's rows (eight at a time read them again, from
// L2) counted.  Time on the GPU, this form / the one with prepared x: 2 MB 8.1 /
// 10.3 us, 18 MB 11.8 / 12.3 us (with SwiGLU 14.4 / 12.3), 20 MB 12.3 / 13.0 us, 25 MB
// 16.4 / 16.4 us, 36 MB 20.5 / 16.4 us; on the host this form saves a launch, a tensor
// map and the workspace, some 6 us of 20.
bool matvec_small_takes(int Kd, int E, int N, bool swiglu, int rows)
{
    const int64_t active = E < rows ? E : rows;
    const double reads = (double)(active + rows / 8) * N * (swiglu ? 2 : 1);
    return reads * (Kd / 2) <= (double)MOEDC_SMALL_BYTES;
}

int launch_matvec_small(const moedc::MatvecArgs& b, int group, void* out, cudaStream_t stream)
{
    moedc::MatvecArgs a = b;
    a.chunk_rows = 8;
    if (a.f16)
        return group == 32   ? launch_small_scale<__half, 32>(a, out, stream)
               : group == 64 ? launch_small_scale<__half, 64>(a, out, stream)
                             : launch_small_scale<__half, 128>(a, out, stream);
    return group == 32   ? launch_small_scale<__nv_bfloat16, 32>(a, out, stream)
           : group == 64 ? launch_small_scale<__nv_bfloat16, 64>(a, out, stream)
                         : launch_small_scale<__nv_bfloat16, 128>(a, out, stream);
}

}  // namespace moedc_host
