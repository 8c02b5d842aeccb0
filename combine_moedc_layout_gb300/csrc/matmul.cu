// Entry points of the 16-bit products of packed expert rows, and the elementwise
// gradient of the gate.
#include "matmul.cuh"

namespace moedc {

// A thread owns eight channels of a row: 6 bytes read and 4 written for each, HBM, and where the
// rows are few the operations too (65536 rows x 2048: 216 us with cold caches, 6.2 TB/s; 8192
// rows 35 us, 4.7).
//   du = dh g s;  dg = dh u s (1 + g (1 - s)),  s = 1 / (1 + exp(-g))
// from left to right, each operation rounded by itself, as the formulas read: the result is
// rounded to 16 bits, and the products of the backward pass take it from there, so a last bit
// that another order turns is one of the gradients'.  Where exp(-g) overflows, s is exp(g).
template <typename T>
__global__ void swiglu_grad_kernel(const T* __restrict__ dh, int64_t ld, const T* products, int rows, int N,
                                   T* dproducts)   // may be one buffer
{
    pdl_enter();
    const int vecs = N / 8;
    const int64_t n = (int64_t)rows * vecs;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / vecs;
        const int c = (int)(i - row * vecs) * 8;
        const T* p = products + row * 2 * N + c;
        T* d = dproducts + row * 2 * N + c;
        float h[8], g[8], u[8];
        Unit<T, 8>::widen(__ldg(reinterpret_cast<const uint4*>(dh + row * ld + c)), h);
        Unit<T, 8>::widen(*reinterpret_cast<const uint4*>(p), g);
        Unit<T, 8>::widen(*reinterpret_cast<const uint4*>(p + N), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = expf(-g[j]);
            const float s = isinf(e) ? expf(g[j]) : __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
            const float slope = __fadd_rn(1.0f, __fmul_rn(g[j], __fadd_rn(1.0f, -s)));
            const float dg = __fmul_rn(__fmul_rn(__fmul_rn(h[j], u[j]), s), slope);
            u[j] = __fmul_rn(__fmul_rn(h[j], g[j]), s);
            g[j] = dg;
        }
        *reinterpret_cast<uint4*>(d) = Unit<T, 8>::round(g);
        *reinterpret_cast<uint4*>(d + N) = Unit<T, 8>::round(u);
    }
}

}  // namespace moedc

namespace moedc_host {
namespace {

// what the calls over packed rows have in common
bool groups_ok(int E, int rows, const int32_t* offsets, const int32_t* counts, const int32_t* dev_status)
{
    if (E < 1 || E > MOEDC_MAX_E || rows < 0) return false;
    if (!counts && (offsets || E != 1)) return false;
    if (counts && !offsets && rows % E != 0) return false;
    return dev_status && aligned(offsets, 4) && aligned(counts, 4) && aligned(dev_status, 4);
}
bool dim_ok(int n) { return n >= 8 && n % 8 == 0; }
bool type_ok(int dtype) { return dtype == MOEDC_BF16 || dtype == MOEDC_F16; }

moedc::MmArgs args(int E, int N, int K, int rows, const int32_t* offsets, const int32_t* counts, int dtype, int32_t* status)
{
    moedc::MmArgs a{};
    a.E = E;
    a.N = N;
    a.K = K;
    a.rows = a.x_rows = rows;
    a.slots = rows / E;
    a.offsets = offsets;
    a.counts = counts;
    a.status = status;
    a.f16 = dtype == MOEDC_F16;
    a.vec = true;
    a.wait_extra = test_wait_extra();
    return a;
}

// units are counted in 32 bits
bool units_ok(int64_t rows, int64_t E, int64_t columns) { return (rows / 256 + E) * (columns / 128 + 1) <= INT32_MAX; }

template <typename T>
void launch_swiglu_grad(const void* dh, int64_t ld, const void* products, int rows, int N, void* out, cudaStream_t stream)
{
    const int64_t want = ((int64_t)rows * (N / 8) + 255) / 256, most = 16 * (int64_t)sm_count();
    launch(moedc::swiglu_grad_kernel<T>, (int)(want < most ? want : most), 256, 0, stream, static_cast<const T*>(dh), ld,
           static_cast<const T*>(products), rows, N, static_cast<T*>(out));
}

}  // namespace
}  // namespace moedc_host

extern "C" int moedc_matmul(const void* x, int64_t ldx, int dtype, int Kd, const void* w, int E, int N, int flags,
                            const int32_t* offsets, const int32_t* counts, int rows, void* out, void* products,
                            int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    const bool gated = (flags & MOEDC_SWIGLU) != 0;
    if (!type_ok(dtype) || !dim_ok(Kd) || !dim_ok(N) || (flags & ~MOEDC_SWIGLU) != 0 || (products && !gated) ||
        !groups_ok(E, rows, offsets, counts, dev_status))
        return MOEDC_ERR_ARG;
    if (!w || ldx < Kd || ldx % 8 != 0 || N > INT32_MAX / 2 || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) ||
        !aligned(products, 16) || !units_ok(rows, E, N))
        return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!x || !out) return MOEDC_ERR_ARG;
    moedc::MmArgs a = args(E, N, Kd, rows, offsets, counts, dtype, dev_status);
    a.gated = gated;
    a.out = out;
    a.extra = products;
    return launch_mm_forward(a, x, ldx, w, stream);
}

extern "C" int moedc_swiglu_grad(const void* dh, int64_t lddh, const void* products, int dtype, int rows, int N,
                                 void* dproducts, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!type_ok(dtype) || !dim_ok(N) || rows < 0 || lddh < N || lddh % 8 != 0 || !aligned(dh, 16) ||
        !aligned(products, 16) || !aligned(dproducts, 16))
        return MOEDC_ERR_ARG;
    if (rows == 0) return MOEDC_OK;
    if (!dh || !products || !dproducts) return MOEDC_ERR_ARG;
    clear_stale_error();
    if (dtype == MOEDC_F16) launch_swiglu_grad<__half>(dh, lddh, products, rows, N, dproducts, stream);
    else launch_swiglu_grad<__nv_bfloat16>(dh, lddh, products, rows, N, dproducts, stream);
    return launch_status();
}

extern "C" int moedc_matmul_grad(const void* dout, int64_t lddout, const void* x, int64_t ldx, const void* w, int dtype,
                                 int Kd, int E, int N, const int32_t* offsets, const int32_t* counts, int rows, void* dx,
                                 void* dw, int dw_dtype, int32_t* dev_status, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!type_ok(dtype) || !dim_ok(Kd) || !dim_ok(N) || !groups_ok(E, rows, offsets, counts, dev_status))
        return MOEDC_ERR_ARG;
    if (dw && dw_dtype != dtype && dw_dtype != MOEDC_F32) return MOEDC_ERR_ARG;
    if (lddout < N || lddout % 8 != 0 || !aligned(dout, 16) || !aligned(dx, 16) || !aligned(dw, 16) ||
        !units_ok(rows, E, Kd) || (int64_t)E * (N / 256 + 1) * (Kd / 256 + 1) > INT32_MAX)
        return MOEDC_ERR_ARG;
    if (dx && (!w || !aligned(w, 16))) return MOEDC_ERR_ARG;
    if (dw && (ldx < Kd || ldx % 8 != 0 || !aligned(x, 16))) return MOEDC_ERR_ARG;
    if (rows == 0) {
        if (!dw) return MOEDC_OK;
        clear_stale_error();
        (void)cudaMemsetAsync(dw, 0, (size_t)E * N * Kd * lm_dtype_size(dw_dtype), stream);
        return launch_status();
    }
    if (!dout || (dw && !x)) return MOEDC_ERR_ARG;
    if (dx) {
        moedc::MmArgs a = args(E, Kd, N, rows, offsets, counts, dtype, dev_status);
        a.out = dx;
        const int st = launch_mm_dx(a, dout, lddout, w, stream);
        if (st != MOEDC_OK) return st;
    }
    if (dw) {
        moedc::MmArgs a = args(E, Kd, 0, rows, offsets, counts, dtype, dev_status);
        a.M = N;
        a.out = dw;
        a.f32 = dw_dtype == MOEDC_F32;
        return launch_mm_dw(a, dout, lddout, x, ldx, stream);
    }
    return MOEDC_OK;
}
