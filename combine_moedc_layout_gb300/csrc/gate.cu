// Top-k router and its gradient: one warp per token.
//
// With l the token's logits, key = l + bias and the chosen set C the K largest
// keys, the weights are softmax(l) or sigmoid(l), over all experts or
// renormalised over C, times scale.  The gradient follows from w alone:
// with p = w / scale and d the weights' gradient on C,
//   softmax            dl_e = scale * p_e * (d_e - sum_C p d), d_e = 0 outside C
//   sigmoid            dl_e = scale * d_e * s_e (1 - s_e)
//   sigmoid over C     dl_e = scale * s_e (1 - s_e) / S * (d_e - sum_C p d)
// and only the softmax over all experts reaches outside C.
#include <cfloat>
#include <climits>

#include "lm_common.cuh"

namespace moedc {

constexpr int kGateWarps = 4;

struct GateArgs {
    const void* logits;
    int64_t ld;
    int T, E, K;
    const float* bias;
    bool sigmoid, normalize;
    float scale;
};

// +inf counts as the largest finite value, so that exp(l - max) stays a number
// (a NaN stays one)
__device__ __forceinline__ float gate_logit(float l) { return l > FLT_MAX ? FLT_MAX : l; }

// Order-preserving map of the selection key to unsigned; 0 for an expert that
// cannot be chosen (logit or key NaN or -inf).  The +0 makes -0 tie with +0.
__device__ __forceinline__ unsigned gate_key(float l, float b)
{
    const float key = l + b + 0.0f;
    if (!(l > -INFINITY) || !(key > -INFINITY)) return 0u;
    const unsigned u = __float_as_uint(key);
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}

// s (1 - s) of s = sigmoid(l), without the cancellation of 1 - s
__device__ __forceinline__ float sigmoid_slope(float l)
{
    const float e = expf(-fabsf(l));
    return e / ((1.0f + e) * (1.0f + e));
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Lane i < K holds chosen expert i (e < 0: none): its p = w / scale, and the
// sum S of the sigmoids over the chosen.  `den` and `top` are the softmax's
// denominator and maximum over all experts, used when not renormalised.
struct GateWeights {
    float p, total;
};
__device__ __forceinline__ GateWeights gate_weights(const GateArgs& a, bool live, float l,
                                                    float top, float den)
{
    GateWeights g{0.0f, 0.0f};
    if (a.sigmoid) {
        const float s = live ? sigmoid(l) : 0.0f;
        g.p = s;
        if (a.normalize) {
            g.total = warp_sum(s);
            g.p = g.total > 0.0f ? s / g.total : 0.0f;
        }
    } else if (a.normalize) {
        const float m = warp_max(live ? l : -FLT_MAX);
        const float ex = live ? expf(l - m) : 0.0f;
        const float sum = warp_sum(ex);
        g.p = live ? ex / sum : 0.0f;
    } else {
        g.p = live ? expf(l - top) / den : 0.0f;
    }
    return g;
}

// N experts per lane: expert e = lane + 32 j
template <typename T, int N>
__global__ void __launch_bounds__(kGateWarps * kWarp)
gate_kernel(GateArgs a, int32_t* __restrict__ topk_idx, float* __restrict__ topk_weights)
{
    pdl_enter();
    const int lane = threadIdx.x % kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kGateWarps;
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + threadIdx.x / kWarp; t < a.T; t += nwarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float l[N];
        unsigned key[N];
        float top = -FLT_MAX, den = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + kWarp * j;
            l[j] = e < a.E ? gate_logit(to_f32(row[e])) : -INFINITY;
            key[j] = gate_key(l[j], a.bias && e < a.E ? __ldg(a.bias + e) : 0.0f);
        }
        if (!a.sigmoid && !a.normalize) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (key[j]) top = fmaxf(top, l[j]);
            top = warp_max(top);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (key[j]) den += expf(l[j] - top);
            den = warp_sum(den);
        }
        int mine = -1;   // lane i: the i-th chosen expert
        for (int i = 0; i < a.K; ++i) {
            unsigned best = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) best = max(best, key[j]);
            const unsigned m = __reduce_max_sync(0xffffffffu, best);
            if (m == 0) break;
            int e = INT_MAX;
#pragma unroll
            for (int j = N - 1; j >= 0; --j)
                if (key[j] == m) e = lane + kWarp * j;
            const int win = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (lane + kWarp * j == win) key[j] = 0;
            if (lane == i) mine = win;
        }
        const float lc = mine >= 0 ? gate_logit(to_f32(row[mine])) : 0.0f;
        const GateWeights g = gate_weights(a, mine >= 0, lc, top, den);
        if (lane < a.K) {
            topk_idx[t * a.K + lane] = mine;
            topk_weights[t * a.K + lane] = g.p * a.scale;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kGateWarps * kWarp)
gate_grad_kernel(GateArgs a, const int32_t* __restrict__ topk_idx,
                 const float* __restrict__ dweights, T* __restrict__ dlogits)
{
    extern __shared__ float s_rows[];   // [kGateWarps][E]
    pdl_enter();
    const int lane = threadIdx.x % kWarp;
    float* acc = s_rows + (threadIdx.x / kWarp) * a.E;
    const int64_t nwarps = (int64_t)gridDim.x * kGateWarps;
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + threadIdx.x / kWarp; t < a.T; t += nwarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        int e = -1;
        float d = 0.0f, l = 0.0f;
        if (lane < a.K) {
            e = topk_idx[t * a.K + lane];
            if (e >= a.E || e < 0) e = -1;
            if (e >= 0) {
                l = gate_logit(to_f32(row[e]));
                if (!gate_key(l, a.bias ? a.bias[e] : 0.0f)) e = -1;
            }
            if (e >= 0) d = dweights[t * a.K + lane];
        }
        float top = -FLT_MAX, den = 0.0f;
        const bool dense = !a.sigmoid && !a.normalize;
        if (dense) {
            for (int c = lane; c < a.E; c += kWarp) {
                const float v = gate_logit(to_f32(row[c]));
                if (gate_key(v, a.bias ? a.bias[c] : 0.0f)) top = fmaxf(top, v);
            }
            top = warp_max(top);
            for (int c = lane; c < a.E; c += kWarp) {
                const float v = gate_logit(to_f32(row[c]));
                if (gate_key(v, a.bias ? a.bias[c] : 0.0f)) den += expf(v - top);
            }
            den = warp_sum(den);
        }
        const GateWeights g = gate_weights(a, e >= 0, l, top, den);
        const float dot = (a.sigmoid && !a.normalize) ? 0.0f : warp_sum(g.p * d);
        float own;
        if (a.sigmoid)
            own = a.normalize ? (g.total > 0.0f ? sigmoid_slope(l) / g.total * (d - dot) : 0.0f)
                              : sigmoid_slope(l) * d;
        else
            own = dense ? g.p * d : g.p * (d - dot);
        __syncwarp();
        for (int c = lane; c < a.E; c += kWarp) {
            float v = 0.0f;
            if (dense) {
                const float lg = gate_logit(to_f32(row[c]));
                if (gate_key(lg, a.bias ? a.bias[c] : 0.0f)) v = -expf(lg - top) / den * dot;
            }
            acc[c] = v;
        }
        __syncwarp();
        if (e >= 0) atomicAdd(acc + e, own);   // distinct experts: one addition each
        __syncwarp();
        for (int c = lane; c < a.E; c += kWarp)
            dlogits[t * a.E + c] = from_f32<T>(acc[c] * a.scale);
    }
}

}  // namespace moedc

namespace moedc_host {
namespace {

constexpr int kGateFlags = MOEDC_GATE_SIGMOID | MOEDC_GATE_NORMALIZE;

bool gate_args_ok(const void* logits, int64_t ld, int dtype, int T, int E, int K,
                  const float* bias, int flags)
{
    return T >= 0 && E >= 1 && E <= MOEDC_MAX_E && K >= 1 && K <= MOEDC_MAX_K && K <= E &&
           lm_dtype_ok(dtype) && (flags & ~kGateFlags) == 0 && ld >= E && ld <= INT32_MAX &&
           aligned(logits, lm_dtype_size(dtype)) && aligned(bias, 4) && (T == 0 || logits);
}

int gate_blocks(const void* kernel, size_t smem, int T)
{
    const int64_t want = ((int64_t)T + moedc::kGateWarps - 1) / moedc::kGateWarps;
    const int64_t most = resident_blocks(kernel, moedc::kGateWarps * moedc::kWarp, smem);
    return (int)(want < most ? want : most);
}

template <typename T, int N>
int launch_gate(const moedc::GateArgs& a, int32_t* idx, float* w, cudaStream_t stream)
{
    auto* k = moedc::gate_kernel<T, N>;
    const int blocks = gate_blocks((const void*)k, 0, a.T);
    clear_stale_error();
    launch(k, blocks, moedc::kGateWarps * moedc::kWarp, 0, stream, a, idx, w);
    return launch_status();
}

template <typename T>
int launch_gate_n(const moedc::GateArgs& a, int32_t* idx, float* w, cudaStream_t stream)
{
    if (a.E <= 64) return launch_gate<T, 2>(a, idx, w, stream);
    if (a.E <= 128) return launch_gate<T, 4>(a, idx, w, stream);
    if (a.E <= 256) return launch_gate<T, 8>(a, idx, w, stream);
    if (a.E <= 512) return launch_gate<T, 16>(a, idx, w, stream);
    return launch_gate<T, 32>(a, idx, w, stream);
}

template <typename T>
int launch_gate_grad(const moedc::GateArgs& a, const int32_t* idx, const float* dw, void* dl,
                     cudaStream_t stream)
{
    auto* k = moedc::gate_grad_kernel<T>;
    const size_t smem = (size_t)moedc::kGateWarps * a.E * sizeof(float);
    const int blocks = gate_blocks((const void*)k, smem, a.T);
    clear_stale_error();
    launch(k, blocks, moedc::kGateWarps * moedc::kWarp, smem, stream, a, idx, dw,
           static_cast<T*>(dl));
    return launch_status();
}

}  // namespace
}  // namespace moedc_host

extern "C" int moedc_gate(const void* logits, int64_t ld_logits, int dtype, int T, int E, int K,
                          const float* bias, int flags, float scale, int32_t* topk_idx,
                          float* topk_weights, cudaStream_t stream)
{
    using namespace moedc_host;
    if (!gate_args_ok(logits, ld_logits, dtype, T, E, K, bias, flags)) return MOEDC_ERR_ARG;
    if (!aligned(topk_idx, 4) || !aligned(topk_weights, 4)) return MOEDC_ERR_ARG;
    if (T == 0) return MOEDC_OK;
    if (!topk_idx || !topk_weights) return MOEDC_ERR_ARG;
    const moedc::GateArgs a{logits, ld_logits, T, E, K, bias, (flags & MOEDC_GATE_SIGMOID) != 0,
                            (flags & MOEDC_GATE_NORMALIZE) != 0, scale};
    return dtype == MOEDC_F32   ? launch_gate_n<float>(a, topk_idx, topk_weights, stream)
           : dtype == MOEDC_F16 ? launch_gate_n<__half>(a, topk_idx, topk_weights, stream)
                                : launch_gate_n<__nv_bfloat16>(a, topk_idx, topk_weights, stream);
}

extern "C" int moedc_gate_grad(const void* logits, int64_t ld_logits, int dtype, int T, int E,
                               int K, const float* bias, int flags, float scale,
                               const int32_t* topk_idx, const float* dweights, void* dlogits,
                               cudaStream_t stream)
{
    using namespace moedc_host;
    if (!gate_args_ok(logits, ld_logits, dtype, T, E, K, bias, flags)) return MOEDC_ERR_ARG;
    if (!aligned(topk_idx, 4) || !aligned(dweights, 4) || !aligned(dlogits, lm_dtype_size(dtype)))
        return MOEDC_ERR_ARG;
    if (T == 0) return MOEDC_OK;
    if (!topk_idx || !dweights || !dlogits) return MOEDC_ERR_ARG;
    const moedc::GateArgs a{logits, ld_logits, T, E, K, bias, (flags & MOEDC_GATE_SIGMOID) != 0,
                            (flags & MOEDC_GATE_NORMALIZE) != 0, scale};
    return dtype == MOEDC_F32   ? launch_gate_grad<float>(a, topk_idx, dweights, dlogits, stream)
           : dtype == MOEDC_F16 ? launch_gate_grad<__half>(a, topk_idx, dweights, dlogits, stream)
                                : launch_gate_grad<__nv_bfloat16>(a, topk_idx, dweights, dlogits,
                                                                  stream);
}
