// Top-k router and its gradient: one warp per token.
//
// With l the token's logits, key = l + bias (or, asked for, the score, softmax or
// sigmoid of l, + bias) and the chosen set C the K largest keys, the weights are softmax(l) or sigmoid(l), over all experts or
// renormalised over C, times scale.  The gradient follows from w alone:
// with p = w / scale and d the weights' gradient on C,
//   softmax            dl_e = scale * p_e * (d_e - sum_C p d), d_e = 0 outside C
//   sigmoid            dl_e = scale * d_e * s_e (1 - s_e)
//   sigmoid over C     dl_e = scale * p_e (1 - s_e) * (d_e - sum_C p d)
// and only the softmax over all experts reaches outside C.
//
// Few tokens cost a launch.  Many are bound by instruction issue (ALU 57%): 32768
// tokens of 256 binary32 experts, top 8, take 22 us, their gradient 16 us, where the
// bytes alone (34 and 71 MB) would take 5 and 11.
#include <cfloat>
#include <climits>

#include "lm_common.cuh"

namespace moedc {

constexpr int kGateWarps = 4;

// What the choice is by
enum class By { logit, logit_bias, score_bias };

struct GateArgs {
    const void* logits;
    int64_t ld;
    int T, E, K;
    const float* bias;
    bool sigmoid, normalize;
    float scale;
};

// +inf counts as the largest finite value in the weights, so that exp(l - max) stays a number
// (a NaN stays one)
__device__ __forceinline__ float gate_logit(float l) { return l > FLT_MAX ? FLT_MAX : l; }

// Order-preserving map to unsigned; 0 for what cannot be chosen (NaN or -inf).
// The +0 makes -0 tie with +0.
__device__ __forceinline__ unsigned gate_order(float key)
{
    const unsigned u = __float_as_uint(key + 0.0f);
    const unsigned m = u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
    return key > -INFINITY ? m : 0u;
}
__device__ __forceinline__ float gate_unorder(unsigned m)
{
    return __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m);
}

// The selection key of a logit and its bias (0 without one).  For a bias on the score,
// which is not known yet, the logit's: 0 where the expert cannot be chosen.
template <By BY> __device__ __forceinline__ unsigned gate_key(float l, float b)
{
    if (BY == By::logit) return gate_order(l);
    if (BY == By::score_bias) return b > -INFINITY ? gate_order(l) : 0u;
    const unsigned m = gate_order(l + b);
    return l > -INFINITY ? m : 0u;
}

// s (1 - s) of s = sigmoid(l), without the cancellation of 1 - s
__device__ __forceinline__ float sigmoid_slope(float l)
{
    const float e = expf(-fabsf(l));
    return e / ((1.0f + e) * (1.0f + e));
}

// Far below 0, where expf(-l) would overflow, the sigmoid is expf(l) (1 + expf(l) is 1).
__device__ __forceinline__ float sigmoid(float l)
{
    return l < -80.0f ? expf(l) : 1.0f / (1.0f + expf(-l));
}

// exp for the dense sums, x <= 0: 2^(x log2 e), the power by ex2.approx (results
// below 2^-126 become 0).  Its relative error of |x| 2^-24 and some ulp is that of
// x itself as a difference of two logits; expf takes four times the instructions.
__device__ __forceinline__ float exp_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Lane i < K holds chosen expert i (live: there is one): its p = w / scale.  `den`
// and `top` are the softmax's denominator and maximum over all experts, used when
// not renormalised.
__device__ __forceinline__ float gate_weight(const GateArgs& a, bool live, float l, float top, float den)
{
    if (a.sigmoid) {
        float s = live ? sigmoid(l) : 0.0f;
        if (!a.normalize) return s;
        float total = warp_sum(s);
        if (total < 1e-30f) {
            // all far below 0, where a sigmoid is exp(l) and loses bits as it underflows: in
            // units of the largest.  One that is 0 in binary32 stays 0.
            const float m = warp_max(s > 0.0f ? l : -FLT_MAX);
            s = s > 0.0f ? expf(l - m) : 0.0f;
            total = warp_sum(s);
        }
        return total > 0.0f ? s / total : 0.0f;
    }
    if (a.normalize) {
        const float m = warp_max(live ? l : -FLT_MAX);
        const float ex = live ? expf(l - m) : 0.0f;
        const float sum = warp_sum(ex);
        return live ? ex / sum : 0.0f;
    }
    return live ? exp_fast(l - top) / den : 0.0f;
}

// A lane's experts: N of them, V neighbours to an access.  Value j holds expert
//   (lane + 32 (j / V)) V + j % V.
template <int V> __device__ __forceinline__ int gate_expert(int lane, int j)
{
    return (lane + kWarp * (j / V)) * V + j % V;
}

// The row's logits (-inf past E) and bias sums' keys.
template <typename T, int N, int V, By BY>
__device__ __forceinline__ void gate_load(const GateArgs& a, const T* row, int lane, float (&l)[N],
                                          unsigned (&key)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += V) {
        const int e = gate_expert<V>(lane, j);
        Pack<T, V> v;
        Pack<float, V> b;
        const bool in = e < a.E, biased = BY != By::logit && in;
        if (in) v = *reinterpret_cast<const Pack<T, V>*>(row + e);
        if (biased) {
#pragma unroll
            for (int c = 0; c < V; ++c) b.v[c] = __ldg(a.bias + e + c);
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const float raw = in ? to_f32(v.v[c]) : -INFINITY;
            key[j + c] = gate_key<BY>(raw, biased ? b.v[c] : 0.0f);
            l[j + c] = fminf(raw, FLT_MAX);       // a NaN has key 0
        }
    }
}

// Softmax over the experts that can be chosen: the maximum, each one's
// exponential in l's place, and their sum.
template <int N, By BY>
__device__ __forceinline__ void gate_softmax(float (&l)[N], const unsigned (&key)[N], float& top,
                                             float& den)
{
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, BY == By::logit_bias ? (key[j] ? gate_order(l[j]) : 0u) : key[j]);
    m = __reduce_max_sync(0xffffffffu, m);
    top = m ? fminf(gate_unorder(m), FLT_MAX) : 0.0f;
    den = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float e = exp_fast(l[j] - top);
        l[j] = key[j] ? e : 0.0f;
        den += l[j];
    }
    den = warp_sum(den);
}

// The keys of a bias on the score: sigmoid(l), or l (the softmax's exponentials by now)
// / den, plus the bias.  32768 tokens of 256 binary32 experts, top 8: softmax 28 us,
// sigmoid 32 us (by the logits 22 and 20).
template <int N, int V>
__device__ __forceinline__ void gate_score_keys(const GateArgs& a, int lane, const float (&l)[N],
                                                unsigned (&key)[N], float den)
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (key[j] == 0) continue;
        const float score = a.sigmoid ? sigmoid(l[j]) : l[j] / den;
        key[j] = gate_order(score + __ldg(a.bias + gate_expert<V>(lane, j)));
    }
}

// The K largest keys of the warp in (key descending, expert ascending) order,
// lane i getting the i-th's expert, -1 where there is none.
//
// The K-th largest of the 32 lanes' own maxima bounds the K-th largest key from
// below, so only the keys at or above it (some ten of 256) are candidates; they
// are packed into a slot each and ranked against one another.  Where more than
// 32 keys tie at the bound, the K maxima are taken one after another instead.
template <int N, int V>
__device__ __forceinline__ int gate_choose(unsigned (&key)[N], int K, int lane, unsigned long long* s_cand)
{
    unsigned mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) mine = max(mine, key[j]);
    unsigned bound = 0;
    for (int i = 0; i < K; ++i) {
        bound = __reduce_max_sync(0xffffffffu, mine);
        if (mine == bound) mine = 0;
    }
    bound = max(bound, 1u);            // 0 cannot be chosen
    int count = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const bool in = key[j] >= bound;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        const int at = count + __popc(who & lanemask_lt());
        if (in && at < kWarp)
            s_cand[at] = (unsigned long long)key[j] << 32 | (unsigned)~gate_expert<V>(lane, j);
        count += __popc(who);
    }
    int chosen = -1;
    if (count <= kWarp) {
        if (lane == 0 && count < kWarp) s_cand[count] = 0;     // an odd count's other half
        __syncwarp();
        const unsigned long long c = lane < count ? s_cand[lane] : 0;
        int rank = 0;
        for (int i = 0; i < count; i += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s_cand + i);
            rank += (o.x > c) + (o.y > c);
        }
        __syncwarp();
        // the candidate of rank i to lane i
        if (lane < count) s_cand[rank] = c;
        __syncwarp();
        if (lane < min(count, K)) chosen = (int)~(unsigned)s_cand[lane];
        __syncwarp();
        return chosen;
    }
    for (int i = 0; i < K; ++i) {
        unsigned best = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) best = max(best, key[j]);
        const unsigned m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0) break;
        int e = INT_MAX;
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
            if (key[j] == m) e = gate_expert<V>(lane, j);
        const int win = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (gate_expert<V>(lane, j) == win) key[j] = 0;
        if (lane == i) chosen = win;
    }
    return chosen;
}

template <typename T, int N, int V, By BY>
__global__ void __launch_bounds__(kGateWarps * kWarp)
gate_kernel(GateArgs a, int32_t* __restrict__ topk_idx, float* __restrict__ topk_weights)
{
    __shared__ __align__(16) unsigned long long s_cand[kGateWarps][kWarp];
    pdl_enter();
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * kGateWarps;
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < a.T; t += nwarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float l[N];
        unsigned key[N];
        gate_load<T, N, V, BY>(a, row, lane, l, key);
        float top = 0.0f, den = 1.0f;
        constexpr bool kScore = BY == By::score_bias;
        if (!a.sigmoid && (!a.normalize || kScore)) gate_softmax<N, BY>(l, key, top, den);
        if (kScore) gate_score_keys<N, V>(a, lane, l, key, den);
        const int mine = gate_choose<N, V>(key, a.K, lane, s_cand[warp]);
        const float lc = mine >= 0 ? gate_logit(to_f32(row[mine])) : 0.0f;
        const float p = gate_weight(a, mine >= 0, lc, top, den);
        if (lane < a.K) {
            topk_idx[t * a.K + lane] = mine;
            topk_weights[t * a.K + lane] = p * a.scale;
        }
    }
}

// DENSE: the softmax over all experts, whose gradient reaches every one.
template <typename T, int N, int V, By BY, bool DENSE>
__global__ void __launch_bounds__(kGateWarps * kWarp)
gate_grad_kernel(GateArgs a, const int32_t* __restrict__ topk_idx,
                 const float* __restrict__ dweights, T* __restrict__ dlogits)
{
    // what the chosen experts get; zero for all others, from row to row
    __shared__ __align__(16) float s_own[kGateWarps][N * kWarp];
    const int lane = threadIdx.x % kWarp;
    float* add = s_own[threadIdx.x / kWarp];
    for (int c = lane; c < N * kWarp; c += kWarp) add[c] = 0.0f;
    __syncwarp();
    pdl_enter();
    const int64_t nwarps = (int64_t)gridDim.x * kGateWarps;
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + threadIdx.x / kWarp; t < a.T; t += nwarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float v[N];
        unsigned key[N];
        float top = 0.0f, den = 1.0f;
        int e = lane < a.K ? topk_idx[t * a.K + lane] : -1;
        float d = lane < a.K ? dweights[t * a.K + lane] : 0.0f;
        if (DENSE) gate_load<T, N, V, BY>(a, row, lane, v, key);
        float l = 0.0f;
        if (e >= 0 && e < a.E) {
            l = gate_logit(to_f32(row[e]));
            if (!gate_key<BY>(l, BY != By::logit ? __ldg(a.bias + e) : 0.0f)) e = -1;
        } else {
            e = -1;
        }
        if (e < 0) d = 0.0f;
        if (DENSE) gate_softmax<N, BY>(v, key, top, den);   // v: the exponentials
        const float p = gate_weight(a, e >= 0, l, top, den);
        const float dot = (a.sigmoid && !a.normalize) ? 0.0f : warp_sum(p * d);
        float own;
        if (a.sigmoid)
            own = a.normalize ? p * sigmoid(-l) * (d - dot) : sigmoid_slope(l) * d;
        else
            own = DENSE ? p * d : p * (d - dot);
        if (e >= 0) atomicAdd(add + e, own * a.scale);   // distinct experts: one addition each
        __syncwarp();
        // a token that chose nothing has den = 0 and no gradient
        const float all = DENSE && den > 0.0f ? -dot * a.scale / den : 0.0f;
#pragma unroll
        for (int j = 0; j < N; j += V) {
            const int c0 = gate_expert<V>(lane, j);
            if (c0 >= a.E) break;
            const Pack<float, V> own_v = *reinterpret_cast<const Pack<float, V>*>(add + c0);
            Pack<T, V> o;
#pragma unroll
            for (int c = 0; c < V; ++c)
                o.v[c] = from_f32<T>(DENSE ? fmaf(v[j + c], all, own_v.v[c]) : own_v.v[c]);
            *reinterpret_cast<Pack<T, V>*>(dlogits + t * a.E + c0) = o;
        }
        __syncwarp();
        if (e >= 0) add[e] = 0.0f;
        __syncwarp();
    }
}

}  // namespace moedc

namespace moedc_host {
namespace {

constexpr int kGateFlags = MOEDC_GATE_SIGMOID | MOEDC_GATE_NORMALIZE | MOEDC_GATE_BIAS_SCORE;

bool gate_args_ok(const void* logits, int64_t ld, int dtype, int T, int E, int K,
                  const float* bias, int flags)
{
    return T >= 0 && E >= 1 && E <= MOEDC_MAX_E && K >= 1 && K <= MOEDC_MAX_K && K <= E &&
           lm_dtype_ok(dtype) && (flags & ~kGateFlags) == 0 && ld >= E && ld <= INT32_MAX &&
           aligned(logits, lm_dtype_size(dtype)) && aligned(bias, 4) && (T == 0 || logits);
}

// without a bias every rule is the logits' order
moedc::By gate_by(const float* bias, int flags)
{
    if (!bias) return moedc::By::logit;
    return flags & MOEDC_GATE_BIAS_SCORE ? moedc::By::score_bias : moedc::By::logit_bias;
}

template <typename... KArgs, typename... Args>
int launch_gate(void (*kernel)(KArgs...), int T, cudaStream_t stream, Args... args)
{
    const int64_t want = ((int64_t)T + moedc::kGateWarps - 1) / moedc::kGateWarps;
    const int64_t most = resident_blocks((const void*)kernel, moedc::kGateWarps * moedc::kWarp, 0);
    clear_stale_error();
    launch(kernel, (int)(want < most ? want : most), moedc::kGateWarps * moedc::kWarp, 0, stream, args...);
    return launch_status();
}

// Four neighbouring experts to an access where rows keep them aligned, one elsewhere.
template <typename T> bool gate_wide(const moedc::GateArgs& a, const void* dlogits)
{
    return a.E % 4 == 0 && a.ld % 4 == 0 && aligned(a.logits, 4 * sizeof(T)) &&
           aligned(dlogits, 4 * sizeof(T));
}

template <typename T, int N, moedc::By BY>
int run_gate_by(const moedc::GateArgs& a, int32_t* idx, float* w, cudaStream_t stream)
{
    return gate_wide<T>(a, nullptr) ? launch_gate(moedc::gate_kernel<T, N, 4, BY>, a.T, stream, a, idx, w)
                                    : launch_gate(moedc::gate_kernel<T, N, 1, BY>, a.T, stream, a, idx, w);
}

template <typename T, int N>
int run_gate(const moedc::GateArgs& a, moedc::By by, int32_t* idx, float* w, cudaStream_t stream)
{
    return by == moedc::By::logit        ? run_gate_by<T, N, moedc::By::logit>(a, idx, w, stream)
           : by == moedc::By::logit_bias ? run_gate_by<T, N, moedc::By::logit_bias>(a, idx, w, stream)
                                         : run_gate_by<T, N, moedc::By::score_bias>(a, idx, w, stream);
}

template <typename T, int N, int V, moedc::By BY>
int run_gate_grad_by(const moedc::GateArgs& a, const int32_t* idx, const float* dw, void* dl, cudaStream_t stream)
{
    T* out = static_cast<T*>(dl);
    return !a.sigmoid && !a.normalize
               ? launch_gate(moedc::gate_grad_kernel<T, N, V, BY, true>, a.T, stream, a, idx, dw, out)
               : launch_gate(moedc::gate_grad_kernel<T, N, V, BY, false>, a.T, stream, a, idx, dw, out);
}

template <typename T, int N, int V>
int run_gate_grad(const moedc::GateArgs& a, moedc::By by, const int32_t* idx, const float* dw, void* dl,
                  cudaStream_t stream)
{
    return by == moedc::By::logit        ? run_gate_grad_by<T, N, V, moedc::By::logit>(a, idx, dw, dl, stream)
           : by == moedc::By::logit_bias ? run_gate_grad_by<T, N, V, moedc::By::logit_bias>(a, idx, dw, dl, stream)
                                         : run_gate_grad_by<T, N, V, moedc::By::score_bias>(a, idx, dw, dl, stream);
}

// Experts of a lane: as many as E needs, in steps that keep the registers few.
#define MOEDC_GATE_N(E, CALL)        \
    (E <= 128   ? CALL(4)            \
     : E <= 256 ? CALL(8)            \
     : E <= 384 ? CALL(12)           \
     : E <= 512 ? CALL(16)           \
                : CALL(32))

template <typename T>
int gate_by_size(const moedc::GateArgs& a, moedc::By by, int32_t* idx, float* w, cudaStream_t stream)
{
#define MOEDC_CALL(N) run_gate<T, N>(a, by, idx, w, stream)
    return MOEDC_GATE_N(a.E, MOEDC_CALL);
#undef MOEDC_CALL
}

template <typename T>
int gate_grad_by_size(const moedc::GateArgs& a, moedc::By by, const int32_t* idx, const float* dw, void* dl,
                      cudaStream_t stream)
{
    const bool wide = gate_wide<T>(a, dl);
#define MOEDC_CALL(N) \
    (wide ? run_gate_grad<T, N, 4>(a, by, idx, dw, dl, stream) : run_gate_grad<T, N, 1>(a, by, idx, dw, dl, stream))
    return MOEDC_GATE_N(a.E, MOEDC_CALL);
#undef MOEDC_CALL
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
    const moedc::By by = gate_by(bias, flags);
    return dtype == MOEDC_F32   ? gate_by_size<float>(a, by, topk_idx, topk_weights, stream)
           : dtype == MOEDC_F16 ? gate_by_size<__half>(a, by, topk_idx, topk_weights, stream)
                                : gate_by_size<__nv_bfloat16>(a, by, topk_idx, topk_weights, stream);
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
    const moedc::By by = gate_by(bias, flags);
    return dtype == MOEDC_F32   ? gate_grad_by_size<float>(a, by, topk_idx, dweights, dlogits, stream)
           : dtype == MOEDC_F16 ? gate_grad_by_size<__half>(a, by, topk_idx, dweights, dlogits, stream)
                                : gate_grad_by_size<__nv_bfloat16>(a, by, topk_idx, dweights,
                                                                  dlogits, stream);
}
