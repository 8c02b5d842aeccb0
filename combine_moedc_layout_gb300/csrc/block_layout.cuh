// The routing layout of a small batch (at most MOEDC_FUSED_MAX_ENTRIES entries)
// rebuilt in one block's shared memory: the single-launch forms of the dispatch
// and of the row sort.
#pragma once

#include "common.cuh"

namespace moedc {

// Block width follows the entry count: every thread holds two routing ids,
// so 128-thread blocks take up to 256 entries and 512-thread blocks the rest.
// Narrow blocks keep more SMs copying when there are few tokens; wide blocks
// shorten each warp's share of the layout when there are many (measured: at 4
// tokens 128 threads beat 512 by 3 us, at 1024 entries 512 beat 128 by 2 us).
constexpr int kFusedIdsPerThread = 2;
constexpr int kFusedNarrow = 128;
constexpr int kFusedWide = MOEDC_FUSED_MAX_ENTRIES / kFusedIdsPerThread;
static_assert(kFusedWide == 512, "wide fused block");

// Shared memory (int32 words) of one block of `threads` for n entries, E experts.
__host__ __device__ constexpr size_t fused_smem_words(int threads, int n, int E)
{
    return 2 * (size_t)n + (size_t)(threads / kWarp + 1) * E;
}

// The layout of all n entries, rebuilt in this block's shared memory: each
// warp owns a contiguous run of 32-entry tiles in (t, k) order; the run is
// counted per expert, the counts are scanned across warps, then equal
// experts are ranked inside each tile in lane order.  On return s_idx holds
// the routing ids, s_slot the slots (-1 for masked / out-of-range entries) and
// s_cnt the per-expert counts.
template <int kThreads>
__device__ __forceinline__ void block_layout(const int32_t* __restrict__ topk_idx, int n, int E,
                                             int32_t* s_idx, int32_t* s_slot, int32_t* s_wcnt,
                                             int32_t* s_cnt)
{
    constexpr int kFusedWarps = kThreads / kWarp;
    const int lane = threadIdx.x % kWarp;
    const int warp = threadIdx.x / kWarp;
    {
        int v[kFusedIdsPerThread];
#pragma unroll
        for (int j = 0; j < kFusedIdsPerThread; ++j) {
            const int i = threadIdx.x + j * kThreads;
            v[j] = i < n ? topk_idx[i] : 0;
        }
        for (int i = threadIdx.x; i < kFusedWarps * E; i += kThreads) s_wcnt[i] = 0;
#pragma unroll
        for (int j = 0; j < kFusedIdsPerThread; ++j) {
            const int i = threadIdx.x + j * kThreads;
            if (i < n) s_idx[i] = v[j];
        }
    }
    __syncthreads();
    const int run = ((n + kFusedWarps * kWarp - 1) / (kFusedWarps * kWarp)) * kWarp;
    const int wbeg = min(n, warp * run);
    const int wend = min(n, wbeg + run);
    int32_t* my = s_wcnt + warp * E;
    for (int i = wbeg + lane; i < wend; i += kWarp) {
        const int e = s_idx[i];
        if (e >= 0 && e < E) atomicAdd(&my[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int acc = 0;
#pragma unroll
        for (int w = 0; w < kFusedWarps; ++w) {
            const int c = s_wcnt[w * E + e];
            s_wcnt[w * E + e] = acc;
            acc += c;
        }
        s_cnt[e] = acc;
    }
    __syncthreads();
    const unsigned lt = lanemask_lt();
    for (int i0 = wbeg; i0 < wend; i0 += kWarp) {
        const int i = i0 + lane;
        const int e = i < wend ? s_idx[i] : -1;
        const bool v = e >= 0 && e < E;
        const unsigned peers = match_expert(e, v);
        int sv = -1;
        if (v) sv = my[e] + __popc(peers & lt);
        __syncwarp();
        if (v && (peers & lt) == 0) my[e] += __popc(peers);
        __syncwarp();
        if (i < wend) s_slot[i] = sv;
    }
    __syncthreads();
}

}  // namespace moedc
