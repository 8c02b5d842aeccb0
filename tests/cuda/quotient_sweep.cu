// Quotients by one divisor against the division: every pair of a divisor's 2^23 mantissas
// with a bf16 dividend's 2^7, an f16 dividend's 2^10, and as many binary32 ones drawn by a
// hash; results, and codes under scales of dispatch's range.
#include <cstdio>

#include "quotient.cuh"

using namespace moedc;

__device__ unsigned hash(unsigned v)
{
    v = (v ^ 61u) ^ (v >> 16);
    v *= 9u;
    v ^= v >> 4;
    v *= 0x27d4eb2du;
    return v ^ (v >> 15);
}

template <int kSteps> __global__ void sweep(int kind, int count, unsigned long long* off)
{
    const unsigned m = blockIdx.x * blockDim.x + threadIdx.x;   // divisor's mantissa
    unsigned long long bad = 0;
    for (int i = 0; i < count; ++i) {
        const unsigned a = kind == 0 ? (unsigned)i << 16 : kind == 1 ? (unsigned)i << 13 : hash(m * 1024u + i) & 0x7fffffu;
        const float x = __uint_as_float(0x3f800000u | a), b = __uint_as_float(0x3f800000u | m);
        const float2 q = Quotient<kSteps>::by(b).of(make_float2(x, -x));
        bad += q.x != __fdiv_rn(x, b) || q.y != __fdiv_rn(-x, b);
        // other exponents: a scale of 2^-22 .. 2^40, a dividend up to 448 times as large
        const float s = ldexpf(b, (int)(hash(m + 77u * i) % 63u) - 22), d = ldexpf(x, ilogbf(s) + (int)(hash(m ^ (i * 7919u)) % 160u) - 151);
        const uint32_t want = pack_e4m3x2(__fdiv_rn(d, s), __fdiv_rn(-d, s));
        bad += Quotient<kSteps>::by(s).codes(d, -d) != want;
    }
    // zeros, numbers that underflow, infinities and NaN, under this divisor and an infinite one
    const float odd[8] = {0.0f, 1e-45f, 1e-38f, 3e-30f, 1e-12f, 3e38f, __int_as_float(0x7f800000), __int_as_float(0x7fc00000)};
    const float under[3] = {__uint_as_float(0x34800000u | m), __uint_as_float(0x7b000000u | m), __int_as_float(0x7f800000)};
    for (int i = 0; i < 24; ++i) {
        const float d = odd[i % 8], s = under[i / 8];
        if (fabsf(d) > 448.0f * s && !isinf(d)) continue;      // a scale is its group's largest by 448
        if (isinf(d) && !isinf(s)) continue;
        bad += Quotient<kSteps>::by(s).codes(d, -d) != pack_e4m3x2(__fdiv_rn(d, s), __fdiv_rn(-d, s));
    }
    if (bad) atomicAdd(off, bad);
}

int main()
{
    unsigned long long *off, n = 0;
    if (cudaMalloc(&off, sizeof n) != cudaSuccess || cudaMemset(off, 0, sizeof n) != cudaSuccess) return 2;
    const int counts[3] = {128, 1024, 1024};
    sweep<1><<<(1 << 23) / 256, 256>>>(0, counts[0], off);
    sweep<1><<<(1 << 23) / 256, 256>>>(1, counts[1], off);
    sweep<2><<<(1 << 23) / 256, 256>>>(2, counts[2], off);
    if (cudaMemcpy(&n, off, sizeof n, cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
    printf("%llu differ\n", n);
    return n != 0;
}
