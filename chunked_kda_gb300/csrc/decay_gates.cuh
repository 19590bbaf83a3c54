// Sums of per-token decays in log2 units as integers of 2^-32: each decay is off by at most 2^-33 (32768 equal
// ones together by 2.6e-6 of what they decay), their sums and the differences of far sums by nothing more.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "sm100.cuh"

namespace kda {
namespace decay {

// A log2 decay in 2^-32 units, from the natural logarithm.  Clamped: 2^-1024 is zero for a float32, so
// -inf clears what it meets.
__device__ __forceinline__ long long fixed(float a) {
    constexpr float kRest = 1.9259629911267e-8f;  // log2(e) - kLog2e
    const float x = fminf(fmaxf(a * kLog2e, -1024.f), 1024.f);
    const float e = fabsf(x) < 1024.f ? fmaf(a, kLog2e, -x) + a * kRest : 0.f;
    return __float2ll_rn(x * 4294967296.f) + __float2int_rn(e * 4294967296.f);
}
// rounded to an integer and a fraction in [0, 1) in 2^-24 units, as the powers below take them
__device__ __forceinline__ void parts(long long g, int& i, int& f) {
    const long long r = (g + 128) >> 8;
    i = (int)(r >> 24);
    f = (int)r & 0xFFFFFF;
}
__device__ __forceinline__ float pow2i(int n) { return __int_as_float(min(max(n + 127, 0), 255) << 23); }
// 2^(n + f / 2^24), |f| < 2^24: the power of the nearest integer times the power series of the rest
// (|z| <= ln(2) / 2: the first left out term is below 2^-26)
__device__ __forceinline__ float pow2(int n, int f) {
    const int r = (f + (1 << 23)) >> 24;
    const float z = (float)(f - (r << 24)) * (0.69314718f / 16777216.f);
    float y = fmaf(1.f / 5040.f, z, 1.f / 720.f);
    y = fmaf(y, z, 1.f / 120.f);
    y = fmaf(y, z, 1.f / 24.f);
    y = fmaf(y, z, 1.f / 6.f);
    y = fmaf(y, z, 0.5f);
    y = fmaf(y, z, 1.f);
    return fmaf(y, z, 1.f) * pow2i(n + r);
}
// the same by the hardware's approximation (2^-22)
__device__ __forceinline__ float pow2_fast(int n, int f) {
    return sm100::ex2_fast((float)f * (1.f / 16777216.f)) * pow2i(n);
}
// The first of a chunk's 64 tokens, two consecutive ones a lane, whose decay is no number (64: none):
// that token's output and all that follow are none either, those before it have nothing to do with it.
__device__ __forceinline__ int first_nan(float a0, float a1) {
    const unsigned even = __ballot_sync(0xffffffffu, a0 != a0), odd = __ballot_sync(0xffffffffu, a1 != a1);
    return min(even ? 2 * (__ffs(even) - 1) : 64, odd ? 2 * __ffs(odd) - 1 : 64);
}
__device__ __forceinline__ float nan_if(bool on) { return on ? __int_as_float(0x7fffffff) : 0.f; }
// Inclusive sums over a warp of two consecutive tokens a lane: G of the lane's two tokens.
__device__ __forceinline__ void pair_sums(float a0, float a1, long long (&G)[2]) {
    const long long g1 = fixed(a1);
    long long g = fixed(a0) + g1;
    const int l = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, g, m);
        if (l >= m) g += y;
    }
    G[0] = g - g1;
    G[1] = g;
}

}  // namespace decay
}  // namespace kda
