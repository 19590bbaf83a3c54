// Sums of per-token decays in log2 units, exact whatever their size: an integer and a fraction in
// 2^-24 units, added as integers, so that differences of far sums lose nothing.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "sm100.cuh"

namespace kda {
namespace decay {

// A log2 decay as an integer (returned in ip) and a fraction in 2^-24 units, from the natural
// logarithm.  Clamped: 2^-1024 is zero for a float32, so -inf clears what it meets.
__device__ __forceinline__ int fixed(float a, int& ip) {
    constexpr float kRest = 1.9259629911267e-8f;  // log2(e) - kLog2e
    const float x = fminf(fmaxf(a * kLog2e, -1024.f), 1024.f), fl = floorf(x);
    const float e = fabsf(x) < 1024.f ? fmaf(a, kLog2e, -x) + a * kRest : 0.f;
    ip = (int)fl;
    return __float2int_rn(((x - fl) + e) * 16777216.f);
}
// the fraction into [0, 1)
__device__ __forceinline__ void carry(int& i, int& f) {
    i += f >> 24;
    f &= 0xFFFFFF;
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
// Inclusive sums over a warp of two consecutive tokens a lane: I, F of the lane's two tokens.
__device__ __forceinline__ void pair_sums(float a0, float a1, int (&I)[2], int (&F)[2]) {
    int i0, i1;
    const int f0 = fixed(a0, i0), f1 = fixed(a1, i1);
    int ii = i0 + i1, ff = f0 + f1;
    const int l = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int yi = __shfl_up_sync(0xffffffffu, ii, m), yf = __shfl_up_sync(0xffffffffu, ff, m);
        if (l >= m) {
            ii += yi;
            ff += yf;
        }
    }
    I[0] = ii - i1;
    F[0] = ff - f1;
    I[1] = ii;
    F[1] = ff;
    carry(I[0], F[0]);
    carry(I[1], F[1]);
}

}  // namespace decay
}  // namespace kda
