// The norm of query and key heads and the rotation of their positions, in one pass.
//
// Per row of D elements (a token's head):
//   y = x [/ sqrt(mean(x^2) + eps) * weight]   or   x / sqrt(sum(x^2) + eps) [* weight]
//   of the first R elements, each pair: (y_a, y_b) <- m (y_a cos - y_b sin, y_b cos + y_a sin),
//   angle = p f,   p = the token's position on the pair's axis, f = inv_freq of the pair.
//
// The angle is wanted modulo a turn only, and positions are integers: f / 2 pi is taken modulo 1 as a 64-bit
// fraction (from 53 bits), and p times it modulo 2^64 is exact.  So an angle is off by p 2^-53 turns however far
// the position; a float32 product is off by 0.06 radians at 10^6.
//
// A block has `tile` consecutive tokens with all their heads: the angles' cosines and sines are formed once a token,
// in shared memory.  A lane has four pairs: a row is split so that both halves of its pairs lie in one lane (two
// loads of four elements, R / 2 apart, or one of eight), and LPR lanes share a row.
#include "common.cuh"
#include "kda_internal.h"
#include "sm100.cuh"

namespace kda {
namespace {

constexpr int NT = 256, kMaxD = 256;

struct Axes {  // the axis of each pair, two bits a pair
    uint32_t bits[kMaxD / 2 / 16];
};

struct Params {
    const void* x[2];
    void* y[2];
    const float* w[2];
    long xs[2], ys[2];  // elements between tokens
    int Hq, heads;      // query heads, all heads
    uint32_t per;       // ceil(2^32 / heads), 0: one head
    int norm;
    float eps;
    const int32_t* pos;
    const float* freq;
    Axes axes;
    int R, D, interleaved;
    float m;
    long tokens;
    int tile;
};

// cosine and sine of pair i at token t, times m
__device__ __forceinline__ float2 turn(const Params& p, long t, int i) {
    const float f = __ldg(p.freq + i);
    const int axis = (p.axes.bits[i >> 4] >> (2 * (i & 15))) & 3;
    const long pos = __ldg(p.pos + axis * p.tokens + t);
    double x = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
    x -= floor(x);
    const unsigned long long a = (unsigned long long)pos * __double2ull_rz(x * 18446744073709551616.0);
    float s, c;
    sincospif((float)(int)(a >> 32) * (1.f / 2147483648.f), &s, &c);
    const float bad = fabsf(f) < __int_as_float(0x7f800000) ? 0.f : __int_as_float(0x7fffffff);
    return make_float2(c * p.m + bad, s * p.m + bad);
}

__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float* r) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = sm100::bf_lo(v.x); r[1] = sm100::bf_hi(v.x); r[2] = sm100::bf_lo(v.y); r[3] = sm100::bf_hi(v.y);
}
__device__ __forceinline__ void ld4(const float* p, float* r) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float* r) {
    *reinterpret_cast<uint2*>(p) = make_uint2(sm100::pack_bf16(r[0], r[1]), sm100::pack_bf16(r[2], r[3]));
}
__device__ __forceinline__ void st4(float* p, const float* r) { *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]); }

__device__ __forceinline__ float factor(const Params& p, float sum) {
    return p.norm == KDA_NORM_NONE ? 1.f : rsqrtf((p.norm == KDA_NORM_RMS ? sum / (float)p.D : sum) + p.eps);
}

// D and R multiples of 8, rows 16-byte aligned.  LPR: lanes a row, D / 8 rounded up to a power of 2.
template <typename T, int LPR>
__global__ void __launch_bounds__(NT) qk_norm_rope_kernel(Params p) {
    extern __shared__ float2 s_turn[];  // [tile][R / 2]
    const int tid = threadIdx.x, half = p.R / 2;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0);
    for (int x = tid; x < nt * half; x += NT) s_turn[x] = turn(p, t0 + x / half, x % half);
    if (half) __syncthreads();

    // the lane's pairs i .. i + 3: elements i and R / 2 + i behind the first half's start, or eight in a row
    const int l = tid % LPR, i = 4 * l;
    const bool on = 2 * i < p.D, rot = i < half;
    const int a = rot && !p.interleaved ? i : 2 * i, b = rot && !p.interleaved ? half + i : 2 * i + 4;
    float w[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[s][e] = on && p.w[s] ? __ldg(p.w[s] + (e < 4 ? a + e : b + e - 4)) : 1.f;

    constexpr int G = NT / LPR, U = 4;  // rows at a time; loads of U rows in flight
    const int rows = nt * p.heads;
    for (int r0 = tid / LPR; r0 < rows; r0 += G * U) {
        float v[U][8];
        int tt[U], hh[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * G;
            tt[u] = p.per ? (int)__umulhi((uint32_t)r, p.per) : r;
            hh[u] = r - tt[u] * p.heads;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
            if (r < rows && on) {
                const int side = hh[u] >= p.Hq;
                const T* src = static_cast<const T*>(p.x[side]) + (t0 + tt[u]) * p.xs[side] + (hh[u] - (side ? p.Hq : 0)) * p.D;
                ld4(src + a, v[u]);
                ld4(src + b, v[u] + 4);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * G;
            if (__all_sync(0xffffffffu, r >= rows)) break;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(v[u][e], v[u][e], sum);
#pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            if (r >= rows || !on) continue;
            const int side = hh[u] >= p.Hq;
            const float f = factor(p, sum);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = v[u][e] * f * (side ? w[1][e] : w[0][e]);
            if (rot) {
                const float2* cs = s_turn + tt[u] * half + i;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 z = cs[e];
                    float& ya = p.interleaved ? y[2 * e] : y[e];
                    float& yb = p.interleaved ? y[2 * e + 1] : y[4 + e];
                    const float xa = ya, xb = yb;
                    ya = xa * z.x - xb * z.y;
                    yb = xb * z.x + xa * z.y;
                }
            }
            T* dst = static_cast<T*>(p.y[side]) + (t0 + tt[u]) * p.ys[side] + (hh[u] - (side ? p.Hq : 0)) * p.D;
            st4(dst + a, y);
            st4(dst + b, y + 4);
        }
    }
}

// Any D, R and alignment: a warp a row, a pair of single elements a lane and step.
template <typename T>
__global__ void __launch_bounds__(NT) qk_norm_rope_any_kernel(Params p) {
    extern __shared__ float2 s_turn[];
    const int tid = threadIdx.x, half = p.R / 2, l = tid & 31;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0);
    for (int x = tid; x < nt * half; x += NT) s_turn[x] = turn(p, t0 + x / half, x % half);
    if (half) __syncthreads();
    constexpr int S = kMaxD / 64;
    for (int r = tid >> 5; r < nt * p.heads; r += NT / 32) {
        const int tt = r / p.heads, hh = r % p.heads, side = hh >= p.Hq, h = hh - (side ? p.Hq : 0);
        const T* src = static_cast<const T*>(p.x[side]) + (t0 + tt) * p.xs[side] + (long)h * p.D;
        T* dst = static_cast<T*>(p.y[side]) + (t0 + tt) * p.ys[side] + (long)h * p.D;
        float va[S], vb[S], sum = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = l + 32 * s;
            const bool apart = i < half && !p.interleaved;
            const int a = apart ? i : 2 * i, b = apart ? half + i : 2 * i + 1;
            va[s] = a < p.D ? to_f32(src[a]) : 0.f;
            vb[s] = b < p.D && a < p.D ? to_f32(src[b]) : 0.f;
            sum = fmaf(va[s], va[s], fmaf(vb[s], vb[s], sum));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float f = factor(p, sum);
        const float* w = side ? p.w[1] : p.w[0];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = l + 32 * s;
            const bool apart = i < half && !p.interleaved;
            const int a = apart ? i : 2 * i, b = apart ? half + i : 2 * i + 1;
            if (a >= p.D) continue;
            float ya = va[s] * f * (w ? __ldg(w + a) : 1.f), yb = b < p.D ? vb[s] * f * (w ? __ldg(w + b) : 1.f) : 0.f;
            if (i < half) {
                const float2 z = s_turn[tt * half + i];
                const float xa = ya, xb = yb;
                ya = xa * z.x - xb * z.y;
                yb = xb * z.x + xa * z.y;
            }
            dst[a] = from_f32<T>(ya);
            if (b < p.D) dst[b] = from_f32<T>(yb);
        }
    }
}

template <typename T>
cudaError_t run(const QkNormArgs& a, Params& p, bool fast) {
    const int grid = (int)((a.tokens + p.tile - 1) / p.tile), bytes = p.tile * (a.R / 2) * (int)sizeof(float2);
    void (*kern)(Params) = qk_norm_rope_any_kernel<T>;
    if (fast) kern = a.D > 128 ? qk_norm_rope_kernel<T, 32> : a.D > 64 ? qk_norm_rope_kernel<T, 16> : a.D > 32 ? qk_norm_rope_kernel<T, 8>
                     : qk_norm_rope_kernel<T, 4>;
    kern<<<grid, NT, bytes, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormArgs& a) {
    Params p{};
    const int Hk = a.k.x ? a.k.heads : 0;
    const QkNormArgs::Side* side[2] = {&a.q, &a.k};
    p.Hq = a.q.heads;
    p.heads = a.q.heads + Hk;
    const int e = a.bf16 ? 2 : 4;
    bool fast = a.D % 8 == 0 && a.R % 8 == 0;
    for (int s = 0; s < (Hk ? 2 : 1); ++s) {
        p.x[s] = side[s]->x;
        p.y[s] = side[s]->y;
        p.w[s] = side[s]->weight;
        p.xs[s] = side[s]->stride;
        p.ys[s] = side[s]->y_stride;
        fast = fast && (((uintptr_t)p.x[s] | (uintptr_t)p.y[s] | (uintptr_t)(p.xs[s] * e) | (uintptr_t)(p.ys[s] * e)) & 15u) == 0;
    }
    p.norm = a.norm;
    p.eps = a.eps;
    p.pos = a.positions;
    p.freq = a.inv_freq;
    for (int i = 0; i < a.R / 2 && a.pair_axes; ++i) p.axes.bits[i >> 4] |= (uint32_t)a.pair_axes[i] << (2 * (i & 15));
    p.R = a.R;
    p.D = a.D;
    p.interleaved = a.interleaved;
    p.m = a.rope_scale;
    p.tokens = a.tokens;
    // rows of a block: enough of them to share a token's angles, and blocks enough for the SMs
    p.tile = 1;
    while (p.tile < 16 && p.tile * p.heads < 64 && a.tokens / (2 * p.tile) >= 1024) p.tile *= 2;
    // r / heads for r < 2^16 rows of a block by a product (exact: r (per heads - 2^32) < 2^32)
    p.per = p.heads > 1 ? (uint32_t)(((1ull << 32) + p.heads - 1) / p.heads) : 0;
    return a.bf16 ? run<__nv_bfloat16>(a, p, fast) : run<float>(a, p, fast);
}

}  // namespace kda
