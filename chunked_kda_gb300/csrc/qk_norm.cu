// The norm of query and key heads and the rotation of their positions, in one pass.
//
// Per row of D elements (a token's head):
//   y = x [/ sqrt(mean(x^2) + eps) * weight]   or   x / sqrt(sum(x^2) + eps) [* weight]
//   of the first R elements, each pair: (y_a, y_b) <- m (y_a cos - y_b sin, y_b cos + y_a sin),
//   angle = p f,   p = the token's position on the pair's axis, f = inv_freq of the pair.
//
// The angle is wanted modulo a turn only, and positions are integers: f / 2 pi is taken modulo 1 as a 64-bit
// fraction (integer product of f's 24 bits and 2^64 / 2 pi), and p times it modulo 2^64 is exact.  So an angle is off by
// p f 2^-65 turns however far the position; a float32 product is off by 0.06 radians at 10^6.
//
// A block has `tile` consecutive tokens with all their heads: the angles' cosines and sines are formed once a token,
// in shared memory, while the first rows are on their way.  A lane has four pairs: a row is split so that both halves of
// its pairs lie in one lane (two loads of four elements, R / 2 apart, or one of eight), and LPR lanes share a row.  The
// next U rows of a lane are on their way while it works on U.
//
// Memory bounds it: each row goes in and out once.  16384 tokens with 64 + 8 heads of 128, RMS norm, rotation: 604 MB in
// 112 us, 5.4 TB/s (angles formed in FP32 for each row, no loads ahead: 260); 20480 tokens with 32 heads, L2 norm, no
// rotation: 60 us, 5.6 TB/s.  U: 1, 2, 3, 4 give 124, 111, 126 and 129 us of the first, 72, 60, 62 and 60 of the second.
// What is missing to a copy's 6.8 TB/s is a row's way from its load through the sum's shuffles to its store, and in the
// first the angles in front of a block's rows.
#include "common.cuh"
#include "kda_internal.h"
#include "sm100.cuh"
#include "tile_ops.cuh"

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
    // |f| = m 2^(e - 150): its turns in 2^-64 are m (2^64 / 2 pi) 2^(e - 150), modulo 2^64
    const uint32_t bits = __float_as_uint(f) & 0x7FFFFFFFu, e = bits >> 23;
    const unsigned long long m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits << 1, unit = 0x28BE60DB9391054Aull;
    const unsigned long long lo = m * unit, hi = __umul64hi(m, unit);
    const int s = 150 - (int)(e ? e : 0u);
    unsigned long long turns = s <= 0 ? (s > -64 ? lo << -s : 0ull) : s < 64 ? (lo >> s) | (hi << (64 - s)) : s < 128 ? hi >> (s - 64) : 0ull;
    if (f < 0.f) turns = 0ull - turns;
    const unsigned long long a = (unsigned long long)pos * turns;
    float si, co;
    sincospif((float)(int)(a >> 32) * (1.f / 2147483648.f), &si, &co);
    const float bad = fabsf(f) < __int_as_float(0x7f800000) ? 0.f : __int_as_float(0x7fffffff);
    return make_float2(co * p.m + bad, si * p.m + bad);
}

// four elements as they lie in memory, and as floats
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(Raw v, float2& a, float2& b) {
        a = make_float2(sm100::bf_lo(v.x), sm100::bf_hi(v.x));
        b = make_float2(sm100::bf_lo(v.y), sm100::bf_hi(v.y));
    }
    static __device__ __forceinline__ Raw pack(float2 a, float2 b) { return make_uint2(sm100::pack_bf16(a.x, a.y), sm100::pack_bf16(b.x, b.y)); }
};
template <>
struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ void unpack(Raw v, float2& a, float2& b) {
        a = make_float2(v.x, v.y);
        b = make_float2(v.z, v.w);
    }
    static __device__ __forceinline__ Raw pack(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
};

__device__ __forceinline__ float factor(const Params& p, float sum) {
    return p.norm == KDA_NORM_NONE ? 1.f : rsqrtf((p.norm == KDA_NORM_RMS ? sum / (float)p.D : sum) + p.eps);
}

// D and R multiples of 8, rows 16-byte aligned.  LPR: lanes a row, D / 8 rounded up to a power of 2.
template <typename T, int LPR>
__global__ void __launch_bounds__(NT, 3) qk_norm_rope_kernel(const __grid_constant__ Params p) {
    using decay::fma2;
    using decay::mul2;
    using F = Four<T>;
    extern __shared__ __align__(16) float s_turn[];  // [tile][3][R / 2]: cosine, sine and its negative
    const int tid = threadIdx.x, half = p.R / 2;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0), rows = nt * p.heads;

    // the lane's pairs i .. i + 3: elements i and R / 2 + i behind the first half's start, or eight in a row
    const int l = tid % LPR, i = 4 * l;
    const bool on = 2 * i < p.D, rot = i < half;
    const int a = rot && !p.interleaved ? i : 2 * i, b = rot && !p.interleaved ? half + i : 2 * i + 4;

    constexpr int G = NT / LPR, U = 2;  // rows at a time; rows of a lane on their way
    const T* xq = static_cast<const T*>(p.x[0]) + t0 * p.xs[0];
    const T* xk = static_cast<const T*>(p.x[1]) + t0 * p.xs[1];
    T* yq = static_cast<T*>(p.y[0]) + t0 * p.ys[0];
    T* yk = static_cast<T*>(p.y[1]) + t0 * p.ys[1];
    // row r of the block: its token there, its side and its head's elements (a block's offsets fit 31 bits)
    auto where = [&](int r, int& tt, int& side, int& at) {
        tt = p.per ? (int)__umulhi((uint32_t)r, p.per) : r;
        const int hh = r - tt * p.heads;
        side = hh >= p.Hq;
        at = (hh - (side ? p.Hq : 0)) * p.D;
    };
    typename F::Raw va[U], vb[U];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            va[u] = vb[u] = typename F::Raw{};
            if (r0 + u * G < rows && on) {
                int tt, side, at;
                where(r0 + u * G, tt, side, at);
                const T* src = (side ? xk : xq) + (at + tt * (int)(side ? p.xs[1] : p.xs[0]));
                va[u] = *reinterpret_cast<const typename F::Raw*>(src + a);
                vb[u] = *reinterpret_cast<const typename F::Raw*>(src + b);
            }
        }
    };
    const int first = tid / LPR;
    fetch(first);
    for (int x = tid; x < nt * half; x += NT) {
        const int t = x / half, j = x % half;
        const float2 z = turn(p, t0 + t, j);
        float* to = s_turn + t * 3 * half + j;
        to[0] = z.x;
        to[half] = z.y;
        to[2 * half] = -z.y;
    }
    if (half) __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += G * U) {
        typename F::Raw ca[U], cb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) { ca[u] = va[u]; cb[u] = vb[u]; }
        fetch(first + r0 + G * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = first + r0 + u * G;
            float2 v[4];
            F::unpack(ca[u], v[0], v[1]);
            F::unpack(cb[u], v[2], v[3]);
            float2 s2 = mul2(v[0], v[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = fma2(v[e], v[e], s2);
            float sum = s2.x + s2.y;
#pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            if (r < rows && on) {
                int tt, side, at;
                where(r, tt, side, at);
                const float f = factor(p, sum);
                const float2 ff = make_float2(f, f);
                const float* w = side ? p.w[1] : p.w[0];
                if (w) {
                    const float4 wa = __ldg(reinterpret_cast<const float4*>(w + a)), wb = __ldg(reinterpret_cast<const float4*>(w + b));
                    v[0] = mul2(v[0], mul2(ff, make_float2(wa.x, wa.y)));
                    v[1] = mul2(v[1], mul2(ff, make_float2(wa.z, wa.w)));
                    v[2] = mul2(v[2], mul2(ff, make_float2(wb.x, wb.y)));
                    v[3] = mul2(v[3], mul2(ff, make_float2(wb.z, wb.w)));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], ff);
                }
                if (rot) {
                    const float* from = s_turn + tt * 3 * half + i;
                    const float4 c = *reinterpret_cast<const float4*>(from), s = *reinterpret_cast<const float4*>(from + half);
                    if (p.interleaved) {
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = make_float2(v[e].x * cc[e] - v[e].y * ss[e], v[e].y * cc[e] + v[e].x * ss[e]);
                    } else {
                        const float4 n = *reinterpret_cast<const float4*>(from + 2 * half);
                        const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
                        const float2 a0 = fma2(v[0], c0, mul2(v[2], make_float2(n.x, n.y))), a1 = fma2(v[1], c1, mul2(v[3], make_float2(n.z, n.w)));
                        v[2] = fma2(v[2], c0, mul2(v[0], make_float2(s.x, s.y)));
                        v[3] = fma2(v[3], c1, mul2(v[1], make_float2(s.z, s.w)));
                        v[0] = a0;
                        v[1] = a1;
                    }
                }
                T* dst = (side ? yk : yq) + (at + tt * (int)(side ? p.ys[1] : p.ys[0]));
                __stcs(reinterpret_cast<typename F::Raw*>(dst + a), F::pack(v[0], v[1]));
                __stcs(reinterpret_cast<typename F::Raw*>(dst + b), F::pack(v[2], v[3]));
            }
        }
    }
}

// Any D, R and alignment: a warp a row, a pair of single elements a lane and step.
template <typename T>
__global__ void __launch_bounds__(NT) qk_norm_rope_any_kernel(Params p) {
    extern __shared__ __align__(16) float s_turn[];
    const int tid = threadIdx.x, half = p.R / 2, l = tid & 31;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0);
    float2* turns = reinterpret_cast<float2*>(s_turn);
    for (int x = tid; x < nt * half; x += NT) turns[x] = turn(p, t0 + x / half, x % half);
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
                const float2 z = turns[tt * half + i];
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
    const int grid = (int)((a.tokens + p.tile - 1) / p.tile), bytes = p.tile * (a.R / 2) * 3 * (int)sizeof(float);
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
    bool fast = a.D % 8 == 0 && a.R % 8 == 0 && (((uintptr_t)a.q.weight | (uintptr_t)(Hk ? a.k.weight : nullptr)) & 15u) == 0;
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
    int dev = 0, sms = 1;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    p.tile = 1;
    const long far = max(max(p.xs[0], p.xs[1]), max(p.ys[0], p.ys[1]));  // a block's offsets fit 31 bits
    while (p.tile < 64 && p.tile * p.heads < 256 && p.tile * a.R <= 4096 && a.tokens / (2 * p.tile) >= 4 * sms && far * 2 * p.tile < (1l << 30)) p.tile *= 2;
    // r / heads for r < 2^16 rows of a block by a product (exact: r (per heads - 2^32) < 2^32)
    p.per = p.heads > 1 ? (uint32_t)(((1ull << 32) + p.heads - 1) / p.heads) : 0;
    return a.bf16 ? run<__nv_bfloat16>(a, p, fast) : run<float>(a, p, fast);
}

}  // namespace kda
