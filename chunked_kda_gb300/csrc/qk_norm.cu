// The norm of query and key heads and the rotation of their positions, in one pass.
//
// Per row of D elements (a token's head):
//   y = x [/ sqrt(mean(x^2) + eps) * weight]   or   x / sqrt(sum(x^2) + eps) [* weight]
//   of the first R elements, each pair: (y_a, y_b) <- m (y_a cos - y_b sin, y_b cos + y_a sin),
//   angle = p f,   p = the token's position on the pair's axis, f = inv_freq of the pair.
//
// The angle is wanted modulo a turn only, and positions are integers: f / 2 pi is taken modulo 1 as a 64-bit
// fraction (integer product of f's 24 bits and 2^64 / 2 pi, cut to 2^-64 turns), and p times it modulo 2^64 is exact.  So an
// angle is off by at most p (1 + f / 2) 2^-64 turns, below 2^-33 (1 + f / 2) for any position; its upper 32 bits are then rounded
// to a float of at most half a turn (2^-25 of it).  A float32 product is off by 0.06 radians at p = 10^6.
//
// A row is split between lanes so that both elements of a pair lie in one lane (two pieces of a row, R / 2 apart, or one
// behind another), and LPR lanes share a row.
//
// Memory bounds it: each row goes in and out once.  16384 tokens with 64 + 8 heads of 128, RMS norm, rotation: 604 MB in
// 101 us, 6.0 TB/s (with angles formed in FP32 for each row and no loads ahead: 260); 20480 tokens with 32 heads, L2 norm,
// no rotation: 57 us, 5.9 TB/s.  Four kernels: many rows, few
// rows, whole words of bf16, and any D, R and alignment.
#include "common.cuh"
#include "kda_internal.h"
#include "sm100.cuh"
#include "tile_ops.cuh"

namespace kda {
namespace {

constexpr int NT = 256, kMaxD = 256;
constexpr int kRingStage = 2048, kRingStages = 3, kRingBlocks = 2;  // bytes of a warp's stage, stages, blocks an SM
__device__ unsigned g_rope_timeouts = 0;

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
    float eps, per_sum;  // 1 / D of a mean, else 1
    const int32_t* pos;
    const float* freq;
    Axes axes;
    int R, D, interleaved;
    float m;
    long tokens;
    int tile;
    // the ring's groups: rows of one, groups of a token's queries, of a token
    int G, q_groups, per_token;
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
    // P elements (4 or 8) as P / 2 pairs
    template <int P>
    static __device__ __forceinline__ void load(const __nv_bfloat16* x, float2* v) {
        if constexpr (P == 4) {
            unpack(*reinterpret_cast<const uint2*>(x), v[0], v[1]);
        } else {
            const uint4 r = *reinterpret_cast<const uint4*>(x);
            unpack(make_uint2(r.x, r.y), v[0], v[1]);
            unpack(make_uint2(r.z, r.w), v[2], v[3]);
        }
    }
    template <int P>
    static __device__ __forceinline__ void store(__nv_bfloat16* y, const float2* v) {
        const uint2 a = pack(v[0], v[1]);
        if constexpr (P == 4) {
            *reinterpret_cast<uint2*>(y) = a;
        } else {
            const uint2 b = pack(v[2], v[3]);
            *reinterpret_cast<uint4*>(y) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
};
template <>
struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ void unpack(Raw v, float2& a, float2& b) {
        a = make_float2(v.x, v.y);
        b = make_float2(v.z, v.w);
    }
    static __device__ __forceinline__ Raw pack(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
    template <int P>
    static __device__ __forceinline__ void load(const float* x, float2* v) {
#pragma unroll
        for (int e = 0; e < P / 4; ++e) unpack(reinterpret_cast<const float4*>(x)[e], v[2 * e], v[2 * e + 1]);
    }
    template <int P>
    static __device__ __forceinline__ void store(float* y, const float2* v) {
#pragma unroll
        for (int e = 0; e < P / 4; ++e) reinterpret_cast<float4*>(y)[e] = pack(v[2 * e], v[2 * e + 1]);
    }
};

__device__ __forceinline__ float factor(const Params& p, float sum) {
    return p.norm == KDA_NORM_NONE ? 1.f : rsqrtf(fmaf(sum, p.per_sum, p.eps));
}

__device__ __forceinline__ void load_weights(const float* wa, const float* wb, float2 (&w)[4]) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(wa)), y = __ldg(reinterpret_cast<const float4*>(wb));
    w[0] = make_float2(x.x, x.y);
    w[1] = make_float2(x.z, x.w);
    w[2] = make_float2(y.x, y.y);
    w[3] = make_float2(y.z, y.w);
}

// A lane's four pairs: the norm's factor, the weights, the rotation.  turns: cosines, R / 2 further sines, as far again
// the sines' negatives, of the lane's first pair.
__device__ __forceinline__ void finish(const Params& p, float f, bool weighted, const float2 (&w)[4], bool rot, const float* turns, float2 (&v)[4]) {
    using decay::fma2;
    using decay::mul2;
    const float2 ff = make_float2(f, f);
    if (weighted) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], mul2(ff, w[e]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], ff);
    }
    if (!rot) return;
    const int half = p.R / 2;
    const float4 c = *reinterpret_cast<const float4*>(turns), s = *reinterpret_cast<const float4*>(turns + half);
    if (p.interleaved) {
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = make_float2(v[e].x * cc[e] - v[e].y * ss[e], v[e].y * cc[e] + v[e].x * ss[e]);
    } else {
        const float4 n = *reinterpret_cast<const float4*>(turns + 2 * half);
        const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
        const float2 a0 = fma2(v[0], c0, mul2(v[2], make_float2(n.x, n.y))), a1 = fma2(v[1], c1, mul2(v[3], make_float2(n.z, n.w)));
        v[2] = fma2(v[2], c0, mul2(v[0], make_float2(s.x, s.y)));
        v[3] = fma2(v[3], c1, mul2(v[1], make_float2(s.z, s.w)));
        v[0] = a0;
        v[1] = a1;
    }
}

// Few rows, D and R multiples of 8, 16-byte aligned.  A block has `tile` consecutive tokens with all their
// heads: the angles' cosines and sines are formed once a token, in shared memory, while the first rows are on their way.  A
// lane has four pairs, LPR lanes a row (D / 8 rounded up to a power of 2).  The next U rows of a lane are on their way while it
// works on U (U: 1, 2, 3, 4 gave 124, 111, 126 and 129 us for 16384 tokens with 72 heads).
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
                const float* w = side ? p.w[1] : p.w[0];
                float2 wv[4];
                if (w) load_weights(w + a, w + b, wv);
                finish(p, factor(p, sum), w != nullptr, wv, rot, s_turn + tt * 3 * half + i, v);
                T* dst = (side ? yk : yq) + (at + tt * (int)(side ? p.ys[1] : p.ys[0]));
                __stcs(reinterpret_cast<typename F::Raw*>(dst + a), F::pack(v[0], v[1]));
                __stcs(reinterpret_cast<typename F::Raw*>(dst + b), F::pack(v[2], v[3]));
            }
        }
    }
}

// Many rows, D and R multiples of 2 P (16, else 8), 16-byte aligned.  A warp has an even share of all groups (up to p.G rows of one token
// and side, one behind another) and a ring of their stages in shared memory, which bulk copies fill and empty; it forms
// the angles of each of its tokens for itself and meets no other warp.  A lane has P pairs of a row, LPR lanes a row (D / 2 P
// rounded up to a power of 2), so that a warp works on few rows at a time and a token's angles stay in registers.
// Three stages of 2 KB for 16 warps an SM: 101 us (16384 tokens, 72 heads, rotation) and 57 us (20480, 32, none); two stages
// 121 and 66, four 101 and 60, six 102 and 63 (more copies under way disturb the stores), three of 4 KB 110 and 61,
// 24 warps with four 130 and 58.  P = 4 (104 of 128 elements rotated, 16384 tokens, 72 heads): 118 us, a block's rows by ordinary
// loads 127.
template <typename T, int P, int LPR>
__global__ void __launch_bounds__(NT, kRingBlocks) qk_norm_rope_ring_kernel(const __grid_constant__ Params p) {
    using decay::fma2;
    using decay::mul2;
    using F = Four<T>;
    constexpr int W = NT / 32, RP = 32 / LPR;  // rows at a time
    extern __shared__ __align__(128) float sm[];
    __shared__ __align__(8) uint64_t s_full[W][kRingStages];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, half = p.R / 2;
    float* turns = sm + w * (kRingStages * kRingStage / 4 + 2 * half);  // cosines, sines of a token
    uint8_t* ring = reinterpret_cast<uint8_t*>(turns + 2 * half);
    const uint32_t bars = sm100::smem_u32(s_full[w]), to = sm100::smem_u32(ring);
    if (lane == 0) {
        for (int s = 0; s < kRingStages; ++s) sm100::mbar_init(bars + 8 * s, 1);
        sm100::fence_mbar_init();
    }
    __syncwarp();
    const long warps = (long)gridDim.x * W, me = (long)blockIdx.x * W + w;
    const long all = p.tokens * p.per_token, first = all * me / warps, count = all * (me + 1) / warps - first;
    struct At {
        long t;  // token
        int g;   // group of the token
    };
    const At begin{first / p.per_token, (int)(first % p.per_token)};
    auto next = [&](At& x) {
        if (++x.g == p.per_token) {
            x.g = 0;
            ++x.t;
        }
    };
    // a group's side, first element behind its token's, and rows
    auto where = [&](At x, int& side, int& at, int& n) {
        side = x.g >= p.q_groups;
        const int first = (x.g - (side ? p.q_groups : 0)) * p.G, heads = side ? p.heads - p.Hq : p.Hq;
        at = first * p.D;
        n = min(p.G, heads - first);
    };
    At ahead = begin;
    long issued = 0;
    auto load = [&](int s) {
        if (issued == count) return;
        if (lane == 0) {
            int side, at, n;
            where(ahead, side, at, n);
            const uint32_t bytes = n * p.D * (uint32_t)sizeof(T);
            sm100::mbar_arrive_expect_tx(bars + 8 * s, bytes);
            sm100::bulk_load(to + s * kRingStage, static_cast<const T*>(p.x[side]) + ahead.t * p.xs[side] + at, bytes, bars + 8 * s);
        }
        next(ahead);
        ++issued;
    };
    for (int s = 0; s < kRingStages; ++s) load(s);

    // the lane's pairs i .. i + P - 1: elements i and R / 2 + i behind the first half's start, or 2 P in a row
    const int l = lane % LPR, row = lane / LPR, i = P * l;
    const bool in = 2 * i < p.D, rot = i < half;
    const int a = rot && !p.interleaved ? i : 2 * i, b = rot && !p.interleaved ? half + i : 2 * i + P;
    float2 co[P / 2] = {}, si[P / 2] = {}, ni[P / 2] = {}, wv[P] = {};
    At now = begin;
    long formed = -1;  // the token whose angles are there
    int s = 0, weights = -1;
    uint32_t phase = 0;
    bool gave_up = false;
    for (long g = 0; g < count; ++g, next(now)) {
        int side, at, n;
        where(now, side, at, n);
        if (half && now.t != formed) {
            __syncwarp();
            for (int j = lane; j < half; j += 32) {
                const float2 z = turn(p, now.t, j);
                turns[j] = z.x;
                turns[half + j] = z.y;
            }
            formed = now.t;
            __syncwarp();
            if (rot)
#pragma unroll
                for (int e = 0; e < P / 2; ++e) {
                    co[e] = *reinterpret_cast<const float2*>(turns + i + 2 * e);
                    si[e] = *reinterpret_cast<const float2*>(turns + half + i + 2 * e);
                    ni[e] = make_float2(-si[e].x, -si[e].y);
                }
        }
        const float* wt = side ? p.w[1] : p.w[0];
        if (wt && in && weights != side) {
#pragma unroll
            for (int e = 0; e < P / 2; ++e) {
                wv[e] = __ldg(reinterpret_cast<const float2*>(wt + a) + e);
                wv[P / 2 + e] = __ldg(reinterpret_cast<const float2*>(wt + b) + e);
            }
            weights = side;
        }
        if (!__all_sync(0xffffffffu, sm100::mbar_wait(bars + 8 * s, phase))) {
            if (lane == 0) atomicAdd(&g_rope_timeouts, 1u);
            gave_up = true;
            break;
        }
        T* x = reinterpret_cast<T*>(ring + s * kRingStage);
        for (int r0 = 0; r0 < n; r0 += RP) {
            const bool on = r0 + row < n && in;
            T* at_row = x + (r0 + row) * p.D;
            float2 v[P];
#pragma unroll
            for (int e = 0; e < P; ++e) v[e] = make_float2(0.f, 0.f);
            if (on) {
                F::template load<P>(at_row + a, v);
                F::template load<P>(at_row + b, v + P / 2);
            }
            float sum = 0.f;
            if (p.norm != KDA_NORM_NONE) {
                float2 s2 = mul2(v[0], v[0]), s3 = mul2(v[P / 2], v[P / 2]);
#pragma unroll
                for (int e = 1; e < P / 2; ++e) {
                    s2 = fma2(v[e], v[e], s2);
                    s3 = fma2(v[P / 2 + e], v[P / 2 + e], s3);
                }
                sum = (s2.x + s2.y) + (s3.x + s3.y);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            }
            if (!on) continue;
            const float f = factor(p, sum);
            const float2 ff = make_float2(f, f);
            if (wt) {
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] = mul2(v[e], mul2(ff, wv[e]));
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] = mul2(v[e], ff);
            }
            if (rot && !p.interleaved) {
#pragma unroll
                for (int e = 0; e < P / 2; ++e) {
                    const float2 first = fma2(v[e], co[e], mul2(v[P / 2 + e], ni[e]));
                    v[P / 2 + e] = fma2(v[P / 2 + e], co[e], mul2(v[e], si[e]));
                    v[e] = first;
                }
            } else if (rot) {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float c = e & 1 ? co[e / 2].y : co[e / 2].x, sn = e & 1 ? si[e / 2].y : si[e / 2].x;
                    v[e] = make_float2(v[e].x * c - v[e].y * sn, v[e].y * c + v[e].x * sn);
                }
            }
            F::template store<P>(at_row + a, v);
            F::template store<P>(at_row + b, v + P / 2);
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            sm100::bulk_store(static_cast<T*>(p.y[side]) + now.t * p.ys[side] + at, to + s * kRingStage, n * p.D * (uint32_t)sizeof(T));
            decay::bulk_commit();
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the stage before this one has been read
        }
        __syncwarp();
        if (g > 0) load(s > 0 ? s - 1 : kRingStages - 1);
        if (++s == kRingStages) {
            s = 0;
            phase ^= 1;
        }
    }
    if (lane == 0) decay::bulk_wait_read();
    if (gave_up)  // the copies still in flight
        for (long g = max(0l, issued - kRingStages); g < issued; ++g)
            sm100::mbar_wait(bars + 8 * (uint32_t)(g % kRingStages), (uint32_t)(g / kRingStages) & 1u);
}

// bf16 rows of whole words of two elements (any even D, any R): a warp U rows at a time, a word a lane and step, S steps (D / 64
// rounded up to a power of 2).  Elements that R / 2 lies between meet through shared memory, as floats.  (Loads and stores of
// single elements, pairs of which a lane holds by itself, took 2 to 3 times the time: half words are stored to half
// sectors.)  16384 tokens with 72 heads of 128, 106 elements rotated: 201 us, single elements 275 to 330.
template <int S>
__global__ void __launch_bounds__(NT) qk_norm_rope_words_kernel(const __grid_constant__ Params p) {
    constexpr int U = S < 4 ? 4 : 2;
    extern __shared__ __align__(16) float s_turn[];
    const int tid = threadIdx.x, half = p.R / 2, words = p.D / 2, l = tid & 31, w = tid >> 5;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0), rows = nt * p.heads;
    float2* turns = reinterpret_cast<float2*>(s_turn);
    float* mix = s_turn + p.tile * p.R + w * U * p.R;  // the warp's rows' first R elements
    for (int x = tid; x < nt * half; x += NT) turns[x] = turn(p, t0 + x / half, x % half);
    if (half) __syncthreads();
    float2 wt[2][S];  // both sides' weights
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = l + 32 * s;
            wt[side][s] = make_float2(1.f, 1.f);
            if (p.w[side] && i < words) wt[side][s] = make_float2(__ldg(p.w[side] + 2 * i), __ldg(p.w[side] + 2 * i + 1));
        }
    for (int r0 = w; r0 < rows; r0 += U * (NT / 32)) {
        uint32_t v[U][S];
        float sum[U];
        int side[U], tt[U];
        long at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * (NT / 32), last = min(r, rows - 1);  // (rows behind the last are formed, too, and not stored)
            tt[u] = p.per ? (int)__umulhi((uint32_t)last, p.per) : last;
            const int hh = last - tt[u] * p.heads;
            side[u] = hh >= p.Hq;
            at[u] = (long)(hh - (side[u] ? p.Hq : 0)) * p.D;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(side[u] ? p.x[1] : p.x[0]) +
                                                                    (t0 + tt[u]) * (side[u] ? p.xs[1] : p.xs[0]) + at[u]);
#pragma unroll
            for (int s = 0; s < S; ++s) v[u][s] = r < rows && l + 32 * s < words ? src[l + 32 * s] : 0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) sum[u] = fmaf(sm100::bf_lo(v[u][s]), sm100::bf_lo(v[u][s]), fmaf(sm100::bf_hi(v[u][s]), sm100::bf_hi(v[u][s]), sum[u]));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], m);
        float2 y[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = factor(p, sum[u]);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int i = l + 32 * s;
                const float2 wv = side[u] ? wt[1][s] : wt[0][s];
                y[u][s] = make_float2(sm100::bf_lo(v[u][s]) * f * wv.x, sm100::bf_hi(v[u][s]) * f * wv.y);
                if (i >= half) continue;
                if (p.interleaved) {
                    const float2 z = turns[tt[u] * half + i], x = y[u][s];
                    y[u][s] = make_float2(x.x * z.x - x.y * z.y, x.y * z.x + x.x * z.y);
                } else {
                    *reinterpret_cast<float2*>(mix + u * p.R + 2 * i) = y[u][s];
                }
            }
        }
        if (half && !p.interleaved) {
            __syncwarp();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int i = l + 32 * s;
                    if (i >= half) continue;
                    const float2 z = turns[tt[u] * half + i];
                    float *a = mix + u * p.R + i, *b = a + half;
                    const float xa = *a, xb = *b;
                    *a = xa * z.x - xb * z.y;
                    *b = xb * z.x + xa * z.y;
                }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (l + 32 * s < half) y[u][s] = *reinterpret_cast<const float2*>(mix + u * p.R + 2 * (l + 32 * s));
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r0 + u * (NT / 32) >= rows) break;
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(side[u] ? p.y[1] : p.y[0]) +
                                                        (t0 + tt[u]) * (side[u] ? p.ys[1] : p.ys[0]) + at[u]);
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (l + 32 * s < words) __stcs(dst + l + 32 * s, sm100::pack_bf16(y[u][s].x, y[u][s].y));
        }
    }
}

// Any D, R and alignment: a warp U rows at a time, a pair of single elements a lane and step.  float32: 8192 tokens with 72
// heads of 128, 34 elements rotated, 110 us (153 with one row at a time).
template <typename T, int S>
__global__ void __launch_bounds__(NT) qk_norm_rope_any_kernel(const __grid_constant__ Params p) {
    constexpr int U = S < 4 ? 4 : 2;
    extern __shared__ __align__(16) float s_turn[];
    const int tid = threadIdx.x, half = p.R / 2, l = tid & 31;
    const long t0 = (long)blockIdx.x * p.tile;
    const int nt = (int)min((long)p.tile, p.tokens - t0), rows = nt * p.heads;
    float2* turns = reinterpret_cast<float2*>(s_turn);
    for (int x = tid; x < nt * half; x += NT) turns[x] = turn(p, t0 + x / half, x % half);
    if (half) __syncthreads();
    int a[S], b[S];
    float wa[2][S], wb[2][S];  // both sides' weights
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int i = l + 32 * s;
        const bool apart = i < half && !p.interleaved;
        a[s] = apart ? i : 2 * i;
        b[s] = apart ? half + i : 2 * i + 1;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const float* w = p.w[side];
            wa[side][s] = w && a[s] < p.D ? __ldg(w + a[s]) : 1.f;
            wb[side][s] = w && b[s] < p.D ? __ldg(w + b[s]) : 1.f;
        }
    }
    for (int r0 = tid >> 5; r0 < rows; r0 += U * (NT / 32)) {
        float va[U][S], vb[U][S], sum[U];
        int side[U], tt[U], at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * (NT / 32);
            tt[u] = p.per ? (int)__umulhi((uint32_t)r, p.per) : r;
            const int hh = r - tt[u] * p.heads;
            side[u] = hh >= p.Hq;
            at[u] = (hh - (side[u] ? p.Hq : 0)) * p.D;
            const T* src = static_cast<const T*>(side[u] ? p.x[1] : p.x[0]) + (t0 + tt[u]) * (side[u] ? p.xs[1] : p.xs[0]) + at[u];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                va[u][s] = r < rows && a[s] < p.D ? to_f32(src[a[s]]) : 0.f;
                vb[u][s] = r < rows && b[s] < p.D ? to_f32(src[b[s]]) : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) sum[u] = fmaf(va[u][s], va[u][s], fmaf(vb[u][s], vb[u][s], sum[u]));
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r0 + u * (NT / 32) >= rows) break;
            const float f = factor(p, sum[u]);
            T* dst = static_cast<T*>(side[u] ? p.y[1] : p.y[0]) + (t0 + tt[u]) * (side[u] ? p.ys[1] : p.ys[0]) + at[u];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (a[s] >= p.D) continue;
                float ya = va[u][s] * f * (side[u] ? wa[1][s] : wa[0][s]), yb = vb[u][s] * f * (side[u] ? wb[1][s] : wb[0][s]);
                if (l + 32 * s < half) {
                    const float2 z = turns[tt[u] * half + l + 32 * s];
                    const float xa = ya, xb = yb;
                    ya = xa * z.x - xb * z.y;
                    yb = xb * z.x + xa * z.y;
                }
                dst[a[s]] = from_f32<T>(ya);
                if (b[s] < p.D) dst[b[s]] = from_f32<T>(yb);
            }
        }
    }
}

template <typename T>
cudaError_t run_ring(const QkNormArgs& a, const Params& p, int sms) {
    auto kern = a.D > 128 ? qk_norm_rope_ring_kernel<T, 8, 16> : a.D > 64 ? qk_norm_rope_ring_kernel<T, 8, 8> : qk_norm_rope_ring_kernel<T, 8, 4>;
    if (a.D % 16 != 0 || a.R % 16 != 0)
        kern = a.D > 128 ? qk_norm_rope_ring_kernel<T, 4, 32> : a.D > 64 ? qk_norm_rope_ring_kernel<T, 4, 16> : a.D > 32 ? qk_norm_rope_ring_kernel<T, 4, 8>
               : qk_norm_rope_ring_kernel<T, 4, 4>;
    const int bytes = NT / 32 * (kRingStages * kRingStage + a.R * (int)sizeof(float));
    // (the limit is the kernel's, not the call's: what the largest one wants, so that calls of several host threads do not meet in it)
    constexpr int most = NT / 32 * (kRingStages * kRingStage + kMaxD * (int)sizeof(float));
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    kern<<<kRingBlocks * sms, NT, bytes, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run(const QkNormArgs& a, Params& p, bool fast, bool words) {
    const int grid = (int)((a.tokens + p.tile - 1) / p.tile);
    int bytes = p.tile * (a.R / 2) * 3 * (int)sizeof(float);
    void (*kern)(Params) = a.D > 128 ? qk_norm_rope_any_kernel<T, 4> : a.D > 64 ? qk_norm_rope_any_kernel<T, 2> : qk_norm_rope_any_kernel<T, 1>;
    if (sizeof(T) == 2 && words) {
        kern = a.D > 128 ? qk_norm_rope_words_kernel<4> : a.D > 64 ? qk_norm_rope_words_kernel<2> : qk_norm_rope_words_kernel<1>;
        bytes = p.tile * a.R * 4 + NT / 32 * (a.D > 128 ? 2 : 4) * a.R * 4;
    }
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
    bool words = a.D % 2 == 0;  // rows of bf16 begin at whole words
    for (int s = 0; s < (Hk ? 2 : 1); ++s) {
        p.x[s] = side[s]->x;
        p.y[s] = side[s]->y;
        p.w[s] = side[s]->weight;
        p.xs[s] = side[s]->stride;
        p.ys[s] = side[s]->y_stride;
        words = words && (((uintptr_t)p.x[s] | (uintptr_t)p.y[s] | (uintptr_t)(p.xs[s] * e) | (uintptr_t)(p.ys[s] * e)) & 3u) == 0;
        fast = fast && (((uintptr_t)p.x[s] | (uintptr_t)p.y[s] | (uintptr_t)(p.xs[s] * e) | (uintptr_t)(p.ys[s] * e)) & 15u) == 0;
    }
    p.norm = a.norm;
    p.eps = a.eps;
    p.per_sum = a.norm == KDA_NORM_RMS ? 1.f / (float)a.D : 1.f;
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
    // Many rows: eight groups a warp, of a kilobyte or more (short ones cost a copy each).  4096 tokens, 40 heads of 128: 19 us, the
    // few rows' kernel 20; below, fewer warps of its own have work: 1024 tokens, 40 heads: 7.8 and 7.8.
    if (fast) {
        p.G = kRingStage / (a.D * e);
        p.q_groups = (p.Hq + p.G - 1) / p.G;
        p.per_token = p.q_groups + (Hk + p.G - 1) / p.G;
        const bool ring = a.tokens * p.per_token >= 8l * kRingBlocks * (NT / 32) * sms && (long)p.heads * a.D * e >= 1024l * p.per_token;
        if (ring) return a.bf16 ? run_ring<__nv_bfloat16>(a, p, sms) : run_ring<float>(a, p, sms);
    }
    return a.bf16 ? run<__nv_bfloat16>(a, p, fast, words) : run<float>(a, p, fast, false);
}

cudaError_t read_rope_timeouts(unsigned* count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, g_rope_timeouts, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_rope_timeouts, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace kda
