// Short causal convolution of each channel, with the inputs before a sequence kept as its state.
//
//   y_t[d] = act(b[d] + sum_{w < W} weight[d][w] x_{t-W+1+w}[d]),  x before the first token from
//   the state [W-1, D] (oldest row first), whose new value is the last W-1 rows of (state, x).
//
// Memory bounds it: x read and y written once.  Grid: blocks of 128 E channels by tiles of TT
// consecutive rows of the packed (or dense) batch, whatever sequences they belong to.  A thread owns
// E consecutive channels (one vector), keeps their weights and the last W - 1 rows in
// registers and walks the tile; at a row where a sequence starts it takes the rows before it from
// the sequence's state and writes the new one.  A sequence's first W - 1 rows, which read its old
// state, all belong to the tile of its first row (which runs over its end for them), so one thread
// reads the old state of a channel before it writes the new: the two may be one buffer.
//
// Rows are loaded U at a time while the U before them are in work: 20480 packed rows x 12288 bf16
// (1.01 GB) in 162 us, 6.2 TB/s, with 8 rows and six blocks on an SM; 4 rows and eight blocks measured
// 168, 6 and seven 176, 12 and five 174, 16 and four 183; stores that stay in the caches 173.  (float32 rows
// are twice the registers: 4 at a time, 20480 x 6144 in 214 us.)  TT trades the reload of
// W - 1 rows and of the weights against the number of blocks: 64 rows where that leaves eight blocks
// an SM, else 16 or 8.
#include <limits.h>

#include "common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

template <typename T>
struct Raw;  // a vector of E elements as it is in memory
template <>
struct Raw<__nv_bfloat16> {
    using V = uint2;  // 8 bytes: a vector of 16 doubles the registers and halves the warps on an SM
    static constexpr int E = 4;
    static __device__ __forceinline__ void get(const uint2& v, float* r) {
        r[0] = __uint_as_float(v.x << 16);
        r[1] = __uint_as_float(v.x & 0xFFFF0000u);
        r[2] = __uint_as_float(v.y << 16);
        r[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint2 put(const float* r) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(r[0], r[1]), b = __floats2bfloat162_rn(r[2], r[3]);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};
template <>
struct Raw<float> {
    using V = float4;
    static constexpr int E = 4;
    static __device__ __forceinline__ void get(const float4& v, float* r) { r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w; }
    static __device__ __forceinline__ float4 put(const float* r) { return make_float4(r[0], r[1], r[2], r[3]); }
};
// one element at a time, for channel counts that are not whole vectors
template <typename T>
struct One {
    using V = T;
    static constexpr int E = 1;
    static __device__ __forceinline__ void get(const T& v, float* r) { r[0] = to_f32(v); }
    static __device__ __forceinline__ T put(const float* r) { return from_f32<T>(r[0]); }
};

// two FP32 multiply-adds in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

template <typename T>
__device__ __forceinline__ float activate(float a, int act) {
    if (act == 0) return a;
    // bf16: the fast exponential and quotient are far more exact than the output's rounding
    const float s = sizeof(T) == 2 ? __fdividef(1.f, 1.f + __expf(-a)) : 1.f / (1.f + expf(-a));
    return act == 1 ? s : a * s;
}

template <int E, int W>
__device__ __forceinline__ void load_weights(const float* __restrict__ weight, const float* __restrict__ bias, int d,
                                             float (&wt)[E][W], float (&b)[E]) {
    const float* p = weight + (size_t)d * W;
    if constexpr (E * W % 4 == 0) {  // (d is a multiple of E: 16-byte aligned)
#pragma unroll
        for (int i = 0; i < E * W; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
            wt[i / W][i % W] = v.x;
            wt[(i + 1) / W][(i + 1) % W] = v.y;
            wt[(i + 2) / W][(i + 2) % W] = v.z;
            wt[(i + 3) / W][(i + 3) % W] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E * W; ++i) wt[i / W][i % W] = __ldg(p + i);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) b[e] = bias ? __ldg(bias + d + e) : 0.f;
}

// one row: its output from the window of the W rows up to it, and the window moved on
template <typename T, typename Io, int W>
__device__ __forceinline__ void row_step(const typename Io::V& raw, const float (&wt)[Io::E][W], const float (&b)[Io::E],
                                         int act, float (&win)[W][Io::E], T* y) {
    constexpr int E = Io::E;
    Io::get(raw, win[W - 1]);
    float out[E];
    if constexpr (E % 2 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float2 acc = make_float2(b[e], b[e + 1]);
#pragma unroll
            for (int w = 0; w < W; ++w)
                acc = fma2(make_float2(wt[e][w], wt[e + 1][w]), make_float2(win[w][e], win[w][e + 1]), acc);
            out[e] = activate<T>(acc.x, act);
            out[e + 1] = activate<T>(acc.y, act);
        }
    } else {
        float acc = b[0];
#pragma unroll
        for (int w = 0; w < W; ++w) acc = fmaf(wt[0][w], win[w][0], acc);
        out[0] = activate<T>(acc, act);
    }
    if constexpr (E > 1) __stcs(reinterpret_cast<typename Io::V*>(y), Io::put(out));
    else *reinterpret_cast<typename Io::V*>(y) = Io::put(out);
#pragma unroll
    for (int w = 0; w < W - 1; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) win[w][e] = win[w + 1][e];
}

// Single tokens: a thread takes Q whole sequences of its channels, with the states and first rows of
// all of them loaded before the first is used.  (The tiles above walk one start after another, each
// with its loads' latency: 33 us for 512 sequences of one token x 12288 channels, 100 MB, against 21 us here, of which
// the kernel's own are 17.  Where the rows are one sequence's after all, its threads walk them one by one.)
template <typename T, typename Io, int W>
__global__ void __launch_bounds__(128) short_conv_seq_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                                                             const float* __restrict__ bias, int act, const T* s0, T* s1,
                                                             const int32_t* __restrict__ cu, int N, int L, int D,
                                                             T* __restrict__ y) {
    using V = typename Io::V;
    constexpr int E = Io::E, Q = 4;
    const int d = E * (blockIdx.x * 128 + threadIdx.x), n0 = Q * blockIdx.y;
    if (d >= D) return;
    long bos[Q], eos[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int n = min(n0 + q, N - 1);
        bos[q] = cu ? (long)__ldg(cu + n) : (long)n * L;
        eos[q] = cu ? (long)__ldg(cu + n + 1) : (long)(n + 1) * L;
    }
    auto at = [&](long t) { return *reinterpret_cast<const V*>(x + (size_t)t * D + d); };
    auto state = [&](int n, int w) { return (((size_t)n * (W - 1) + w) * D + d) / E; };
    const float zero[E] = {};
    V was[Q][W - 1], row[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int n = min(n0 + q, N - 1);
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            was[q][w] = s0 ? reinterpret_cast<const V*>(s0)[state(n, w)] : Io::put(zero);
        row[q] = bos[q] < eos[q] ? at(bos[q]) : Io::put(zero);
    }
    float wt[E][W], b[E];
    load_weights<E, W>(weight, bias, d, wt, b);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (n0 + q >= N) break;
        float win[W][E];
#pragma unroll
        for (int w = 0; w < W - 1; ++w) Io::get(was[q][w], win[w]);
        V raw = row[q];
#pragma unroll 1
        for (long t = bos[q]; t < eos[q]; ++t) {
            if (t > bos[q]) raw = at(t);
            row_step<T, Io, W>(raw, wt, b, act, win, y + (size_t)t * D + d);
        }
        if (s1) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
                reinterpret_cast<V*>(s1)[state(n0 + q, w)] = bos[q] < eos[q] ? Io::put(win[w]) : was[q][w];
        }
    }
}

// the first of the n + 1 non-decreasing offsets that is >= t (n where only the last one may be), by
// a whole warp, 32 of them at a time
__device__ __forceinline__ int first_at_least(const int32_t* __restrict__ cu, int n, long t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const int below = __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(cu + min(i, n)) < t));
        if (below == 0) break;
        hi = min(lo + below * step, hi);
        lo += (below - 1) * step + 1;
    }
    return lo;
}

template <typename T, typename Io, int W>
__global__ void __launch_bounds__(128, W <= 4 ? 6 : sizeof(typename Io::V) > 8 ? 4 : 5) short_conv_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                                                         const float* __restrict__ bias, int act, const T* s0, T* s1,
                                                         const int32_t* __restrict__ cu, int N, int L, long rows, int TT,
                                                         int D, T* __restrict__ y) {
    using V = typename Io::V;
    constexpr int E = Io::E, U = W <= 4 && sizeof(V) <= 8 ? 8 : 4;
    const int d = E * (blockIdx.x * 128 + threadIdx.x);
    const long t0 = (long)blockIdx.y * TT, t1 = min(t0 + TT, rows);
    // packed: starts cu[0..N-1] and the end cu[N]; dense: starts n L, the end N L
    auto start = [&](int n) -> long { return cu ? (long)__ldg(cu + n) : (long)n * L; };
    int m, behind;  // the first sequences that start at t0 and at t1 or behind
    if (cu) {
        m = first_at_least(cu, N, t0);
        behind = first_at_least(cu, N, t1);
    } else {
        m = L > 0 ? (int)((t0 + L - 1) / L) : 0;
        behind = L > 0 ? (int)((t1 + L - 1) / L) : N;
    }
    if (d >= D) return;
    const long end = start(N);
    long next = m < N ? start(m) : LONG_MAX;
    long t = t0, stop = t1;
    const bool inside = next > t0 && m > 0;  // the tile starts inside sequence m - 1
    if (inside) t = max(t0, min(start(m - 1) + W - 1, start(m)));
    if (behind > m) stop = max(t1, min(start(behind - 1) + W - 1, start(behind)));
    stop = min(stop, end);

    float wt[E][W], b[E];
    load_weights<E, W>(weight, bias, d, wt, b);

    auto at = [&](long t) { return *reinterpret_cast<const V*>(x + (size_t)t * D + d); };
    float win[W][E];  // rows t-W+1 .. t
    const V* old = reinterpret_cast<const V*>(s0);
    auto state_row = [&](int n, int w) { return (((size_t)n * (W - 1) + w) * D + d) / E; };
    if (inside && t < stop) {
#pragma unroll
        for (int w = 0; w < W - 1; ++w) Io::get(at(t - (W - 1) + w), win[w]);
    }
    // sequence m starts: its window, and its new state
    auto begin = [&] {
        const long bos = next, eos = start(m + 1);
        V was[W - 1];
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            if (old) was[w] = old[state_row(m, w)];
            else {
                const float zero[E] = {};
                was[w] = Io::put(zero);
            }
            Io::get(was[w], win[w]);
        }
        if (s1) {
            V now[W - 1];
#pragma unroll
            for (int w = 0; w < W - 1; ++w) {
                const long t = eos - (W - 1) + w;  // the row that takes place w
                if (t >= bos) now[w] = at(t);
                else {
#pragma unroll
                    for (int u = 0; u < W - 1; ++u)
                        if (u == (int)(t - bos) + W - 1) now[w] = was[u];
                }
            }
#pragma unroll
            for (int w = 0; w < W - 1; ++w) reinterpret_cast<V*>(s1)[state_row(m, w)] = now[w];
        }
        ++m;
        next = m < N ? eos : LONG_MAX;
    };

    auto step = [&](const V& raw, long t) { row_step<T, Io, W>(raw, wt, b, act, win, y + (size_t)t * D + d); };
    // runs of rows of one sequence, so that the loop over them looks for no start
    while (t < stop) {
        while (next == t) begin();
        const long run = min(stop, next);
        if (t + U <= run) {
            V r[U], ahead[U];
#pragma unroll
            for (int u = 0; u < U; ++u) r[u] = at(t + u);
#pragma unroll 1
            for (; t + 2 * U <= run; t += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) ahead[u] = at(t + U + u);
#pragma unroll
                for (int u = 0; u < U; ++u) step(r[u], t + u);
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = ahead[u];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) step(r[u], t + u);
            t += U;
        }
#pragma unroll 1
        for (; t < run; ++t) step(at(t), t);
    }
    // empty sequences at the end of all: the tile that would hold their first row, or the last one
    while (m < N && (next < t1 || t1 == rows)) begin();
}

template <typename T, typename Io, int W>
cudaError_t launch_io(const ConvArgs& a) {
    const long rows = max(1l, a.cu ? (long)a.T : (long)a.B * a.T);
    const unsigned blocks = (a.D / Io::E + 127) / 128;
    if (rows <= a.N) {
        short_conv_seq_kernel<T, Io, W><<<dim3(blocks, (a.N + 3) / 4), 128, 0, a.stream>>>(
            (const T*)a.x, a.weight, a.bias, a.act, (const T*)a.s0, (T*)a.s1, a.cu, a.N, a.T, a.D, (T*)a.y);
        return cudaGetLastError();
    }
    const int sms = planned_sm_count();
    auto few = [&](int TT) { return (rows + TT - 1) / TT * blocks < 8l * sms; };
    int TT = few(64) ? few(16) ? 8 : 16 : 64;  // at least W - 1
    // (a grid's second dimension holds 65535 tiles)
    while ((rows + TT - 1) / TT > 65535) TT *= 2;
    short_conv_kernel<T, Io, W><<<dim3(blocks, (unsigned)((rows + TT - 1) / TT)), 128, 0, a.stream>>>(
        (const T*)a.x, a.weight, a.bias, a.act, (const T*)a.s0, (T*)a.s1, a.cu, a.N, a.T, rows, TT, a.D, (T*)a.y);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const ConvArgs& a) {
    return a.D % Raw<T>::E == 0 ? launch_io<T, Raw<T>, W>(a) : launch_io<T, One<T>, W>(a);
}

template <typename T>
cudaError_t launch_t(const ConvArgs& a) {
    switch (a.W) {
        case 2: return launch_w<T, 2>(a);
        case 3: return launch_w<T, 3>(a);
        case 4: return launch_w<T, 4>(a);
        case 5: return launch_w<T, 5>(a);
        case 6: return launch_w<T, 6>(a);
        case 7: return launch_w<T, 7>(a);
        default: return launch_w<T, 8>(a);
    }
}

}  // namespace

cudaError_t launch_short_conv(const ConvArgs& a) {
    if (a.N == 0) return cudaSuccess;
    return a.bf16 ? launch_t<__nv_bfloat16>(a) : launch_t<float>(a);
}

}  // namespace kda
