// Short causal convolution of each channel, with the inputs before a sequence kept as its state.
//
//   y_t[d] = act(b[d] + sum_{w < W} weight[d][w] x_{t-W+1+w}[d]),  x before the first token from
//   the state [W-1, D] (oldest row first), whose new value is the last W-1 rows of (state, x).
//
// Grid: chunk slots of TT tokens (ChunkMap; every sequence, an empty one too, has a slot whose
// chunk number is 0) by blocks of channels.  A thread owns E consecutive channels, keeps the last
// W - 1 rows in registers and walks its chunk's tokens.  The slot of a sequence's first chunk also
// writes the sequence's new state, after its threads have read the old one: each thread reads and
// writes only its own channels, so the two may be one buffer.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int TT = 32;

template <typename T, int E>
__device__ __forceinline__ void load_row(const T* p, float* r) {
    if constexpr (E == 1) r[0] = to_f32(*p);
    else if constexpr (sizeof(T) == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = __uint_as_float(w[e] << 16);
            r[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p);
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_row(T* p, const float* r) {
    if constexpr (E == 1) *p = from_f32<T>(r[0]);
    else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(r[2 * e], r[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
    }
}

template <typename T, int W, int E>
__global__ void __launch_bounds__(128) short_conv_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                                                         const float* __restrict__ bias, int act,
                                                         const T* s0, T* s1, ChunkMap cm, int D,
                                                         T* __restrict__ y) {
    int n, t0, len, bos, eos;
    const bool any = cm.map_first(blockIdx.x, n, t0, len, bos, eos);
    if (n < 0) return;
    const int d = E * (blockIdx.y * 128 + threadIdx.x);
    if (d >= D) return;
    const bool first = t0 == bos;
    if (!any && !first) return;
    float win[W][E];  // rows t-W+1 .. t
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
        const int t = t0 - (W - 1) + w;
        if (t >= bos) load_row<T, E>(x + (size_t)t * D + d, win[w]);
        else if (s0) load_row<T, E>(s0 + ((size_t)n * (W - 1) + (t - bos + W - 1)) * D + d, win[w]);
        else {
#pragma unroll
            for (int e = 0; e < E; ++e) win[w][e] = 0.f;
        }
    }
    if (first && s1) {  // the new state: the last W - 1 rows of (state, x)
        const int L = eos - bos;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int t = L - (W - 1) + w;
            float r[E];
            if (t >= 0) load_row<T, E>(x + (size_t)(bos + t) * D + d, r);
            else {
#pragma unroll
                for (int u = 0; u < W - 1; ++u)
                    if (u == t + W - 1) {
#pragma unroll
                        for (int e = 0; e < E; ++e) r[e] = win[u][e];
                    }
            }
            store_row<T, E>(s1 + ((size_t)n * (W - 1) + w) * D + d, r);
        }
    }
    float wt[E][W], b[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        b[e] = bias ? __ldg(bias + d + e) : 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) wt[e][w] = __ldg(weight + (size_t)(d + e) * W + w);
    }
    for (int i = 0; i < len; ++i) {
        load_row<T, E>(x + (size_t)(t0 + i) * D + d, win[W - 1]);
        float out[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float acc = b[e];
#pragma unroll
            for (int w = 0; w < W; ++w) acc = fmaf(wt[e][w], win[w][e], acc);
            const float s = act ? 1.f / (1.f + (sizeof(T) == 2 ? __expf(-acc) : expf(-acc))) : 1.f;
            out[e] = act == 1 ? s : acc * s;
        }
        store_row<T, E>(y + (size_t)(t0 + i) * D + d, out);
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
#pragma unroll
            for (int e = 0; e < E; ++e) win[w][e] = win[w + 1][e];
    }
}

template <typename T, int W, int E>
cudaError_t launch_e(const ConvArgs& a) {
    const ChunkMap cm{a.cu, a.N, a.T, TT};
    // a dense batch of length zero has no chunk, but its states still pass through
    const long slots = a.cu ? (long)a.T / TT + a.N + 1 : (long)a.N * max(1, (a.T + TT - 1) / TT);
    const dim3 grid((unsigned)slots, (a.D / E + 127) / 128);
    short_conv_kernel<T, W, E><<<grid, 128, 0, a.stream>>>((const T*)a.x, a.weight, a.bias, a.act, (const T*)a.s0,
                                                           (T*)a.s1, cm, a.D, (T*)a.y);
    return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const ConvArgs& a) {
    constexpr int E = 16 / sizeof(T);
    return a.D % E == 0 ? launch_e<T, W, E>(a) : launch_e<T, W, 1>(a);
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
