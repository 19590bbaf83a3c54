// The norms of a block: the gated norm of its heads, and the norm around the block with its gate,
// residual and scale.
//
//   gated norm   y = x / sqrt(mean x^2 + eps) * w * act(z)                    one row = one head
//   block norm   n = x [/ sqrt(mean x^2 + eps) * w_post] [* act(z)]
//                h = [r +] scale [* c] * n
//                y = h [/ sqrt(mean h^2 + eps) * w_pre]
//
// Sums, means and the row between the two norms are FP32; h and y are rounded once, and y comes
// from h before its rounding.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

// 16 bytes of T as floats
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float* p, float* r) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* r) {
        *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* r) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = __uint_as_float(w[e] << 16);
            r[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* r) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(r[2 * e], r[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
// 8 consecutive elements, or one
template <typename T, int E>
__device__ __forceinline__ void load_e(const T* p, float* r) {
    if constexpr (E == 1) r[0] = to_f32(*p);
    else {
#pragma unroll
        for (int i = 0; i < E; i += Vec<T>::N) Vec<T>::load(p + i, r + i);
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_e(T* p, const float* r) {
    if constexpr (E == 1) *p = from_f32<T>(r[0]);
    else {
#pragma unroll
        for (int i = 0; i < E; i += Vec<T>::N) Vec<T>::store(p + i, r + i);
    }
}

// act(z): 0 z itself, 1 sigmoid, 2 SiLU.  For bf16 rows the exponential is the fast one: its error
// (about 2^-21 for |z| <= 4, 2^-19 at 16) is far below the output's rounding of 2^-9.
template <typename T>
__device__ __forceinline__ float gate_value(float z, int act) {
    if (act == 0) return z;
    const float s = 1.f / (1.f + (sizeof(T) == 2 ? __expf(-z) : expf(-z)));
    return act == 2 ? z * s : s;
}

// Gated norm: one warp per row, lanes step over the row in pieces of E elements.
template <typename T, int E>
__global__ void __launch_bounds__(256) gated_norm_kernel(const T* __restrict__ x, const T* __restrict__ z,
                                                         const float* __restrict__ w, float eps, int act,
                                                         long rows, int V, T* __restrict__ y) {
    const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    const T* xr = x + row * V;
    float sum = 0.f;
    for (int c = lane * E; c < V; c += 32 * E) {
        float a[E];
        load_e<T, E>(xr + c, a);
#pragma unroll
        for (int i = 0; i < E; ++i) sum = fmaf(a[i], a[i], sum);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const float rs = rsqrtf(sum / V + eps);
    for (int c = lane * E; c < V; c += 32 * E) {
        float a[E], g[E], wv[E];
        load_e<T, E>(xr + c, a);
        load_e<T, E>(z + row * V + c, g);
        if (w) load_e<float, E>(w + c, wv);
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = a[i] * rs * (w ? wv[i] : 1.f) * gate_value<T>(g[i], act);
        store_e<T, E>(y + row * V + c, a);
    }
}

// sum over the block's 256 threads, the same value in all of them
__device__ __forceinline__ float block_sum(float s, float* red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    __syncthreads();  // the readers of an earlier sum are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i];
    return t;
}

// Block norm: one block per row, three passes over it.
template <typename T, typename R, int E>
__global__ void __launch_bounds__(256) block_norm_kernel(BlockNormArgs a) {
    __shared__ float red[8];
    const long row = blockIdx.x;
    const int D = a.D;
    const T* x = (const T*)a.x + row * D;
    const T* z = a.gate ? (const T*)a.gate + row * D : nullptr;
    const R* r = a.residual ? (const R*)a.residual + row * D : nullptr;
    float rs = 1.f;
    if (a.post_w) {
        float sum = 0.f;
        for (int c = threadIdx.x * E; c < D; c += 256 * E) {
            float xv[E];
            load_e<T, E>(x + c, xv);
#pragma unroll
            for (int i = 0; i < E; ++i) sum = fmaf(xv[i], xv[i], sum);
        }
        rs = rsqrtf(block_sum(sum, red) / D + a.eps);
    }
    auto hidden = [&](int c, float* h) {
        float t[E];
        load_e<T, E>(x + c, h);
        if (a.post_w) {
            load_e<float, E>(a.post_w + c, t);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = h[i] * rs * t[i];
        }
        if (z) {
            load_e<T, E>(z + c, t);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] *= gate_value<T>(t[i], a.act);
        }
        if (a.channel_scale) {
            load_e<float, E>(a.channel_scale + c, t);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] *= t[i];
        }
        if (r) {
            load_e<R, E>(r + c, t);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = fmaf(a.scale, h[i], t[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] *= a.scale;
        }
    };
    float sum = 0.f;
    for (int c = threadIdx.x * E; c < D; c += 256 * E) {
        float h[E];
        hidden(c, h);
#pragma unroll
        for (int i = 0; i < E; ++i) sum = fmaf(h[i], h[i], sum);
    }
    const float rp = a.pre_w ? rsqrtf(block_sum(sum, red) / D + a.eps) : 1.f;
    for (int c = threadIdx.x * E; c < D; c += 256 * E) {
        float h[E], t[E];
        hidden(c, h);
        if (a.pre_w) load_e<float, E>(a.pre_w + c, t);
        float yv[E];
#pragma unroll
        for (int i = 0; i < E; ++i) yv[i] = a.pre_w ? h[i] * rp * t[i] : h[i];
        if (a.h) store_e<R, E>((R*)a.h + row * D + c, h);
        if (a.y) store_e<T, E>((T*)a.y + row * D + c, yv);
    }
}

template <typename T, typename R>
cudaError_t launch_block(const BlockNormArgs& a) {
    if (a.D % 8 == 0) block_norm_kernel<T, R, 8><<<(unsigned)a.rows, 256, 0, a.stream>>>(a);
    else block_norm_kernel<T, R, 1><<<(unsigned)a.rows, 256, 0, a.stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gated(const GatedNormArgs& a) {
    const unsigned grid = (unsigned)((a.rows + 7) / 8);
    if (a.V % 8 == 0)
        gated_norm_kernel<T, 8><<<grid, 256, 0, a.stream>>>((const T*)a.x, (const T*)a.gate, a.weight, a.eps,
                                                            a.act, a.rows, a.V, (T*)a.y);
    else
        gated_norm_kernel<T, 1><<<grid, 256, 0, a.stream>>>((const T*)a.x, (const T*)a.gate, a.weight, a.eps,
                                                            a.act, a.rows, a.V, (T*)a.y);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs& a) {
    if (a.rows == 0) return cudaSuccess;
    return a.bf16 ? launch_gated<__nv_bfloat16>(a) : launch_gated<float>(a);
}

cudaError_t launch_block_norm(const BlockNormArgs& a) {
    if (a.rows == 0) return cudaSuccess;
    if (a.bf16)
        return a.res_bf16 ? launch_block<__nv_bfloat16, __nv_bfloat16>(a) : launch_block<__nv_bfloat16, float>(a);
    return a.res_bf16 ? launch_block<float, __nv_bfloat16>(a) : launch_block<float, float>(a);
}

}  // namespace kda
