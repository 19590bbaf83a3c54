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
#include "sm100.cuh"

namespace kda {
namespace {

// 16 bytes of T as floats.  Outputs may be inputs (y is x or gate, h is the stream), so these are ordinary loads,
// and no pointer to such rows is __restrict__: each thread reads its elements before it writes them.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float* p, float* r) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* r) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(r[0], r[1], r[2], r[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* r) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
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
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
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

// E weights, which no output is
template <int E>
__device__ __forceinline__ void load_weights(const float* p, float* r) {
    if constexpr (E == 1) r[0] = __ldg(p);
    else {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
            r[i] = a.x; r[i + 1] = a.y; r[i + 2] = a.z; r[i + 3] = a.w;
        }
    }
}

// 8 consecutive elements in shared memory
template <typename T>
__device__ __forceinline__ void load_s(const T* p, float* r) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = __uint_as_float(w[e] << 16);
            r[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
}

// act(z): 0 z itself, 1 sigmoid, 2 SiLU.  For bf16 rows the exponential is the fast one: its error
// (about 2^-21 for |z| <= 4, 2^-19 at 16) is far below the output's rounding of 2^-9.
template <typename T>
__device__ __forceinline__ float gate_value(float z, int act) {
    if (act == 0) return z;
    const float s = sizeof(T) == 2 ? __fdividef(1.f, 1.f + __expf(-z)) : 1.f / (1.f + expf(-z));
    return act == 2 ? z * s : s;
}

// Gated norm of short rows: G lanes share a row, a vector of 16 bytes each (V of at most 32 vectors),
// so a warp holds 32 / G rows.  Memory bounds it: 16384 x 64 rows of 128 bf16 (805 MB) in 130 us,
// 6.2 TB/s.  Small blocks with few registers keep the most bytes in flight: blocks of 256 threads
// measured 138 us, and two or four rows a lane group, their loads issued together, 158 and 241 us.
constexpr int kRowThreads = 128;
template <typename T, int G>
__global__ void __launch_bounds__(kRowThreads) gated_norm_rows_kernel(const T* x, const T* z,
                                                                      const float* __restrict__ w, float eps, int act,
                                                                      long rows, int V, T* y) {
    constexpr int E = Vec<T>::N;
    const int c = (threadIdx.x % G) * E;
    const long row = (long)blockIdx.x * (kRowThreads / G) + threadIdx.x / G;
    const bool in = c < V && row < rows;
    float a[E], g[E], wv[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        a[i] = g[i] = 0.f;
        wv[i] = 1.f;
    }
    if (in) {
        Vec<T>::load(x + row * V + c, a);
        Vec<T>::load(z + row * V + c, g);
        if (w) load_weights<E>(w + c, wv);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) sum = fmaf(a[i], a[i], sum);
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const float rs = rsqrtf(sum / V + eps);
    if (!in) return;
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] = a[i] * rs * wv[i] * gate_value<T>(g[i], act);
    Vec<T>::store(y + row * V + c, a);
}

// Gated norm, any row length: one warp per row, lanes step over the row in pieces of E elements,
// twice.
template <typename T, int E>
__global__ void __launch_bounds__(256) gated_norm_kernel(const T* x, const T* z,
                                                         const float* __restrict__ w, float eps, int act,
                                                         long rows, int V, T* y) {
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
        if (w) load_weights<E>(w + c, wv);
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = a[i] * rs * (w ? wv[i] : 1.f) * gate_value<T>(g[i], act);
        store_e<T, E>(y + row * V + c, a);
    }
}

// sum over the block's threads, the same value in all of them; `red` is used once
template <int NT>
__device__ __forceinline__ float block_sum(float s, float* red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) s += red[i];
    }
    return s;
}

// E elements of h (before the residual where there is one) from x
template <typename T, int E, bool kShared = false>
__device__ __forceinline__ void scaled(const BlockNormArgs& a, const T* z, int c, float rs, float* h) {
    float t[E];
    if (a.post_w) {
        load_weights<E>(a.post_w + c, t);
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] = h[i] * rs * t[i];
    }
    if (z) {
        if constexpr (kShared) load_s<T>(z + c, t);
        else load_e<T, E>(z + c, t);
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] *= gate_value<T>(t[i], a.act);
    }
    if (a.channel_scale) {
        load_weights<E>(a.channel_scale + c, t);
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] *= t[i];
    }
}

// Block norm, one block of NT threads per row, the row in registers between the two norms: P pieces
// of 8 elements a thread.  Memory bounds it: 16384 rows of 8192 (bf16, float32 stream; 1.61 GB) in
// 278 us, 5.8 TB/s.  Rows of many threads keep few registers a thread, so that several rows are in
// flight on an SM while others wait for their sums: 256 threads of four pieces measured 340 us, 1024
// of one 287.
template <typename T, typename R, int NT, int P>
__global__ void __launch_bounds__(NT) block_norm_kernel(BlockNormArgs a) {
    __shared__ float red[2][NT / 32];
    const long row = blockIdx.x;
    const int D = a.D;
    const T* x = (const T*)a.x + row * D;
    const T* z = a.gate ? (const T*)a.gate + row * D : nullptr;
    const R* r = a.residual ? (const R*)a.residual + row * D : nullptr;
    float h[P][8], t[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (threadIdx.x + p * NT);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[p][i] = t[p][i] = 0.f;
        if (c < D) {
            load_e<T, 8>(x + c, h[p]);
            if (r) load_e<R, 8>(r + c, t[p]);
        }
    }
    float rs = 1.f;
    if (a.post_w) {
        float sum = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[p][i], h[p][i], sum);
        rs = rsqrtf(block_sum<NT>(sum, red[0]) / D + a.eps);
    }
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (threadIdx.x + p * NT);
        if (c >= D) continue;
        scaled<T, 8>(a, z, c, rs, h[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[p][i] = fmaf(a.scale, h[p][i], t[p][i]);
            sum = fmaf(h[p][i], h[p][i], sum);
        }
        if (a.h) store_e<R, 8>((R*)a.h + row * D + c, h[p]);
    }
    if (!a.y) return;
    const float rp = a.pre_w ? rsqrtf(block_sum<NT>(sum, red[1]) / D + a.eps) : 1.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (threadIdx.x + p * NT);
        if (c >= D) continue;
        if (a.pre_w) {
            float w[8];
            load_weights<8>(a.pre_w + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[p][i] *= rp * w[i];
        }
        store_e<T, 8>((T*)a.y + row * D + c, h[p]);
    }
}

// Many long rows: two blocks stay on each SM and take every gridDim.x-th row, the rows after the one in
// work on their way into shared memory (bulk copies, a ring of `stages` rows), so that no load waits
// for the two sums of the row before it.  16384 rows of 8192 (bf16, float32 stream; 1.61 GB) in 245 us,
// 6.6 TB/s, against the 278 us of a block per row.  One block of 1024 threads, whose stores wait for
// its own sums, measured 300 us; two of 256 threads 321; pieces of 4 elements 258.
// A wait that gives up (a copy that never lands) makes that block's remaining rows NaN and is counted.
constexpr int kRingThreads = 512;
constexpr int kRingBytes = 108 * 1024;  // of shared memory for each of the two blocks
constexpr int kRingStages = 8;
__device__ unsigned g_norm_timeouts = 0;

template <typename T, typename R>
__global__ void __launch_bounds__(kRingThreads, 2) block_norm_ring_kernel(BlockNormArgs a, int stages) {
    constexpr int P = 2;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][2][kRingThreads / 32];
    __shared__ uint64_t full[kRingStages];
    const int D = a.D, tid = threadIdx.x;
    const uint32_t xb = D * sizeof(T), rb = a.residual ? D * sizeof(R) : 0, zb = a.gate ? xb : 0, row_bytes = xb + rb + zb;
    const uint32_t base = sm100::smem_u32(ring);
    auto bar = [&](int s) { return sm100::smem_u32(&full[s]); };
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) sm100::mbar_init(bar(s), 1);
        sm100::fence_mbar_init();
    }
    __syncthreads();
    auto load = [&](long row, int s) {  // one thread
        const uint32_t at = base + s * row_bytes;
        sm100::mbar_arrive_expect_tx(bar(s), row_bytes);
        sm100::bulk_load(at, (const T*)a.x + row * D, xb, bar(s));
        if (rb) sm100::bulk_load(at + xb, (const R*)a.residual + row * D, rb, bar(s));
        if (zb) sm100::bulk_load(at + xb + rb, (const T*)a.gate + row * D, zb, bar(s));
    };
    if (tid == 0)
        for (int s = 0; s < stages; ++s)
            if (blockIdx.x + (long)s * gridDim.x < a.rows) load(blockIdx.x + (long)s * gridDim.x, s);
    int s = 0;
    uint32_t phase = 0, odd = 0, gave_up = 0;
    for (long row = blockIdx.x; row < a.rows; row += gridDim.x, odd ^= 1) {
        if (!sm100::mbar_wait(bar(s), phase, gave_up ? 1u : 1u << 22)) {
            if (!gave_up && tid == 0) atomicAdd(&g_norm_timeouts, 1u);
            gave_up = 1;
        }
        const T* x = reinterpret_cast<const T*>(ring + s * row_bytes);
        const R* r = rb ? reinterpret_cast<const R*>(ring + s * row_bytes + xb) : nullptr;
        const T* z = zb ? reinterpret_cast<const T*>(ring + s * row_bytes + xb + rb) : nullptr;
        float h[P][8];
        float rs = 1.f, sum = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = 8 * (tid + p * kRingThreads);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[p][i] = 0.f;
            if (c < D) load_s<T>(x + c, h[p]);
            if (gave_up) h[p][0] = __int_as_float(0x7fc00000);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(h[p][i], h[p][i], sum);
        }
        if (a.post_w) rs = rsqrtf(block_sum<kRingThreads>(sum, red[odd][0]) / D + a.eps);
        sum = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = 8 * (tid + p * kRingThreads);
            if (c >= D) continue;
            scaled<T, 8, true>(a, z, c, rs, h[p]);
            float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (r) load_s<R>(r + c, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[p][i] = fmaf(a.scale, h[p][i], t[i]);
                sum = fmaf(h[p][i], h[p][i], sum);
            }
            if (a.h) store_e<R, 8>((R*)a.h + row * D + c, h[p]);
        }
        // (the sum's barrier also says that every thread has read the row)
        const float rp = rsqrtf(block_sum<kRingThreads>(sum, red[odd][1]) / D + a.eps);
        if (tid == 0 && !gave_up && row + (long)stages * gridDim.x < a.rows) load(row + (long)stages * gridDim.x, s);
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
        if (!a.y) continue;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = 8 * (tid + p * kRingThreads);
            if (c >= D) continue;
            if (a.pre_w) {
                float w[8];
                load_weights<8>(a.pre_w + c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[p][i] *= rp * w[i];
            }
            store_e<T, 8>((T*)a.y + row * D + c, h[p]);
        }
    }
    if (gave_up && tid == 0)  // the copies still in flight
        for (int i = 0; i < stages; ++i) {
            sm100::mbar_wait(bar(s), phase);
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
}

// Rows that no block holds in registers, or of a length that is not whole vectors: three passes.
template <typename T, typename R, int E>
__global__ void __launch_bounds__(256) block_norm_any_kernel(BlockNormArgs a) {
    __shared__ float red[2][8];
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
        rs = rsqrtf(block_sum<256>(sum, red[0]) / D + a.eps);
    }
    auto hidden = [&](int c, float* h) {
        load_e<T, E>(x + c, h);
        scaled<T, E>(a, z, c, rs, h);
        float t[E];
        if (r) load_e<R, E>(r + c, t);
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] = fmaf(a.scale, h[i], r ? t[i] : 0.f);
    };
    float sum = 0.f;
    if (a.pre_w)
        for (int c = threadIdx.x * E; c < D; c += 256 * E) {
            float h[E];
            hidden(c, h);
#pragma unroll
            for (int i = 0; i < E; ++i) sum = fmaf(h[i], h[i], sum);
        }
    const float rp = a.pre_w ? rsqrtf(block_sum<256>(sum, red[1]) / D + a.eps) : 1.f;
    for (int c = threadIdx.x * E; c < D; c += 256 * E) {
        float h[E], t[E];
        hidden(c, h);
        if (a.h) store_e<R, E>((R*)a.h + row * D + c, h);
        if (a.pre_w) {
            load_weights<E>(a.pre_w + c, t);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] *= rp * t[i];
        }
        if (a.y) store_e<T, E>((T*)a.y + row * D + c, h);
    }
}

template <typename T, typename R>
cudaError_t launch_block(const BlockNormArgs& a) {
    // Rows too long for one piece a thread, enough of them for 8 a multiprocessor, and two fit the ring.
    // 1.07 to 1.6 GB with / without the ring: 16384 x 8192 bf16 with a float32 stream 250 / 278 us, a bf16 one
    // 176 / 241, none 160 / 221; 26214 x 5120 260 / 346, gated 294 / 436; float32 332 / 363.  At 4096
    // and below a block per row is ahead (4096: 250 / 238; 2048: 343 / 231).  Beyond 8192 the ring's kernel has no
    // registers for a third piece: a block of 1024 threads per row there, 10922 x 12288 (bf16, float32 stream, 1.61 GB)
    // in 397 us, 8192 x 16384 in 341.
    if (a.D % 8 == 0 && a.D > 8 * kRingThreads && a.D <= 16 * kRingThreads) {
        const int row_bytes = a.D * (int)((a.gate ? 2 : 1) * sizeof(T) + (a.residual ? sizeof(R) : 0));
        const int stages = min(kRingStages, kRingBytes / row_bytes), sms = planned_sm_count();
        if (stages >= 2 && a.rows >= 8l * sms) {
            auto kern = block_norm_ring_kernel<T, R>;
            const int bytes = stages * row_bytes;
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess) return e;
            kern<<<2 * sms, kRingThreads, bytes, a.stream>>>(a, stages);
            return cudaGetLastError();
        }
    }
    const unsigned g = (unsigned)a.rows;
    // threads for a row: one piece of 8 elements each up to 4096 elements, two up to 16384
    if (a.D % 8 != 0) block_norm_any_kernel<T, R, 1><<<g, 256, 0, a.stream>>>(a);
    else if (a.D <= 256) block_norm_kernel<T, R, 32, 1><<<g, 32, 0, a.stream>>>(a);
    else if (a.D <= 1024) block_norm_kernel<T, R, 128, 1><<<g, 128, 0, a.stream>>>(a);
    else if (a.D <= 2048) block_norm_kernel<T, R, 256, 1><<<g, 256, 0, a.stream>>>(a);
    else if (a.D <= 4096) block_norm_kernel<T, R, 512, 1><<<g, 512, 0, a.stream>>>(a);
    else if (a.D <= 8192) block_norm_kernel<T, R, 512, 2><<<g, 512, 0, a.stream>>>(a);
    else if (a.D <= 16384) block_norm_kernel<T, R, 1024, 2><<<g, 1024, 0, a.stream>>>(a);
    else block_norm_any_kernel<T, R, 8><<<g, 256, 0, a.stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int G>
void gated_rows(const GatedNormArgs& a) {
    constexpr int rows = kRowThreads / G;
    gated_norm_rows_kernel<T, G><<<(unsigned)((a.rows + rows - 1) / rows), kRowThreads, 0, a.stream>>>(
        (const T*)a.x, (const T*)a.gate, a.weight, a.eps, a.act, a.rows, a.V, (T*)a.y);
}

template <typename T>
cudaError_t launch_gated(const GatedNormArgs& a) {
    constexpr int E = Vec<T>::N;
    const unsigned grid = (unsigned)((a.rows + 7) / 8);
    if (a.V % E != 0)
        gated_norm_kernel<T, 1><<<grid, 256, 0, a.stream>>>((const T*)a.x, (const T*)a.gate, a.weight, a.eps, a.act,
                                                            a.rows, a.V, (T*)a.y);
    else if (a.V <= 4 * E) gated_rows<T, 4>(a);
    else if (a.V <= 8 * E) gated_rows<T, 8>(a);
    else if (a.V <= 16 * E) gated_rows<T, 16>(a);
    else if (a.V <= 32 * E) gated_rows<T, 32>(a);
    else
        gated_norm_kernel<T, E><<<grid, 256, 0, a.stream>>>((const T*)a.x, (const T*)a.gate, a.weight, a.eps, a.act,
                                                            a.rows, a.V, (T*)a.y);
    return cudaGetLastError();
}

}  // namespace

cudaError_t read_norm_timeouts(unsigned* count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, g_norm_timeouts, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_norm_timeouts, &zero, sizeof(unsigned));
    }
    return e;
}

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
