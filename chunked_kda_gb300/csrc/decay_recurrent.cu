// Linear attention with a decay for each head, token by token (decode, short prompts).
//
// Per (sequence, head), state S (K x V, rows = key channels) in FP32:
//   S = e^a S + k v^T;   o = S^T q / sqrt(K),   a = decay of the token and head (or of the head).
//
// One program per (sequence, head, block of BV value columns) holds its K x BV block of S in
// registers.  Warp w owns rows [w KP/8, (w+1) KP/8) (KP = K rounded up to 64, 128 or 256, rows
// beyond K masked), lane l owns BV/32 consecutive columns, so a state row moves as whole vectors.
// A warp's rows are consecutive key channels: their q and k elements are the same for all its
// lanes and come as 16-byte loads, without shared memory.  The only reduction is o's sum over
// the rows: per thread, then across the warps through shared memory, two buffers by token parity
// so that one barrier a token is enough.
//
// Memory bounds it: the state goes in and out once.  512 sequences of one token, 32 heads of 128 x 128
// (2.17 GB) in 310 us, 7.0 TB/s.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

template <int N>
__device__ __forceinline__ void ld_state(const float* p, float* r) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        r[0] = x.x; r[1] = x.y;
    }
}
template <int N>
__device__ __forceinline__ void st_state(float* p, const float* r) {
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(r[0], r[1], r[2], r[3]);
    else *reinterpret_cast<float2*>(p) = make_float2(r[0], r[1]);
}
// 8 consecutive elements from a 16-byte aligned address
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float* r) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r[2 * e] = __uint_as_float(w[e] << 16);
        r[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void ld8(const float* p, float* r) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
}

// MASKED = false when K == KP and BV divides V: no row or column checks.
template <typename InT, typename OutT, int KP, int BV, bool MASKED>
__global__ void __launch_bounds__(256, 2) decay_recurrent_kernel(
    const InT* __restrict__ q, const InT* __restrict__ k, const InT* __restrict__ v,
    const float* __restrict__ decay, int decay_stride, const float* h0, float* hT,
    const int32_t* __restrict__ cu, int T, int H, int hr, int K, int V, OutT* __restrict__ o) {
    constexpr int RPW = KP / 8, VPT = BV / 32;
    __shared__ float s_red[2][8][BV];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int v0 = blockIdx.x * BV, h = blockIdx.y, n = blockIdx.z;
    long bos, eos;
    if (cu) { bos = __ldg(cu + n); eos = __ldg(cu + n + 1); }
    else    { bos = (long)n * T; eos = bos + T; }

    const int row0 = warp * RPW, col = v0 + lane * VPT;
    const size_t st = ((size_t)n * H + h) * (size_t)K * V;
    float S[RPW][VPT];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) S[r][j] = 0.f;
        if (!h0) continue;
        const float* src = h0 + st + (size_t)(row0 + r) * V + col;
        if constexpr (!MASKED) ld_state<VPT>(src, S[r]);
        else if (row0 + r < K) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (col + j < V) S[r][j] = src[j];
        }
    }
    const float scale = rsqrtf((float)K);
    const int Hq = H / hr, hq = h / hr;
    int buf = 0;
    for (long t = bos; t < eos; ++t, buf ^= 1) {
        const size_t qk = ((size_t)t * Hq + hq) * K + row0, vo = ((size_t)t * H + h) * V;
        const float dec = expf(__ldg(decay + (size_t)t * decay_stride + h));
        float kr[RPW], qr[RPW], vr[VPT], op[VPT];
        if constexpr (!MASKED) {
#pragma unroll
            for (int r = 0; r < RPW; r += 8) { ld8(k + qk + r, kr + r); ld8(q + qk + r, qr + r); }
        } else {
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const bool in = row0 + r < K;
                kr[r] = in ? to_f32(k[qk + r]) : 0.f;
                qr[r] = in ? to_f32(q[qk + r]) : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            vr[j] = (!MASKED || col + j < V) ? to_f32(v[vo + col + j]) : 0.f;
            op[j] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < RPW; ++r)
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                S[r][j] = fmaf(S[r][j], dec, kr[r] * vr[j]);
                op[j] = fmaf(S[r][j], qr[r], op[j]);
            }
#pragma unroll
        for (int j = 0; j < VPT; ++j) s_red[buf][warp][lane * VPT + j] = op[j];
        __syncthreads();
        if (tid < BV && (!MASKED || v0 + tid < V)) {
            float acc = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) acc += s_red[buf][w][tid];
            o[vo + v0 + tid] = from_f32<OutT>(acc * scale);
        }
    }
    // every thread has read its part of h0 above and no other program touches it: hT may be h0
    if (!hT) return;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        float* dst = hT + st + (size_t)(row0 + r) * V + col;
        if constexpr (!MASKED) st_state<VPT>(dst, S[r]);
        else if (row0 + r < K) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (col + j < V) dst[j] = S[r][j];
        }
    }
}

template <typename InT, typename OutT, int KP, int BV>
cudaError_t launch_b(const DecayArgs& a) {
    const dim3 grid((a.V + BV - 1) / BV, a.H, a.N);
    const bool masked = a.K != KP || a.V % BV != 0;
    auto kern = masked ? decay_recurrent_kernel<InT, OutT, KP, BV, true>
                       : decay_recurrent_kernel<InT, OutT, KP, BV, false>;
    kern<<<grid, 256, 0, a.stream>>>((const InT*)a.q, (const InT*)a.k, (const InT*)a.v, a.decay,
                                     a.per_token ? a.H : 0, a.h0, a.hT, a.cu, a.T, a.H, a.H / a.Hk, a.K,
                                     a.V, (OutT*)a.o);
    return cudaGetLastError();
}

template <typename InT, typename OutT>
cudaError_t launch_k(const DecayArgs& a) {
    // at most 64 state floats per thread (KP BV / 256)
    if (a.K <= 64) return a.V > 64 ? launch_b<InT, OutT, 64, 128>(a) : launch_b<InT, OutT, 64, 64>(a);
    if (a.K <= 128) return a.V > 64 ? launch_b<InT, OutT, 128, 128>(a) : launch_b<InT, OutT, 128, 64>(a);
    return launch_b<InT, OutT, 256, 64>(a);
}

}  // namespace

cudaError_t launch_decay_recurrent(const DecayArgs& a) {
    if (a.N == 0) return cudaSuccess;
    if (!a.qkv_bf16) return launch_k<float, float>(a);
    return a.o_f32 ? launch_k<__nv_bfloat16, float>(a) : launch_k<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace kda
