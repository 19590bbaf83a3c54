// A token's decay and beta of the gated delta rule, as its entry points take them: given, or activated here.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "kda_internal.h"

namespace kda {
namespace delta {

struct Gates {
    const void* g;
    const void* beta;
    const float* A_log;
    const float* dt_bias;
    int H;
    bool g_bf16, beta_bf16, raw, logits;

    Gates() = default;
    explicit Gates(const DeltaArgs& a)
        : g(a.g), beta(a.beta), A_log(a.A_log), dt_bias(a.dt_bias), H(a.H), g_bf16(a.g_bf16), beta_bf16(a.beta_bf16),
          raw(a.mode == 2), logits((a.flags & KDA_FLAG_BETA_LOGITS) != 0) {}

    // a head's exp(A_log) and dt_bias, read once
    struct Head {
        float expA, dtb;
    };
    __device__ __forceinline__ Head head(int h) const {
        return {raw ? expf(__ldg(A_log + h)) : 0.f, raw && dt_bias ? __ldg(dt_bias + h) : 0.f};
    }
    __device__ __forceinline__ static float load(const void* p, bool bf16, size_t i) {
        return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : __ldg(static_cast<const float*>(p) + i);
    }
    // token t's numbers in head h as they lie there
    __device__ __forceinline__ float raw_decay(size_t t, int h) const { return load(g, g_bf16, t * H + h); }
    __device__ __forceinline__ float raw_rate(size_t t, int h) const { return load(beta, beta_bf16, t * H + h); }
    // the natural-log decay and the rate that they stand for
    __device__ __forceinline__ float decay_of(float x, Head c) const { return raw ? gate_act(x, c.expA, c.dtb, 2, 0.f) : x; }
    __device__ __forceinline__ float rate_of(float b) const { return logits ? 1.f / (1.f + expf(-b)) : b; }
    __device__ __forceinline__ float decay(size_t t, int h, Head c) const { return decay_of(raw_decay(t, h), c); }
    __device__ __forceinline__ float rate(size_t t, int h) const { return rate_of(raw_rate(t, h)); }
};

// 1 / |x| of a query or key from its sum of squares.  A sum that is not finite makes the row none (0, as 1 / sqrt gives it
// for what overflows, would leave the row out in silence).
__device__ __forceinline__ float row_norm(float sum) {
    return fabsf(sum) < __int_as_float(0x7f800000) ? rsqrtf(sum + kQNormEps) : __int_as_float(0x7fffffff);
}

}  // namespace delta
}  // namespace kda
