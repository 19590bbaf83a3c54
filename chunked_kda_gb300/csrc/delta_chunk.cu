// The gated delta rule with a decay for each head, the form for prompts: which kernels run it.  On the tensor cores where
// the operands' types hold what the call is given and asked for: bf16 inputs and output, heads that TMA's 16-byte rows and
// a panel of 128 key channels take (4 x 4096 tokens, 64 heads of 128 x 128: 0.61 ms, in FP32 6.3; 64 tokens, 32 heads: 15 us,
// 45).  All else in FP32.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

size_t delta_chunk_workspace_bytes(bool qkv_bf16, bool o_f32, int B, int T, int H, int K, int V, int N, bool packed) {
    (void)N;
    return delta_tensor_dims(qkv_bf16 && !o_f32, K, V) ? delta_tensor_workspace_bytes(B, T, H, K, V, packed) : delta_simt_workspace_bytes(B, T, H);
}

cudaError_t launch_delta_chunk(const DeltaArgs& a) {
    return delta_tensor_dims(a.qkv_bf16 && !a.o_f32, a.K, a.V) ? launch_delta_tensor(a) : launch_delta_simt(a);
}

}  // namespace kda
