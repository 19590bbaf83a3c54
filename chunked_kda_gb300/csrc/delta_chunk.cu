// The gated delta rule with a decay for each head, the form for prompts: which kernels run it.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

size_t delta_chunk_workspace_bytes(bool qkv_bf16, bool o_f32, int B, int T, int H, int K, int V, int N, bool packed) {
    (void)qkv_bf16; (void)o_f32; (void)K; (void)V; (void)N; (void)packed;
    return delta_simt_workspace_bytes(B, T, H);
}

cudaError_t launch_delta_chunk(const DeltaArgs& a) { return launch_delta_simt(a); }

}  // namespace kda
