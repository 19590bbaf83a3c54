// Linear attention with a decay for each head, the form for prompts: which kernel runs it.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

size_t decay_chunk_workspace_bytes(bool qkv_bf16, int B, int T, int H, int K, int V, int N, bool packed) {
    return decay_tensor_dims(qkv_bf16, K, V) ? decay_tensor_workspace_bytes(B, T, H, K, V, N, packed) : 0;
}

cudaError_t launch_decay_chunk(const DecayArgs& a) {
    return decay_tensor_dims(a.qkv_bf16, a.K, a.V) ? launch_decay_tensor(a) : launch_decay_recurrent(a);
}

}  // namespace kda
