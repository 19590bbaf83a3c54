// Linear attention with a decay for each head, the form for prompts: which kernels run it.
//
//   bf16 with head sizes that the tensor-core kernel has      decay_tensor.cu
//   else, at most kShort tokens a sequence can have           decay_recurrent.cu: one launch, no scratch
//   else                                                      decay_simt.cu: FP32, all chunks at once
// float32, 2 heads of 64 x 64: T = 64 in 25 us token by token (27 in chunks), T = 128 in 45 (29), T = 256 in
// 86 (29): below 64 the chunks' three launches cost more than the tokens' order.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

static constexpr int kShort = 64;

size_t decay_chunk_workspace_bytes(bool qkv_bf16, int B, int T, int H, int K, int V, int N, bool packed) {
    if (decay_tensor_dims(qkv_bf16, K, V)) return decay_tensor_workspace_bytes(B, T, H, K, V, N, packed);
    return T <= kShort ? 0 : decay_simt_workspace_bytes(B, T, H, K, V, N, packed);
}

cudaError_t launch_decay_chunk(const DecayArgs& a) {
    if (decay_tensor_dims(a.qkv_bf16, a.K, a.V)) return launch_decay_tensor(a);
    return a.T <= kShort ? launch_decay_recurrent(a) : launch_decay_simt(a);
}

}  // namespace kda
