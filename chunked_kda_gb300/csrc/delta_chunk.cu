// The gated delta rule with a decay for each head, the form for prompts: which kernels run it.  On the tensor cores where
// the operands' types hold what the call is given and asked for: bf16 inputs and output, heads that TMA's 16-byte rows and
// a panel of 128 key channels take (4 x 4096 tokens, 64 heads of 128 x 128: 0.61 ms, in FP32 6.4; 64 tokens, 32 heads: 15 us,
// 45).  All else in FP32.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {
// A few tokens a sequence: token by token.  32 heads of 128 x 128, 512 sequences of 2, 4, 6 tokens: 449, 748, 1066 us, in bf16 chunks
// 1260, in FP32 ones 4020; 8 sequences of 4, 12: 21, 47 us, in chunks 27, in FP32 ones 66; 15 units of 4, 12: 16, 35, in
// chunks 15, in FP32 ones 19.  (Packed lengths are not known here, and one long sequence among short ones would cost a pass
// over its state for each token.)
bool by_token(bool tensor, int B, int T, int H, bool packed) {
    const int sms = planned_sm_count();
    return !packed && (T <= 4 || (!tensor && T <= 16 && sms > 0 && (long)B * H >= sms));
}
}  // namespace

size_t delta_chunk_workspace_bytes(bool qkv_bf16, bool o_f32, int B, int T, int H, int K, int V, bool packed) {
    const bool tensor = delta_tensor_dims(qkv_bf16 && !o_f32, K, V);
    if (by_token(tensor, B, T, H, packed)) return 0;
    return tensor ? delta_tensor_workspace_bytes(B, T, H, K, V, packed) : delta_simt_workspace_bytes(B, T, H);
}

cudaError_t launch_delta_chunk(const DeltaArgs& a) {
    const bool tensor = delta_tensor_dims(a.qkv_bf16 && !a.o_f32, a.K, a.V);
    if (by_token(tensor, a.B, a.T, a.H, a.cu != nullptr)) return launch_delta_recurrent(a);
    return tensor ? launch_delta_tensor(a) : launch_delta_simt(a);
}

}  // namespace kda
