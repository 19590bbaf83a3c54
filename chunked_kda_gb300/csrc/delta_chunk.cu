// The gated delta rule with a decay for each head, the form for prompts: which kernels run it.  On the tensor cores where
// the operands' types hold what the call is given and asked for: bf16 inputs and output, heads that TMA's 16-byte rows and
// a panel of 128 key channels take (4 x 4096 tokens, 64 heads of 128 x 128: 0.62 ms, in FP32 6.4; 64 tokens, 32 heads: 16 us,
// 51).  All else in FP32.
#include "common.cuh"
#include "kda_internal.h"

namespace kda {

namespace {
// A few tokens a sequence: token by token.  A token is a pass over the state, a chunk of few rows costs what a whole one does, and
// its kernels have one unit an SM at a time (the FP32 ones a few).  us token by token / in chunks, heads of 128 x 128:
//   units up to the SMs     8 units    bf16 3 tokens 16/16, 4 18/16      FP32 6 tokens 23/23, 7 26/23
//                           128             3 18/18, 4 20/18                  6 25/37, 7 27/39 (the fewest units decide)
//   up to four an SM        256             5 31/31, 6 35/33                  12 53/61, 13 57/63
//                           512             5 53/57, 6 61/57                  12 104/104, 13 113/106
//   more                    640             6 70/70, 7 78/70                  16 139/139, 18 154/148
//                           2048            7 180/190, 8 201/190              16 352/383, 19 416/410
//                           16384, 8192     7 1221/1296, 8 1376/1301          16 1309/1503, 19 1542/1612
// (smaller heads later, 8192 units of 64 x 64: 7 174/584; FP32 heads of 256 x 256 in bf16 earlier: 12 4326/4989, 16 5720/5165).
// Packed lengths are not known here, and one long sequence among short ones would cost a pass over its state for each token.
bool by_token(bool tensor, int B, int T, int H, int V, bool packed) {
    const long sms = max(1, planned_sm_count()), units = (long)B * H * (tensor ? (V + 127) / 128 : 1);
    const int few = tensor ? 3 : 6, some = tensor ? 5 : 12, many = tensor ? 7 : 16;
    return !packed && T <= (units <= sms ? few : units <= 4 * sms ? some : many);
}
}  // namespace

size_t delta_chunk_workspace_bytes(bool qkv_bf16, bool o_f32, int B, int T, int H, int K, int V, bool packed) {
    const bool tensor = delta_tensor_dims(qkv_bf16 && !o_f32, K, V);
    if (by_token(tensor, B, T, H, V, packed)) return 0;
    return tensor ? delta_tensor_workspace_bytes(B, T, H, K, V, packed) : delta_simt_workspace_bytes(B, T, H);
}

cudaError_t launch_delta_chunk(const DeltaArgs& a) {
    const bool tensor = delta_tensor_dims(a.qkv_bf16 && !a.o_f32, a.K, a.V);
    if (by_token(tensor, a.B, a.T, a.H, a.V, a.cu != nullptr)) return launch_delta_recurrent(a);
    return tensor ? launch_delta_tensor(a) : launch_delta_simt(a);
}

}  // namespace kda
