// C ABI of the operators around the recurrence (decayed linear attention, gated and block norms,
// short convolution): host-side validation and dispatch.  The contract: include/kda.h.
#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

kda_status fail(kda_status st, const char* msg) {
    kda::record_error(msg);
    return st;
}
bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
bool act_ok(kda_act a) { return a == KDA_ACT_NONE || a == KDA_ACT_SIGMOID || a == KDA_ACT_SILU; }
template <typename... P>
bool aligned(P... ptrs) {
    const void* all[] = {ptrs...};
    for (const void* p : all)
        if (((uintptr_t)p & 15u) != 0) return false;
    return true;
}
const char* const kMisaligned = "pointers must be 16-byte aligned";

// A buffer of a call.  Blocks of one launch read and write in no order, so an output may share memory with an
// input only where each element is read by the thread that later writes it: the very same buffer, where the
// kernels keep to that.
struct Buffer {
    const void* p;
    size_t bytes;
};
bool apart(Buffer a, Buffer b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return !x || !y || !a.bytes || !b.bytes || x + a.bytes <= y || y + b.bytes <= x;
}
bool same_or_apart(Buffer a, Buffer b) { return (a.p == b.p && a.bytes == b.bytes) || apart(a, b); }
template <typename... B>
bool all_apart(Buffer a, B... b) {
    return (apart(a, b) && ...);
}

kda_status check_decay(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const float* decay, bool per_token,
                       const float* h0, const float* hT, const int32_t* cu, int n_seqs, int B, int T, int H,
                       int n_qk_heads, int K, int V, const void* o, kda_dtype o_dtype, int* N) {
    if (n_qk_heads < 0 || (n_qk_heads > 0 && (H <= 0 || H % n_qk_heads != 0)))
        return fail(KDA_ERR_INVALID_ARG, "n_qk_heads must divide H");
    const kda_status st = kda::check_sequences(cu, n_seqs, B, T, H, N);
    if (st != KDA_OK) return st;
    if (H > 65535) return fail(KDA_ERR_INVALID_ARG, "H must be <= 65535");
    if (!dtype_ok(qkv_dtype)) return fail(KDA_ERR_UNSUPPORTED, "qkv dtype");
    if (o_dtype != qkv_dtype && o_dtype != KDA_F32)
        return fail(KDA_ERR_UNSUPPORTED, "o dtype must be the qkv dtype or float32");
    if (K < 1 || K > 256 || V < 1 || V > 256) return fail(KDA_ERR_UNSUPPORTED, "K and V must be in [1, 256]");
    if ((long long)B * T > 0 && *N > 0 && (!q || !k || !v || !decay || !o))
        return fail(KDA_ERR_INVALID_ARG, "null q, k, v, decay or o");
    if (!aligned(q, k, v, h0, hT, o)) return fail(KDA_ERR_INVALID_ARG, kMisaligned);
    // (a token's decays out of a batch with few heads lie anywhere, and are read one by one)
    if (((uintptr_t)decay & 3u) != 0) return fail(KDA_ERR_INVALID_ARG, "decay must be 4-byte aligned");
    if (*N == 0) return KDA_OK;
    const size_t e = qkv_dtype == KDA_BF16 ? 2 : 4, tokens = (size_t)B * T, Hk = n_qk_heads > 0 ? n_qk_heads : H;
    const size_t qk = tokens * Hk * K * e, state = (size_t)*N * H * K * V * 4;
    const Buffer bq{q, qk}, bk{k, qk}, bv{v, tokens * H * V * e}, bd{decay, (per_token ? tokens : 1) * H * 4};
    const Buffer b0{h0, state}, bT{hT, state}, bo{o, tokens * H * V * (o_dtype == KDA_BF16 ? 2 : 4)};
    const Buffer bc{cu, cu ? (size_t)(*N + 1) * 4 : 0};
    if (!all_apart(bo, bq, bk, bd, b0, bT, bc) || !same_or_apart(bo, bv))
        return fail(KDA_ERR_INVALID_ARG, "o must not overlap an input or a state");
    if (!all_apart(bT, bq, bk, bv, bd, bc) || !same_or_apart(bT, b0))
        return fail(KDA_ERR_INVALID_ARG, "final_state must not overlap an input (it may be initial_state)");
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_decay_chunk_workspace_bytes(kda_dtype qkv_dtype, int B, int T, int H, int K, int V, int n_seqs) {
    if (!dtype_ok(qkv_dtype) || B < 0 || T < 0 || H <= 0 || n_seqs < 0 || K < 1 || K > 256 || V < 1 || V > 256)
        return 0;
    const bool packed = n_seqs > 0;
    return kda::decay_chunk_workspace_bytes(qkv_dtype == KDA_BF16, B, T, H, K, V, packed ? n_seqs : B, packed);
}

kda_status kda_decay_chunk_fwd(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                               const float* decay, int decay_per_token, const float* initial_state,
                               float* final_state, const int32_t* cu_seqlens, int n_seqs, int B, int T, int H,
                               int n_qk_heads, int K, int V, void* o, kda_dtype o_dtype, void* workspace,
                               size_t workspace_bytes, int32_t* status, kda_stream_t stream) {
    kda::record_error("");
    int N = 0;
    const kda_status st = check_decay(q, k, v, qkv_dtype, decay, decay_per_token != 0, initial_state, final_state,
                                      cu_seqlens, n_seqs, B, T, H, n_qk_heads, K, V, o, o_dtype, &N);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    const size_t need = kda::decay_chunk_workspace_bytes(qkv_dtype == KDA_BF16, B, T, H, K, V, N, cu_seqlens != nullptr);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(KDA_ERR_INVALID_ARG, "workspace smaller than kda_decay_chunk_workspace_bytes()");
    if (((uintptr_t)workspace & 255u) != 0) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (((uintptr_t)status & 3u) != 0) return fail(KDA_ERR_INVALID_ARG, "status must be 4-byte aligned");
    const kda::DecayArgs a{q, k, v, qkv_dtype == KDA_BF16, decay, decay_per_token != 0, initial_state, final_state,
                           cu_seqlens, N, B, T, H, n_qk_heads > 0 ? n_qk_heads : H, K, V, o, o_dtype == KDA_F32,
                           workspace, reinterpret_cast<int*>(status), (cudaStream_t)stream};
    return kda::launch_status(kda::launch_decay_chunk(a));
}

kda_status kda_decay_recurrent_fwd(const void* q, const void* k, const void* v, kda_dtype qkv_dtype,
                                   const float* decay, int decay_per_token, const float* initial_state,
                                   float* final_state, const int32_t* cu_seqlens, int n_seqs, int B, int T, int H,
                                   int n_qk_heads, int K, int V, void* o, kda_dtype o_dtype, kda_stream_t stream) {
    kda::record_error("");
    int N = 0;
    const kda_status st = check_decay(q, k, v, qkv_dtype, decay, decay_per_token != 0, initial_state, final_state,
                                      cu_seqlens, n_seqs, B, T, H, n_qk_heads, K, V, o, o_dtype, &N);
    if (st != KDA_OK) return st;
    const kda::DecayArgs a{q, k, v, qkv_dtype == KDA_BF16, decay, decay_per_token != 0, initial_state, final_state,
                           cu_seqlens, N, B, T, H, n_qk_heads > 0 ? n_qk_heads : H, K, V, o, o_dtype == KDA_F32,
                           nullptr, nullptr, (cudaStream_t)stream};
    return kda::launch_status(kda::launch_decay_recurrent(a));
}

kda_status kda_gated_norm_fwd(const void* x, const void* gate, kda_dtype dtype, const float* weight, float eps,
                              kda_act act, int64_t rows, int V, void* y, kda_stream_t stream) {
    kda::record_error("");
    if (!dtype_ok(dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype");
    if (!act_ok(act)) return fail(KDA_ERR_INVALID_ARG, "act");
    if (rows < 0 || rows >= (1ll << 31)) return fail(KDA_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
    if (V < 1 || V > (1 << 20)) return fail(KDA_ERR_INVALID_ARG, "V must be in [1, 2^20]");
    if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    if (rows == 0) return KDA_OK;
    if (!x || !gate || !y) return fail(KDA_ERR_INVALID_ARG, "null x, gate or y");
    if (!aligned(x, gate, weight, y)) return fail(KDA_ERR_INVALID_ARG, kMisaligned);
    const size_t bytes = (size_t)rows * V * (dtype == KDA_BF16 ? 2 : 4);
    const Buffer by{y, bytes};
    if (!same_or_apart(by, {x, bytes}) || !same_or_apart(by, {gate, bytes}) || !apart(by, {weight, (size_t)V * 4}))
        return fail(KDA_ERR_INVALID_ARG, "y must not overlap weight, or x or gate in part (it may be x or gate)");
    const kda::GatedNormArgs a{x, gate, dtype == KDA_BF16, weight, eps, (int)act, (long)rows, V, y, (cudaStream_t)stream};
    return kda::launch_status(kda::launch_gated_norm(a));
}

kda_status kda_block_norm_fwd(const void* x, kda_dtype dtype, const void* residual, kda_dtype residual_dtype,
                              const float* post_weight, const void* gate, kda_act act, float scale,
                              const float* channel_scale, const float* pre_weight, float eps, int64_t rows, int D,
                              void* h_out, void* y_out, kda_stream_t stream) {
    kda::record_error("");
    if (!dtype_ok(dtype) || !dtype_ok(residual_dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype");
    if (!act_ok(act)) return fail(KDA_ERR_INVALID_ARG, "act");
    if (rows < 0 || rows >= (1ll << 31)) return fail(KDA_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
    if (D < 1 || D > (1 << 20)) return fail(KDA_ERR_INVALID_ARG, "D must be in [1, 2^20]");
    if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    if (rows == 0) return KDA_OK;
    if (!x || (!h_out && !y_out)) return fail(KDA_ERR_INVALID_ARG, "null x, or neither h_out nor y_out");
    if (!aligned(x, residual, post_weight, gate, channel_scale, pre_weight, h_out, y_out))
        return fail(KDA_ERR_INVALID_ARG, kMisaligned);
    const size_t n = (size_t)rows * D, bytes = n * (dtype == KDA_BF16 ? 2 : 4), per = (size_t)D * 4;
    const Buffer bx{x, bytes}, bz{gate, bytes}, br{residual, n * (residual_dtype == KDA_BF16 ? 2 : 4)};
    const Buffer bh{h_out, br.bytes}, by{y_out, bytes};
    if (!apart(bh, by)) return fail(KDA_ERR_INVALID_ARG, "h_out and y_out must not overlap");
    for (const Buffer& out : {bh, by})
        if (!same_or_apart(out, bx) || !same_or_apart(out, bz) || !same_or_apart(out, br) ||
            !all_apart(out, Buffer{post_weight, per}, Buffer{channel_scale, per}, Buffer{pre_weight, per}))
            return fail(KDA_ERR_INVALID_ARG, "h_out and y_out must not overlap a weight, or an input in part");
    const kda::BlockNormArgs a{x, dtype == KDA_BF16, residual, residual_dtype == KDA_BF16, post_weight, gate, (int)act,
                               scale, channel_scale, pre_weight, eps, (long)rows, D, h_out, y_out, (cudaStream_t)stream};
    return kda::launch_status(kda::launch_block_norm(a));
}

kda_status kda_short_conv_fwd(const void* x, kda_dtype dtype, const float* weight, const float* bias, kda_act act,
                              int W, const void* initial_state, void* final_state, const int32_t* cu_seqlens,
                              int n_seqs, int B, int T, int D, void* y, kda_stream_t stream) {
    kda::record_error("");
    if (D < 1 || D > (1 << 20)) return fail(KDA_ERR_INVALID_ARG, "D must be in [1, 2^20]");
    int N = 0;
    const kda_status st = kda::check_sequences(cu_seqlens, n_seqs, B, T, D, &N);
    if (st != KDA_OK) return st;
    if (!dtype_ok(dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype");
    if (!act_ok(act)) return fail(KDA_ERR_INVALID_ARG, "act");
    if (W < 2 || W > 8) return fail(KDA_ERR_UNSUPPORTED, "W must be in [2, 8]");
    if (N == 0) return KDA_OK;
    if ((long long)B * T > 0 && (!x || !weight || !y)) return fail(KDA_ERR_INVALID_ARG, "null x, weight or y");
    if ((long long)B * T == 0 && !final_state) return KDA_OK;
    if (!weight) return fail(KDA_ERR_INVALID_ARG, "null weight");
    if (!aligned(x, weight, bias, initial_state, final_state, y)) return fail(KDA_ERR_INVALID_ARG, kMisaligned);
    const size_t e = dtype == KDA_BF16 ? 2 : 4, bytes = (size_t)B * T * D * e, state = (size_t)N * (W - 1) * D * e;
    const Buffer bx{x, bytes}, by{y, bytes}, b0{initial_state, state}, b1{final_state, state};
    const Buffer bw{weight, (size_t)D * W * 4}, bb{bias, (size_t)D * 4}, bc{cu_seqlens, cu_seqlens ? (size_t)(N + 1) * 4 : 0};
    if (!all_apart(by, bx, bw, bb, b0, b1, bc))  // (a tile reads the W - 1 rows before it, which another block writes)
        return fail(KDA_ERR_INVALID_ARG, "y must not overlap x, a weight or a state");
    if (!all_apart(b1, bx, bw, bb, bc) || !same_or_apart(b1, b0))
        return fail(KDA_ERR_INVALID_ARG, "final_state must not overlap an input (it may be initial_state)");
    const kda::ConvArgs a{x, dtype == KDA_BF16, weight, bias, (int)act, W, initial_state, final_state, cu_seqlens,
                          N, B, T, D, y, (cudaStream_t)stream};
    return kda::launch_status(kda::launch_short_conv(a));
}

}  // extern "C"
