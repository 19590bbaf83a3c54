// C ABI of the gated delta rule with a decay for each head, and of the norm and rotation of queries and keys:
// host-side validation and dispatch.  The contract: include/kda.h.
#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

kda_status fail(kda_status st, const char* msg) {
    kda::record_error(msg);
    return st;
}
bool dtype_ok(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }
size_t size_of(kda_dtype t) { return t == KDA_BF16 ? 2 : 4; }
template <typename... P>
bool aligned(uintptr_t to, P... ptrs) {
    const void* all[] = {ptrs...};
    for (const void* p : all)
        if (((uintptr_t)p & (to - 1)) != 0) return false;
    return true;
}

// A buffer of a call.  Blocks of one launch read and write in no order, so an output may share memory with an
// input only where each element is read by the thread that later writes it.
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

// `rows` pieces of `width` bytes, `stride` bytes apart
struct Rows {
    const void* p;
    size_t rows, width, stride;
    Buffer span() const { return {p, rows ? (rows - 1) * stride + width : 0}; }
};
bool apart(const Rows& a, const Rows& b) {
    if (apart(a.span(), b.span())) return true;
    if (a.stride != b.stride) return false;
    // side by side in rows of one length: the second's pieces begin `at` bytes behind the first's
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p, S = a.stride;
    const size_t at = y >= x ? (y - x) % S : (S - (x - y) % S) % S;
    return at >= a.width && S - at >= b.width;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride && a.width == b.width; }

kda_status check_delta(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const void* g, kda_dtype g_dtype,
                       const float* A_log, const float* dt_bias, kda_gate_mode mode, const void* beta, kda_dtype beta_dtype,
                       const float* h0, const float* hT, const int32_t* cu, int n_seqs, int B, int T, int H, int n_qk_heads,
                       int K, int V, const void* o, kda_dtype o_dtype, unsigned flags, int* N) {
    if (flags & ~(KDA_FLAG_Q_L2NORM | KDA_FLAG_K_L2NORM | KDA_FLAG_BETA_LOGITS))
        return fail(KDA_ERR_INVALID_ARG, "unknown flag bits");
    if (n_qk_heads < 0 || (n_qk_heads > 0 && (H <= 0 || H % n_qk_heads != 0)))
        return fail(KDA_ERR_INVALID_ARG, "n_qk_heads must divide H");
    const kda_status st = kda::check_sequences(cu, n_seqs, B, T, H, N);
    if (st != KDA_OK) return st;
    if (H > 65535) return fail(KDA_ERR_INVALID_ARG, "H must be <= 65535");
    // (a chunk's rows, and those asked for ahead, are counted in 32 bits past the last token)
    if ((long long)B * T > (1ll << 31) - 256) return fail(KDA_ERR_INVALID_ARG, "B * T must be at most 2^31 - 256");
    if (!dtype_ok(qkv_dtype)) return fail(KDA_ERR_UNSUPPORTED, "qkv dtype");
    if (!dtype_ok(g_dtype)) return fail(KDA_ERR_UNSUPPORTED, "g dtype");
    if (beta_dtype != qkv_dtype && beta_dtype != KDA_F32)
        return fail(KDA_ERR_UNSUPPORTED, "beta dtype must be the qkv dtype or float32");
    if (o_dtype != qkv_dtype && o_dtype != KDA_F32)
        return fail(KDA_ERR_UNSUPPORTED, "o dtype must be the qkv dtype or float32");
    if (K < 1 || K > 256 || V < 1 || V > 256) return fail(KDA_ERR_UNSUPPORTED, "K and V must be in [1, 256]");
    if (mode != KDA_GATE_PRE && mode != KDA_GATE_NONSAFE)
        return fail(KDA_ERR_UNSUPPORTED, "gate mode must be KDA_GATE_PRE or KDA_GATE_NONSAFE");
    if (*N > 0 && mode == KDA_GATE_NONSAFE && !A_log) return fail(KDA_ERR_INVALID_ARG, "A_log is required by KDA_GATE_NONSAFE");
    if ((long long)B * T > 0 && *N > 0 && (!q || !k || !v || !g || !beta || !o))
        return fail(KDA_ERR_INVALID_ARG, "null q, k, v, g, beta or o");
    if (!aligned(16, q, k, v, h0, hT, o)) return fail(KDA_ERR_INVALID_ARG, "q, k, v, o and the states must be 16-byte aligned");
    // (a token's gates out of a batch with few heads lie anywhere, and are read one by one)
    if (!aligned(size_of(g_dtype), g) || !aligned(size_of(beta_dtype), beta) || !aligned(4, A_log, dt_bias))
        return fail(KDA_ERR_INVALID_ARG, "g, beta, A_log and dt_bias must be aligned to their elements");
    if (*N == 0) return KDA_OK;
    const size_t e = size_of(qkv_dtype), tokens = (size_t)B * T, Hk = n_qk_heads > 0 ? n_qk_heads : H;
    const size_t qk = tokens * Hk * K * e, state = (size_t)*N * H * K * V * 4, heads = (size_t)H * 4;
    const bool raw = mode == KDA_GATE_NONSAFE;
    const Buffer bq{q, qk}, bk{k, qk}, bv{v, tokens * H * V * e}, bg{g, tokens * H * size_of(g_dtype)};
    const Buffer bb{beta, tokens * H * size_of(beta_dtype)}, bA{raw ? A_log : nullptr, heads}, bd{raw ? dt_bias : nullptr, heads};
    const Buffer b0{h0, state}, bT{hT, state}, bo{o, tokens * H * V * size_of(o_dtype)};
    const Buffer bc{cu, cu ? (size_t)(*N + 1) * 4 : 0};
    if (!all_apart(bo, bq, bk, bg, bb, bA, bd, b0, bT, bc) || !same_or_apart(bo, bv))
        return fail(KDA_ERR_INVALID_ARG, "o must not overlap an input or a state (it may be v)");
    if (!all_apart(bT, bq, bk, bv, bg, bb, bA, bd, bc) || !same_or_apart(bT, b0))
        return fail(KDA_ERR_INVALID_ARG, "final_state must not overlap an input (it may be initial_state)");
    return KDA_OK;
}

kda::DeltaArgs args_of(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const void* g, kda_dtype g_dtype,
                       const float* A_log, const float* dt_bias, kda_gate_mode mode, const void* beta, kda_dtype beta_dtype,
                       const float* h0, float* hT, const int32_t* cu, int N, int B, int T, int H, int n_qk_heads, int K,
                       int V, void* o, kda_dtype o_dtype, unsigned flags, kda_stream_t stream) {
    return {q, k, v, qkv_dtype == KDA_BF16, g, g_dtype == KDA_BF16, A_log, dt_bias, (int)mode, beta, beta_dtype == KDA_BF16, h0, hT,
            cu, N, B, T, H, n_qk_heads > 0 ? n_qk_heads : H, K, V, o, o_dtype == KDA_F32, flags, nullptr, nullptr,
            (cudaStream_t)stream};
}

}  // namespace

extern "C" {

size_t kda_delta_chunk_workspace_bytes(kda_dtype qkv_dtype, kda_dtype o_dtype, int B, int T, int H, int K, int V, int n_seqs) {
    if (!dtype_ok(qkv_dtype) || !dtype_ok(o_dtype) || B < 0 || T < 0 || H <= 0 || n_seqs < 0 || K < 1 || K > 256 || V < 1 || V > 256)
        return 0;
    const bool packed = n_seqs > 0;
    return kda::delta_chunk_workspace_bytes(qkv_dtype == KDA_BF16, o_dtype == KDA_F32, B, T, H, K, V, packed);
}

kda_status kda_delta_chunk_fwd(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const void* g,
                               kda_dtype g_dtype, const float* A_log, const float* dt_bias, kda_gate_mode mode,
                               const void* beta, kda_dtype beta_dtype, const float* initial_state, float* final_state,
                               const int32_t* cu_seqlens, int n_seqs, int B, int T, int H, int n_qk_heads, int K, int V,
                               void* o, kda_dtype o_dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                               int32_t* status, kda_stream_t stream) {
    kda::record_error("");
    int N = 0;
    const kda_status st = check_delta(q, k, v, qkv_dtype, g, g_dtype, A_log, dt_bias, mode, beta, beta_dtype, initial_state,
                                      final_state, cu_seqlens, n_seqs, B, T, H, n_qk_heads, K, V, o, o_dtype, flags, &N);
    if (st != KDA_OK) return st;
    if (N == 0) return KDA_OK;
    kda::DeltaArgs a = args_of(q, k, v, qkv_dtype, g, g_dtype, A_log, dt_bias, mode, beta, beta_dtype, initial_state,
                               final_state, cu_seqlens, N, B, T, H, n_qk_heads, K, V, o, o_dtype, flags, stream);
    const size_t need = kda::delta_chunk_workspace_bytes(a.qkv_bf16, a.o_f32, B, T, H, K, V, cu_seqlens != nullptr);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(KDA_ERR_INVALID_ARG, "workspace smaller than kda_delta_chunk_workspace_bytes()");
    if (!aligned(256, workspace)) return fail(KDA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (!aligned(4, status)) return fail(KDA_ERR_INVALID_ARG, "status must be 4-byte aligned");
    a.ws = workspace;
    a.status = reinterpret_cast<int*>(status);
    return kda::launch_status(kda::launch_delta_chunk(a));
}

kda_status kda_delta_recurrent_fwd(const void* q, const void* k, const void* v, kda_dtype qkv_dtype, const void* g,
                                   kda_dtype g_dtype, const float* A_log, const float* dt_bias, kda_gate_mode mode,
                                   const void* beta, kda_dtype beta_dtype, const float* initial_state, float* final_state,
                                   const int32_t* cu_seqlens, int n_seqs, int B, int T, int H, int n_qk_heads, int K,
                                   int V, void* o, kda_dtype o_dtype, unsigned flags, kda_stream_t stream) {
    kda::record_error("");
    int N = 0;
    const kda_status st = check_delta(q, k, v, qkv_dtype, g, g_dtype, A_log, dt_bias, mode, beta, beta_dtype, initial_state,
                                      final_state, cu_seqlens, n_seqs, B, T, H, n_qk_heads, K, V, o, o_dtype, flags, &N);
    if (st != KDA_OK) return st;
    return kda::launch_status(kda::launch_delta_recurrent(
        args_of(q, k, v, qkv_dtype, g, g_dtype, A_log, dt_bias, mode, beta, beta_dtype, initial_state, final_state, cu_seqlens,
                N, B, T, H, n_qk_heads, K, V, o, o_dtype, flags, stream)));
}

kda_status kda_qk_norm_rope_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, kda_dtype dtype,
                                const float* q_weight, const float* k_weight, kda_norm norm, float eps,
                                const int32_t* positions, int n_axes, const float* inv_freq,
                                const unsigned char* pair_axes, int R, int interleaved, float rope_scale,
                                int64_t tokens, int Hq, int Hk, int D, void* q_out, int64_t q_out_stride, void* k_out,
                                int64_t k_out_stride, kda_stream_t stream) {
    kda::record_error("");
    if (!dtype_ok(dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype");
    if (norm != KDA_NORM_NONE && norm != KDA_NORM_RMS && norm != KDA_NORM_L2) return fail(KDA_ERR_INVALID_ARG, "norm");
    if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps must be >= 0");
    if (D < 1 || D > 256) return fail(KDA_ERR_UNSUPPORTED, "D must be in [1, 256]");
    if (R < 0 || R > D || R % 2 != 0) return fail(KDA_ERR_INVALID_ARG, "R must be even and in [0, D]");
    if (Hq < 1 || Hk < 0 || (long)Hq + Hk > 4096) return fail(KDA_ERR_INVALID_ARG, "Hq must be >= 1, Hk >= 0, both together <= 4096");
    if (tokens < 0 || tokens >= (1ll << 31)) return fail(KDA_ERR_INVALID_ARG, "tokens must be in [0, 2^31)");
    if (R > 0 && (n_axes < 1 || n_axes > 4)) return fail(KDA_ERR_INVALID_ARG, "n_axes must be in [1, 4]");
    if (R > 0 && pair_axes)
        for (int i = 0; i < R / 2; ++i)
            if (pair_axes[i] >= n_axes) return fail(KDA_ERR_INVALID_ARG, "pair_axes must be below n_axes");
    if (tokens == 0) return KDA_OK;
    if (!q || !q_out || (Hk > 0 && (!k || !k_out))) return fail(KDA_ERR_INVALID_ARG, "null q, k, q_out or k_out");
    if (R > 0 && (!positions || !inv_freq)) return fail(KDA_ERR_INVALID_ARG, "null positions or inv_freq");
    const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hk * D, far = 1ll << 40;
    if (q_stride < wq || q_out_stride < wq || q_stride > far || q_out_stride > far ||
        (Hk > 0 && (k_stride < wk || k_out_stride < wk || k_stride > far || k_out_stride > far)))
        return fail(KDA_ERR_INVALID_ARG, "a token's stride must be at least its heads' elements");
    const size_t e = size_of(dtype), n = (size_t)tokens;
    if (!aligned(e, q, q_out) || (Hk > 0 && !aligned(e, k, k_out)) || !aligned(4, positions, inv_freq, q_weight, k_weight))
        return fail(KDA_ERR_INVALID_ARG, "pointers must be aligned to their elements");
    const Rows iq{q, n, wq * e, q_stride * e}, oq{q_out, n, wq * e, q_out_stride * e};
    const Rows ik{Hk ? k : nullptr, n, wk * e, k_stride * e}, ok{Hk ? k_out : nullptr, n, wk * e, k_out_stride * e};
    const Buffer bp{R ? positions : nullptr, (size_t)n_axes * n * 4}, bf{R ? inv_freq : nullptr, (size_t)R * 2};
    const Buffer bwq{q_weight, (size_t)D * 4}, bwk{k_weight, (size_t)D * 4};
    if (Hk && !apart(oq, ok)) return fail(KDA_ERR_INVALID_ARG, "q_out and k_out must not overlap");
    if (!(same(oq, iq) || apart(oq, iq)) || (Hk && (!(same(ok, ik) || apart(ok, ik)) || !apart(oq, ik) || !apart(ok, iq))))
        return fail(KDA_ERR_INVALID_ARG, "q_out and k_out must not overlap q or k (q_out may be q, k_out k)");
    for (const Rows& o : {oq, ok})
        if (!all_apart(o.span(), bp, bf, bwq, bwk))
            return fail(KDA_ERR_INVALID_ARG, "q_out and k_out must not overlap the positions, frequencies or weights");
    const kda::QkNormArgs a{{q, (long)q_stride, q_weight, q_out, (long)q_out_stride, Hq},
                            {Hk ? k : nullptr, (long)k_stride, k_weight, k_out, (long)k_out_stride, Hk},
                            dtype == KDA_BF16, (int)norm, eps, positions, n_axes, inv_freq, pair_axes, R, interleaved != 0,
                            rope_scale, (long)tokens, D, (cudaStream_t)stream};
    return kda::launch_status(kda::launch_qk_norm_rope(a));
}

}  // extern "C"
