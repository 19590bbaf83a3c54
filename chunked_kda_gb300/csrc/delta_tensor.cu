// The gated delta rule with a decay for each head in chunks of 64 tokens, bf16 inputs, on the tensor cores (tcgen05
// with TMEM accumulators, TMA loads).
//
// Per chunk of a (sequence, head, block of 128 value channels), G_i the decay's sum in log2 units up to and including
// row i, l the last row, s = 1/sqrt(K), S the incoming state:
//   A_ij = beta_i 2^(G_i - G_j) k_i . k_j  (j < i),   T = (1 + A)^-1 diag(beta)
//   U = T (V - diag(2^G) K S),   O = s diag(2^G) Q S + P U,   P_ij = s 2^(G_i - G_j) q_i . k_j  (j <= i)
//   S <- 2^G_l S + K^T diag(2^(G_l - G)) U
// The decay is a number per row, so q, k and v enter the products as they are, and every factor is one of a row of
// a result.  As products, with value channels (M = 128) on TMEM lanes:
//   scores [k; q] k^T (rows of k on lanes 0-63, of q on lanes 64-127);   Y^T = S^T k^T;   O1^T = S^T q^T;
//   U^T = R^T T^T with R = V - diag(2^G) Y;   O2^T = U^T P^T;   D^T = U'^T k with U' = diag(2^(G_l - G)) U, added to S^T.
// Row norms of q and k, where the call asks for them, are factors of rows as well.
//
// Roundings.  The state is a float32 output and feeds every later chunk: what leads to it has 24 bits.  S, R, T and
// U' are operands as three bf16 terms each (the products of R and T without the three smallest), a chunk's addition
// is summed by itself and added to S in rounded FP32, S is held in registers between chunks.  The output is bf16:
// O1 reads S's first term (its rounding to bf16), O2 is a tf32 product of U as it stands in TMEM (cut) and P.
//
// What is not finite must not reach back through masked zeros (0 times it is NaN).  A gate, beta or key: the rows from
// its token on are treated like rows behind the sequence, and the outputs from there on and the state are NaN.  A
// value: its place in R is cleared and noted (MARK), the channel's outputs from there on and its state are NaN.
//
// One CTA per unit and SM, 15 warps: 0-7 the chain (R, U' and S in turn, and the output while they wait for products),
// 8-11 the preparation of the next chunk (scores, inverse), 12 all products, 13 loads, 14 gates.  Every wait is
// bounded (a CTA that gives up lets its copies and MMAs finish, frees its TMEM and returns).  What happens rarely is
// out of line and loops are rolled: together the roles' loops have to fit the instruction caches.
#include "common.cuh"
#include "decay_gates.cuh"
#include "delta_gates.cuh"
#include "kda_internal.h"
#include "sm100.cuh"
#include "tile_ops.cuh"

namespace kda {
namespace delta {
namespace {

using namespace kda::decay;

__device__ unsigned int g_delta_timeouts = 0;

constexpr int C = 64, KD = 128, VB = 128, NTHR = 480, NKQ = 3, NV = 2, NG = 3, kRanked = 128;

// Barriers.  A phase's waiters see its parity alone: each barrier's next phase needs (through others) that all waiters of the
// last one have gone on.  Where that does not follow from the chain's order there is a barrier for each slot of the ring or parity.
enum { B_KQ = 0, B_V = B_KQ + NKQ, B_G = B_V + NV, B_F = B_G + NG, B_SC = B_F + 2, B_SCREAD, B_S = B_SCREAD + 2, B_Y, B_O1, B_R, B_T, B_U, B_UD, B_D,
       B_O2, B_O2READ, B_OFREE, B_KQFREE = B_OFREE + 2, B_VFREE = B_KQFREE + NKQ, B_GFREE = B_VFREE + NV, B_DRAIN = B_GFREE + NG, B_NEVER, NBAR };

// shared memory: stages of k and q (by 64 channels: 64 rows of k, then of q), of v; T's terms; P and, behind its reader,
// the staged output; the third term of R and U'; the matrix of the inverse
constexpr uint32_t KQ_BYTES = 32768, PANEL = 16384, QROWS = 8192, V_BYTES = 16384, T_TERM = 8192;
constexpr uint32_t L_KQ = 0, L_V = L_KQ + NKQ * KQ_BYTES, L_T = L_V + NV * V_BYTES, L_P = L_T + 3 * T_TERM, L_LO = L_P + 2 * 16384;
constexpr uint32_t L_X = L_LO + 16384, LDX = 68, L_G = L_X + 64 * LDX * 4;
// a chunk's factors, one slot of a ring of NG: byte offsets of its float arrays
constexpr uint32_t GT_G = 0;      // [64][2] G_i as integer and fraction
constexpr uint32_t GT_COL = 512;  // [64] 2^(G_m - G_j), m the last of j's 16 rows
constexpr uint32_t GT_ROW = 768;  // [64] s 2^G_i
constexpr uint32_t GT_KEY = 1024; // [64] -2^G_i / |k_i|
constexpr uint32_t GT_UPD = 1280; // [64] 2^(G_l - G_i) / |k_i|
constexpr uint32_t GT_BETA = 1536;
constexpr uint32_t GT_LAST = 1792;  // 2^G_l
constexpr uint32_t GT_LEN = 1796;   // rows that count: up to the sequence's end, or the first that is not finite
constexpr uint32_t GT_BYTES = 1808;
constexpr uint32_t L_RQ = L_G + NG * GT_BYTES;   // [2][64] 1 / |q_i|
constexpr uint32_t L_MARK = L_RQ + 2 * 256;      // [2][128] each channel's first row that is not finite, 64: none
constexpr uint32_t L_BAR = (L_MARK + 2 * 512 + 7) / 8 * 8, L_MISC = (L_BAR + 8 * NBAR + 15) / 16 * 16, L_END = L_MISC + 32;
constexpr uint32_t SMEM_BYTES = L_END + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of a block");
// TMEM columns: S's three terms; D, whose first half is O1's place; Y, then U; the first two terms of R, then of U'; scores, then O2
constexpr uint32_t TS = 0, TD = 192, TO1 = 192, TY = 320, TZ = 384, TSC = 448, TCOLS = 512;
// words of L_MISC
enum { M_TMEM = 0, M_UNUSED, M_ABORT, M_ODD, M_BAD0, M_BAD1 };  // M_ODD: bit (c & 1): marks of that chunk

struct Params {
    Gates gates;
    const float* h0;
    float* hT;
    const int32_t* cu;
    void* o;
    int N, T, H, hr, K, V;
    int vblocks;
    unsigned flags;
    int* status;
    int stall_chunk;
};

struct Sync {
    uint32_t bars;
    volatile uint32_t* abort_flag;
    int* status;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
    __device__ __forceinline__ void give_up() const {
        atomicAdd(&g_delta_timeouts, 1u);
        if (status) atomicOr(status, KDA_DEVICE_WAIT_GAVE_UP);
        *abort_flag = 1u;
    }
    // (out of line: one copy, so that the loops stay in the instruction caches)
    __device__ __noinline__ void slow_wait(int i, uint32_t parity, uint32_t limit) const {
        if (!*abort_flag && !mbar_wait_unless(bar(i), parity, abort_flag, limit)) give_up();
    }
    __device__ __forceinline__ bool aborted() const { return *abort_flag != 0u; }
    __device__ __forceinline__ bool stopped() const { return __any_sync(0xffffffffu, aborted()); }  // by a whole warp
    // A whole warp's wait.  After a wait that gave up all others return at once: the warps run through their loops
    // (their named barriers stay in step) on whatever is there, and nothing is stored.
    __device__ __forceinline__ void wait(int i, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return;
        slow_wait(i, parity, 1u << 22);
        __syncwarp();
    }
};

__device__ __forceinline__ uint32_t lo_kq_mn(uint32_t addr) { return (addr >> 4) | ((PANEL >> 4) << 16); }  // MN-major, panels of k
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t t, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(t));
}
// Both floats in three bf16 terms: the first two rounded, the third cut (what is left then has at most eight bits).
__device__ __forceinline__ uint32_t round2(float2& x) {
    const uint32_t r = pack_bf16(x.x, x.y);
    x = fma2(make_float2(bf_lo(r), bf_hi(r)), make_float2(-1.f, -1.f), x);
    return r;
}
__device__ __forceinline__ uint32_t top2(float2 x) { return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632); }
__device__ __forceinline__ float power(float2 a, float2 b) { return ex2_fast((a.x - b.x) + (a.y - b.y)); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// X <- (1 + X)^-1 in place, X strictly lower triangular, by 128 threads (named barrier 2).  The diagonal blocks of 16 by
// substitution, a warp a block and a column a lane, then twice the block below two inverted ones, -X22 (X21 X11).
__device__ __forceinline__ void invert(uint32_t X, int t) {
    const int w = t >> 5, l = t & 31;
    auto at = [&](int i, int c) { return X + 4u * (LDX * i + c); };
    {
        const int b = 16 * w, c = l & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == c ? 1.f : 0.f, y2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 a = lds4(at(b + i, b + m));
                y = fmaf(-a.x, x[m], y);
                if (m + 1 < i) y2 = fmaf(-a.y, x[m + 1], y2);
                if (m + 2 < i) y = fmaf(-a.z, x[m + 2], y);
                if (m + 3 < i) y2 = fmaf(-a.w, x[m + 3], y2);
            }
            x[i] = y + y2;  // (0 above the diagonal: all that comes before is)
        }
        __syncwarp();
        if (l < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) sts(at(b + i, b + c), x[i]);
    }
    bar_sync(2, 128);
    {   // 16 -> 32: two warps a pair, a row and four columns a thread
        const int o = 32 * (w >> 1), i = (t & 63) >> 2, c = 4 * (t & 3);
#pragma unroll 1
        for (int step = 0; step < 2; ++step) {  // X21 X11, then -X22 of that
            const uint32_t left = step ? at(o + 16 + i, o + 16) : at(o + 16 + i, o), right = step ? at(o + 16, o + c) : at(o, o + c);
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < 16; m += 4) {
                const float4 a = lds4(left + 4 * m);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 r = lds4(right + 4 * LDX * (m + e));
                    y[0] = fmaf(av[e], r.x, y[0]);
                    y[1] = fmaf(av[e], r.y, y[1]);
                    y[2] = fmaf(av[e], r.z, y[2]);
                    y[3] = fmaf(av[e], r.w, y[3]);
                }
            }
            bar_sync(2, 128);
            const float s = step ? -1.f : 1.f;
            sts2(at(o + 16 + i, o + c), s * y[0], s * y[1]);
            sts2(at(o + 16 + i, o + c + 2), s * y[2], s * y[3]);
            bar_sync(2, 128);
        }
    }
    {   // 32 -> 64: two rows and four columns a thread
        const int i = 2 * (t >> 3), c = 4 * (t & 7);
#pragma unroll 1
        for (int step = 0; step < 2; ++step) {
            const uint32_t left = step ? at(32 + i, 32) : at(32 + i, 0), right = step ? at(32, c) : at(0, c);
            float y[2][4] = {};
#pragma unroll 2
            for (int m = 0; m < 32; m += 4) {
                const float4 a = lds4(left + 4 * m), b = lds4(left + 4 * (LDX + m));
                const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 r = lds4(right + 4 * LDX * (m + e));
                    y[0][0] = fmaf(av[e], r.x, y[0][0]);
                    y[0][1] = fmaf(av[e], r.y, y[0][1]);
                    y[0][2] = fmaf(av[e], r.z, y[0][2]);
                    y[0][3] = fmaf(av[e], r.w, y[0][3]);
                    y[1][0] = fmaf(bv[e], r.x, y[1][0]);
                    y[1][1] = fmaf(bv[e], r.y, y[1][1]);
                    y[1][2] = fmaf(bv[e], r.z, y[1][2]);
                    y[1][3] = fmaf(bv[e], r.w, y[1][3]);
                }
            }
            bar_sync(2, 128);
            const float s = step ? -1.f : 1.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sts2(at(32 + i + r, c), s * y[r][0], s * y[r][1]);
                sts2(at(32 + i + r, c + 2), s * y[r][2], s * y[r][3]);
            }
            bar_sync(2, 128);
        }
    }
}

// |x|^2 of a row of a stage (one panel of 64 channels)
__device__ __forceinline__ float row_square(uint32_t panel, int row) {
    float s = 0.f;
#pragma unroll 1
    for (int p = 0; p < 8; ++p) {
        uint32_t v[4];
        ld_s128(panel + sw128(row, p), v);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(bf_lo(v[e]), bf_lo(v[e]), fmaf(bf_hi(v[e]), bf_hi(v[e]), s));
    }
    return s;
}

// 16 lanes x 32 columns, as ld16x32 has them
__device__ __forceinline__ void st16x32(uint32_t t, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
// Where a fragment of Y (or, vt = 0, of U) at t, of 16 channels from ch0 and 32 rows from row0, makes a place of R
// that is not finite, both Y and v are cleared there, and the channel's first such row is noted.  By one warp, out of
// line: it runs where something is wrong, if ever.
__device__ __noinline__ void clear_odd(uint32_t t, uint32_t vt, uint32_t key, int ch0, int row0, int len, uint32_t marks, volatile uint32_t* flag,
                                       uint32_t bit) {
    float a[16];
    ld16x32(t, a);
    tmem_wait_ld();
    const int l = threadIdx.x & 31;
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
        const int ch = ch0 + 8 * ((e >> 1) & 1) + (l >> 2), row = row0 + 8 * (e >> 2) + 2 * (l & 3) + (e & 1);
        const uint32_t at = vt + ((ch >> 6) & 1) * 8192u + sw128(row, (ch >> 3) & 7) + 2 * (ch & 7);
        const float r = vt ? fmaf(lds(key + 4 * row), a[e], __uint_as_float((uint32_t)lds16(at) << 16)) : a[e];
        if (finite(r) || row >= len) continue;
        a[e] = 0.f;
        if (vt) sts16(at, 0);
        asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(marks + 4 * ch), "r"(row) : "memory");
        atomicOr(const_cast<uint32_t*>(flag), bit);
    }
    __syncwarp();
    st16x32(t, a);
    tmem_wait_st();
}
// rows of a channel's staged output that are none
__device__ __noinline__ void nan_rows(uint32_t stage, uint32_t mark, int ch, int len, int rows) {
#pragma unroll 1
    for (int r = min(len, __float_as_int(lds(mark + 4 * ch))); r < rows; ++r)
        sts16(stage + (ch >> 6) * 8192u + sw128(r, (ch >> 3) & 7) + 2 * (ch & 7), 0x7FFF);
    sts(mark + 4 * ch, __int_as_float(C));
}

__global__ void __launch_bounds__(NTHR, 1)
delta_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L_MISC);
    const Sync sy{sb + L_BAR, misc + M_ABORT, p.status};
    auto gates = [&](int c) { return sb + L_G + (uint32_t)(c % NG) * GT_BYTES; };
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), l = tid & 31;

    // ---- the unit: heads fastest, then value blocks
    const int h = blockIdx.x, vb = blockIdx.y;
    int n = blockIdx.z;
    if (p.cu && p.N <= kRanked) {
        // The blocks start in order: the longest sequences first, so that none is left for the end
        int* ranked = reinterpret_cast<int*>(smem);
        if (tid < p.N) {
            const int mine = __ldg(p.cu + tid + 1) - __ldg(p.cu + tid);
            int rank = 0;
            for (int m = 0; m < p.N; ++m) {
                const int other = __ldg(p.cu + m + 1) - __ldg(p.cu + m);
                rank += other > mine || (other == mine && m < tid);
            }
            ranked[rank] = tid;
        }
        __syncthreads();
        n = ranked[blockIdx.z];
        fence_proxy_async_smem();  // (a stage's place)
        __syncthreads();
    }
    int bos, eos;
    if (p.cu) { bos = __ldg(p.cu + n); eos = __ldg(p.cu + n + 1); }
    else      { bos = n * p.T; eos = bos + p.T; }
    const int nt = __shfl_sync(0xffffffffu, (eos - bos + C - 1) / C, 0);
    const int hq = h / p.hr, vc0 = vb * VB;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int count = 1;
            if (i == B_S || i == B_R || i == B_UD || i == B_O2READ) count = 8;
            if ((i >= B_F && i < B_F + 2) || (i >= B_SCREAD && i < B_SCREAD + 2) || i == B_T) count = 4;
            mbar_init(sy.bar(i), count);
        }
        fence_mbar_init();
        misc[M_ABORT] = misc[M_ODD] = 0;
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_o);
    }
    for (int x = tid; x < 2 * VB; x += NTHR) sts(sb + L_MARK + 4 * x, __int_as_float(C));
    if (w == 12) tmem_alloc(sb + L_MISC + 4 * M_TMEM, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[M_TMEM], 0);
    auto arrive = [&](int bar) {
        __syncwarp();
        if (l == 0) mbar_arrive(sy.bar(bar));
    };

    if (w == 12) {
        // ------------------------------------------------ all products
        auto scores = [&](int c) {
            sy.wait(B_KQ + c % NKQ, (c / NKQ) & 1);
            tc_fence_after();
            if (!sy.stopped() && elect()) {
                const uint32_t a = lo_k(sb + L_KQ + (c % NKQ) * KQ_BYTES);
#pragma unroll
                for (int kk = 0; kk < KD / 16; ++kk) {
                    const uint32_t d = (kk >> 2) * (PANEL >> 4) + (kk & 3) * 2;
                    umma_bf16(tmem + TSC, desc(a + d), desc(a + d), idesc_bf16(128, 64, 0, 0), kk > 0);
                }
                umma_commit(sy.bar(B_SC));
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int c = -1; c < nt; ++c) {
            const uint32_t st = sb + L_KQ + ((c + NKQ) % NKQ) * KQ_BYTES;
            if (c >= 0) {
                if (c == p.stall_chunk) sy.slow_wait(B_NEVER, 0, 2000);
                sy.wait(B_S, c & 1);  // S's terms; D of the last chunk has been taken
                if (sy.stopped()) break;
                tc_fence_after();
                if (elect()) {
                    const uint32_t k = lo_k(st);
#pragma unroll
                    for (int t = 2; t >= 0; --t)
#pragma unroll
                        for (int kk = 0; kk < KD / 16; ++kk)
                            umma_bf16_ta(tmem + TY, tmem + TS + 64 * t + 8 * kk, desc(k + (kk >> 2) * (PANEL >> 4) + (kk & 3) * 2),
                                         idesc_bf16(128, 64, 0, 0), t < 2 || kk > 0);
                    umma_commit(sy.bar(B_Y));
                    const uint32_t q = lo_k(st + QROWS);
#pragma unroll
                    for (int kk = 0; kk < KD / 16; ++kk)
                        umma_bf16_ta(tmem + TO1, tmem + TS + 8 * kk, desc(q + (kk >> 2) * (PANEL >> 4) + (kk & 3) * 2),
                                     idesc_bf16(128, 64, 0, 0), kk > 0);
                    umma_commit(sy.bar(B_O1));
                }
                __syncwarp();
            }
            if (c + 1 < nt) {
                if (c > 0) sy.wait(B_O2READ, (c - 1) & 1);
                if (c == 0) sy.wait(B_SCREAD, 0);
                scores(c + 1);
            }
            if (c < 0) continue;
            sy.wait(B_T, c & 1);
            sy.wait(B_R, c & 1);
            if (sy.stopped()) break;
            tc_fence_after();
            if (elect()) {  // the smallest products first
                mbar_arrive(sy.bar(B_VFREE + c % NV));  // (v has been read into R, the last chunk's output has been formed)
                if (c > 0) mbar_arrive(sy.bar(B_GFREE + (c - 1) % NG));
                const uint32_t T = lo_k(sb + L_T), lo = lo_mn(sb + L_LO);
                bool more = false;
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int t = 0; t <= sum; ++t)  // term t of T, term sum - t of R
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t b = desc(T + t * (T_TERM >> 4) + kk * 2);
                            if (sum - t == 2) umma_bf16(tmem + TY, desc(lo + kk * 128), b, idesc_bf16(128, 64, 1, 0), more);
                            else umma_bf16_ta(tmem + TY, tmem + TZ + 32 * (sum - t) + 8 * kk, b, idesc_bf16(128, 64, 0, 0), more);
                            more = true;
                        }
                umma_commit(sy.bar(B_U));
            }
            __syncwarp();
            sy.wait(B_UD, c & 1);  // (and O1, scaled, lies in O2's place)
            if (sy.stopped()) break;
            tc_fence_after();
            if (elect()) {
                const uint32_t k = lo_kq_mn(st), lo = lo_mn(sb + L_LO), P = lo_k(sb + L_P + (c & 1) * 16384);
#pragma unroll
                for (int t = 2; t >= 0; --t)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (t == 2) umma_bf16(tmem + TD, desc(lo + kk * 128), desc(k + kk * 128), idesc_bf16(128, KD, 1, 1), kk > 0);
                        else umma_bf16_ta(tmem + TD, tmem + TZ + 32 * t + 8 * kk, desc(k + kk * 128), idesc_bf16(128, KD, 0, 1), 1);
                    }
                umma_commit(sy.bar(B_D));
                umma_commit(sy.bar(B_KQFREE + c % NKQ));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_tf32_ta(tmem + TSC, tmem + TY + 8 * kk, desc(P + (kk >> 2) * 512 + (kk & 3) * 2), idesc_tf32(128, 64), 1);
                umma_commit(sy.bar(B_O2));
            }
            __syncwarp();
        }
        if (sy.stopped()) {  // leave no MMA in flight behind
            if (elect()) {
                umma_commit(sy.bar(B_DRAIN));
                mbar_wait(sy.bar(B_DRAIN), 0);
            }
            __syncwarp();
        }
    } else if (w == 13) {
        // ------------------------------------------------ loads
        int c = 0;
#pragma unroll 1
        for (; c < nt; ++c) {
            if (c >= NKQ) sy.wait(B_KQFREE + c % NKQ, (c / NKQ - 1) & 1);
            if (c >= NV) sy.wait(B_VFREE + c % NV, (c / NV - 1) & 1);
            if (sy.stopped()) break;
            if (elect()) {
                const uint32_t v = sb + L_V + (c % NV) * V_BYTES, kq = sb + L_KQ + (c % NKQ) * KQ_BYTES;
                const uint32_t fv = sy.bar(B_V + c % NV), fkq = sy.bar(B_KQ + c % NKQ);
                mbar_arrive_expect_tx(fkq, KQ_BYTES);
#pragma unroll
                for (int x = 0; x < KD / 64; ++x) {
                    tma_load_3d(kq + x * PANEL, &tm_k, 64 * x, hq, bos + c * C, fkq);
                    tma_load_3d(kq + x * PANEL + QROWS, &tm_q, 64 * x, hq, bos + c * C, fkq);
                }
                mbar_arrive_expect_tx(fv, V_BYTES);
#pragma unroll
                for (int x = 0; x < VB / 64; ++x) tma_load_3d(v + x * 8192, &tm_v, vc0 + 64 * x, h, bos + c * C, fv);
            }
            __syncwarp();
        }
        if (sy.stopped()) {  // leave no copy in flight behind
            if (elect()) {
                for (int x = max(0, c - NKQ); x < c; ++x) mbar_wait(sy.bar(B_KQ + x % NKQ), (x / NKQ) & 1);
                for (int x = max(0, c - NV); x < c; ++x) mbar_wait(sy.bar(B_V + x % NV), (x / NV) & 1);
            }
            __syncwarp();
        }
    } else if (w == 14) {
        // ------------------------------------------------ gates: a chunk's decays and rates, two tokens a lane
        const Gates::Head head = p.gates.head(h);
        const float scale = rsqrtf((float)p.K);
        float ra[2], rb[2];  // as they lie in memory, asked for a chunk before they are used
        auto ask = [&](int c) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = bos + c * C + 2 * l + e;
                ra[e] = t < eos ? p.gates.raw_decay(t, h) : 0.f;
                rb[e] = t < eos ? p.gates.raw_rate(t, h) : 0.f;
            }
        };
        if (nt > 0) ask(0);
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const uint32_t gt = gates(c);
            const int left = eos - (bos + c * C);
            float a[2], b[2];
            bool ok[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a[e] = 2 * l + e < left ? p.gates.decay_of(ra[e], head) : 0.f;
                b[e] = 2 * l + e < left ? p.gates.rate_of(rb[e]) : 0.f;
            }
            if (c + 1 < nt) ask(c + 1);
            const float none = __int_as_float(0x7fffffff);
            ok[0] = a[0] < 3e38f && finite(b[0]);
            ok[1] = a[1] < 3e38f && finite(b[1]);
            const int bad = first_nan(ok[0] ? 0.f : none, ok[1] ? 0.f : none);
            int I[2], F[2];
            long long G[2];
            pair_sums(a[0], a[1], G);
            parts(G[0], I[0], F[0]);
            parts(G[1], I[1], F[1]);
            const int Il = __shfl_sync(0xffffffffu, I[1], 31), Fl = __shfl_sync(0xffffffffu, F[1], 31);
            const int Im = __shfl_sync(0xffffffffu, I[1], l | 7), Fm = __shfl_sync(0xffffffffu, F[1], l | 7);
            if (c >= NG) sy.wait(B_GFREE + c % NG, (c / NG - 1) & 1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * l + e;
                sts2(gt + GT_G + 8 * i, (float)I[e], (float)F[e] * (1.f / 16777216.f));
                const float r = pow2(I[e], F[e]);
                sts(gt + GT_ROW + 4 * i, scale * r);
                sts(gt + GT_KEY + 4 * i, -r);
                sts(gt + GT_UPD + 4 * i, i < bad ? pow2(Il - I[e], Fl - F[e]) : 0.f);
                sts(gt + GT_COL + 4 * i, pow2_fast(Im - I[e], Fm - F[e]));
                sts(gt + GT_BETA + 4 * i, i < bad ? b[e] : 0.f);
            }
            if (l == 0) {
                sts(gt + GT_LAST, pow2(Il, Fl));
                sts(gt + GT_LEN, __int_as_float(min(bad, left)));
            }
            arrive(B_G + c % NG);
        }
    } else if (w < 8) {
        // ------------------------------------------------ the chain: R, U' and S, value channels on lanes; the output
        const int qd = w & 3, half = w >> 2;
        const uint32_t lane = (uint32_t)(32 * qd) << 16;
        const int vl = 32 * qd + l;
        const bool mine = vc0 + vl < p.V;
        const int rows = min(64, p.K - 64 * half);  // of this warp's 64 key channels
        float S[64];
        {
            const float* from = p.h0 + ((size_t)n * p.H + h) * (size_t)p.K * p.V + (size_t)(64 * half) * p.V + vc0 + vl;
#pragma unroll
            for (int j = 0; j < 64; ++j, from += p.V) S[j] = p.h0 && mine && j < rows ? *from : 0.f;
        }
        // a lane's row of the four 8 x 8 blocks of a fragment load: channels + 0, + 8, rows + 0, + 8
        const int lrow = 32 * half + (l & 7) + ((l >> 4) << 3), lpiece = 4 * (qd & 1) + ((l >> 3) & 1);
        const uint32_t lo = sb + L_LO + (qd >> 1) * 8192u;
        const uint32_t zcol = tmem + TZ + lane + 16 * half, ycol = tmem + TY + lane + 32 * half;
        const int pair = 4 * (32 * half + 2 * (l & 3));  // byte offset of a lane's first two rows' factors
        // the terms of sixteen channels' fragments (x[2 G + 0 / 1]: rows 8 G + 2 (l % 4) of channels l / 4 / + 8)
        auto write_fragments = [&](int y, float2 (&x)[8]) {
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = round2(x[e]);
            st16x16(zcol + ((uint32_t)(16 * y) << 16), r);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = round2(x[e]);
            st16x16(zcol + ((uint32_t)(16 * y) << 16) + 32, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = top2(x[e]);
#pragma unroll
            for (int g = 0; g < 4; g += 2) stmatrix4_t(lo + sw128(lrow + 8 * g, lpiece + 2 * y), r + 2 * g);
        };
        auto marked = [&](int c) { return ((misc[M_ODD] >> (c & 1)) & 1u) != 0u; };
        const float2 zero = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0;; ++c) {
            // ---- S behind chunk c - 1, its terms for chunk c
            float last = 1.f;
            if (c > 0) {
                last = lds(gates(c - 1) + GT_LAST);
                if (marked(c - 1)) last += nan_if(__float_as_int(lds(sb + L_MARK + 512 * ((c - 1) & 1) + 4 * vl)) < C);
                sy.wait(B_D, (c - 1) & 1);
                tc_fence_after();
            }
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                if (c > 0) {
                    float d[16];
                    tmem_ld16(tmem + TD + lane + 64 * half + x, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 s = fma2(make_float2(last, last), make_float2(S[x + j], S[x + j + 1]), make_float2(d[j], d[j + 1]));
                        S[x + j] = s.x;
                        S[x + j + 1] = s.y;
                    }
                }
                uint32_t t0[8], t1[8], t2[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2 y = make_float2(S[x + 2 * j], S[x + 2 * j + 1]);
                    t0[j] = round2(y);
                    t1[j] = round2(y);
                    t2[j] = top2(y);
                }
                const uint32_t at = tmem + TS + lane + 32 * half + x / 2;
                tmem_st8(at, t0);
                tmem_st8(at + 64, t1);
                tmem_st8(at + 128, t2);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(B_S);
            if (c > 0) {
                // ---- chunk c - 1's output, through P's place
                const int b = (c - 1) & 1, t0 = bos + (c - 1) * C, n_rows = min(C, eos - t0);
                const uint32_t rq = sb + L_RQ + 256 * b, stage = sb + L_P + b * 16384;
                const int len = __float_as_int(lds(gates(c - 1) + GT_LEN));
                sy.wait(B_O2, b);
                tc_fence_after();
#pragma unroll 1
                for (int y = 0; y < 2; ++y) {
                    float o[16];
                    ld16x32(tmem + TSC + lane + ((uint32_t)(16 * y) << 16) + 32 * half, o);
                    tmem_wait_ld();
                    uint32_t r[8];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 m = lds2(rq + pair + 32 * g);
                        const float2 y0 = mul2(m, make_float2(o[4 * g], o[4 * g + 1])), y1 = mul2(m, make_float2(o[4 * g + 2], o[4 * g + 3]));
                        r[2 * g] = pack_bf16(y0.x, y0.y);
                        r[2 * g + 1] = pack_bf16(y1.x, y1.y);
                    }
#pragma unroll
                    for (int g = 0; g < 4; g += 2) stmatrix4_t(stage + (qd >> 1) * 8192u + sw128(lrow + 8 * g, lpiece + 2 * y), r + 2 * g);
                }
                tc_fence_before();
                arrive(B_O2READ);
                const bool odd = len < n_rows || marked(c - 1);
                if (odd) {
                    bar_sync(1, 256);  // (a channel's rows are two warps')
                    if (half == 0) nan_rows(stage, sb + L_MARK + 512 * b, vl, len, n_rows);
                }
                fence_proxy_async_smem();
                bar_sync(1, 256);
                if (odd && tid == 0) atomicAnd(const_cast<uint32_t*>(misc + M_ODD), ~(1u << b));
                if (!sy.stopped()) {
                    if (n_rows == C) {
                        if (tid == 0) {
#pragma unroll
                            for (int x = 0; x < VB / 64; ++x)
                                if (vc0 + 64 * x < p.V) tma_store_3d(&tm_o, stage + x * 8192, vc0 + 64 * x, h, t0);
                            bulk_commit();
                        }
                    } else {  // the sequence's last rows
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((size_t)t0 * p.H + h) * p.V + vc0;
#pragma unroll 1
                        for (int x = tid; x < n_rows * (VB / 8); x += 256) {
                            const int row = x / (VB / 8), ch = x % (VB / 8);
                            uint32_t v[4];
                            ld_s128(stage + (ch >> 3) * 8192u + sw128(row, ch & 7), v);
                            if (vc0 + 8 * ch < p.V) *reinterpret_cast<uint4*>(dst + (size_t)row * p.H * p.V + 8 * ch) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
            }
            if (c == nt) break;
            // ---- R
            const uint32_t gt = gates(c), vt = sb + L_V + (c % NV) * V_BYTES;
            sy.wait(B_F + (c & 1), (c >> 1) & 1);
            sy.wait(B_V + c % NV, (c / NV) & 1);
            const int len = __float_as_int(lds(gt + GT_LEN));
            sy.wait(B_Y, c & 1);
            tc_fence_after();
            if (len < C) {  // rows that do not count, for D
                const uint32_t kt = sb + L_KQ + (c % NKQ) * KQ_BYTES;
#pragma unroll 1
                for (int x = tid; x < C * (KD / 8); x += 256)
                    if ((x & 63) >= len) st_s128(kt + (x >> 9) * PANEL + sw128(x & 63, (x >> 6) & 7), 0, 0, 0, 0);
            }
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
                float2 x[8];
                const uint32_t at = ycol + ((uint32_t)(16 * y) << 16);
#pragma unroll 1
                for (int again = 0; again < 2; ++again) {
                    float a[16];
                    float2 odd = zero;
                    uint32_t r[8];
                    ld16x32(at, a);
                    ldmatrix4_t(vt + (qd >> 1) * 8192u + sw128(lrow, lpiece + 2 * y), r);
                    ldmatrix4_t(vt + (qd >> 1) * 8192u + sw128(lrow + 16, lpiece + 2 * y), r + 4);
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 f = lds2(gt + GT_KEY + pair + 32 * g);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = 2 * g + e;
                            x[i] = fma2(f, make_float2(a[4 * g + 2 * e], a[4 * g + 2 * e + 1]), make_float2(bf_lo(r[i]), bf_hi(r[i])));
                        }
                    }
                    if (len < C) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int j = 32 * half + 8 * (e >> 1) + 2 * (l & 3);
                            if (j >= len) x[e].x = 0.f;
                            if (j + 1 >= len) x[e].y = 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) odd = fma2(x[e], zero, odd);
                    if (!__any_sync(0xffffffffu, odd.x != 0.f || odd.y != 0.f)) break;
                    clear_odd(at, vt, gt + GT_KEY, 32 * qd + 16 * y, 32 * half, len, sb + L_MARK + 512 * (c & 1), misc + M_ODD, 1u << (c & 1));
                }
                write_fragments(y, x);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(B_R);
            if (c > 0 && tid == 0) {  // the staged output has left
                bulk_wait_read();
                mbar_arrive(sy.bar(B_OFREE + ((c - 1) & 1)));
            }
            __syncwarp();
            // ---- O1 with its rows' factors, where O2 will be added to it
            if (c == 0) sy.wait(B_SCREAD, 0);
            if (c + 1 < nt) sy.wait(B_SCREAD + ((c + 1) & 1), ((c + 1) >> 1) & 1);
            sy.wait(B_O1, c & 1);
            tc_fence_after();
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
                float o[16];
                const uint32_t at = tmem + lane + ((uint32_t)(16 * y) << 16) + 32 * half;
                ld16x32(at + TO1, o);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 f = lds2(gt + GT_ROW + pair + 32 * g);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 s = mul2(f, make_float2(o[4 * g + 2 * e], o[4 * g + 2 * e + 1]));
                        o[4 * g + 2 * e] = s.x;
                        o[4 * g + 2 * e + 1] = s.y;
                    }
                }
                st16x32(at + TSC, o);
            }
            // ---- U'
            sy.wait(B_U, c & 1);
            tc_fence_after();
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
                float a[16];
                float2 x[8], odd = zero;
                const uint32_t at = ycol + ((uint32_t)(16 * y) << 16);
                ld16x32(at, a);
                tmem_wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 f = lds2(gt + GT_UPD + pair + 32 * g);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 u = make_float2(a[4 * g + 2 * e], a[4 * g + 2 * e + 1]);
                        odd = fma2(u, zero, odd);
                        x[2 * g + e] = mul2(f, u);
                    }
                }
                // (U itself is O2's operand)
                if (__any_sync(0xffffffffu, odd.x != 0.f || odd.y != 0.f))
                    clear_odd(at, 0, 0, 32 * qd + 16 * y, 32 * half, C, sb + L_MARK + 512 * (c & 1), misc + M_ODD, 1u << (c & 1));
                write_fragments(y, x);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(B_UD);
        }
        if (tid == 0) bulk_wait();
        if (p.hT && mine && !sy.aborted()) {
            float* to = p.hT + ((size_t)n * p.H + h) * (size_t)p.K * p.V + (size_t)(64 * half) * p.V + vc0 + vl;
#pragma unroll
            for (int j = 0; j < 64; ++j, to += p.V)
                if (j < rows) *to = S[j];
        }
    } else if (w < 12) {
        // ------------------------------------------------ preparation: T and P of a chunk
        const int t = tid - 256, i = t & 63;
        const bool query = t >= 64, hi = (t & 32) != 0;
        const uint32_t sc = tmem + TSC + ((uint32_t)(32 * (w & 3)) << 16), X = sb + L_X;
        const float scale = rsqrtf((float)p.K);
        const bool qnorm = (p.flags & KDA_FLAG_Q_L2NORM) != 0, knorm = (p.flags & KDA_FLAG_K_L2NORM) != 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const uint32_t gt = gates(c);
            sy.wait(B_G + c % NG, (c / NG) & 1);
            sy.wait(B_SC, c & 1);
            tc_fence_after();
            // keys that are not finite (their square), and the rows' norms
            if (!query) {
                float x[32], kk = 0.f;
                ld32(sc + (hi ? 32 : 0), x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) kk = j == l ? x[j] : kk;
                const unsigned odd = __ballot_sync(0xffffffffu, !finite(kk) && i < __float_as_int(lds(gt + GT_LEN)));
                if (l == 0) misc[M_BAD0 + (hi ? 1 : 0)] = odd ? (hi ? 32 : 0) + __ffs(odd) - 1 : C;
                sts(X + 4 * (LDX * i + 64), knorm && finite(kk) ? rsqrtf(kk + kQNormEps) : 1.f);
            } else {
                float s = 0.f;
                if (qnorm) {
                    const uint32_t q = sb + L_KQ + (c % NKQ) * KQ_BYTES + QROWS;
#pragma unroll 1
                    for (int x = 0; x < KD / 64; ++x) s += row_square(q + x * PANEL, i);
                }
                sts(sb + L_RQ + 256 * (c & 1) + 4 * i, qnorm ? rsqrtf(s + kQNormEps) : 1.f);
            }
            bar_sync(2, 128);
            const int full = __float_as_int(lds(gt + GT_LEN)), len = min(full, (int)min(misc[M_BAD0], misc[M_BAD1]));
            const float rk = lds(X + 4 * (LDX * i + 64));
            bar_sync(2, 128);
            if (!query) {
                if (knorm || len < full) {
                    sts(gt + GT_KEY + 4 * i, rk * lds(gt + GT_KEY + 4 * i));
                    sts(gt + GT_UPD + 4 * i, i < len ? rk * lds(gt + GT_UPD + 4 * i) : 0.f);
                    if (i >= len) sts(gt + GT_BETA + 4 * i, 0.f);
                }
                if (i == 0) {
                    sts(gt + GT_LEN, __int_as_float(len));
                    if (len < min(C, eos - (bos + c * C))) sts(gt + GT_LAST, __int_as_float(0x7fffffff));
                }
            }
            arrive(B_F + (c & 1));
            if (c >= 2) sy.wait(B_OFREE + (c & 1), ((c - 2) >> 1) & 1);  // P's place
            // A's rows (lanes with keys) into X, P's rows (with queries) as a tf32 operand: the score times
            // f 2^(G_i - G_j), 0 where j > last.  Left of the row's 32 the factor parts into the row's and the column's,
            // both <= 1; within them each is formed by itself.
            const int last = i < len ? i - (query ? 0 : 1) : -1;
            const float f = query ? scale : lds(gt + GT_BETA + 4 * i) * rk;
            const float2 gi = lds2(gt + GT_G + 8 * i);
#pragma unroll 1
            for (int b = 0; b < 8; ++b) {  // eight columns each
                float x[8];
                if (b < (hi ? 8 : 4)) {
                    tmem_ld8(sc + 8 * b, x);
                    tmem_wait_ld();
                    if (hi && b < 4) {
                        const float r = last < 0 ? 0.f : f * power(gi, lds2(gt + GT_G + 8 * (8 * b | 15)));
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            const float4 m = lds4(gt + GT_COL + 4 * (8 * b + j));
                            x[j] = last < 0 ? 0.f : x[j] * (r * m.x);
                            x[j + 1] = last < 0 ? 0.f : x[j + 1] * (r * m.y);
                            x[j + 2] = last < 0 ? 0.f : x[j + 2] * (r * m.z);
                            x[j + 3] = last < 0 ? 0.f : x[j + 3] * (r * m.w);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const float4 g = lds4(gt + GT_G + 8 * (8 * b + j));
                            x[j] = 8 * b + j <= last ? x[j] * f * power(gi, make_float2(g.x, g.y)) : 0.f;
                            x[j + 1] = 8 * b + j + 1 <= last ? x[j + 1] * f * power(gi, make_float2(g.z, g.w)) : 0.f;
                        }
                    }
                    if (knorm)
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= lds(X + 4 * (LDX * (8 * b + j) + 64));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = 0.f;
                }
                const uint32_t to = query ? sb + L_P + (c & 1) * 16384 + (b >> 2) * 8192 : X + 4 * (LDX * i + 8 * b);
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = query ? to_tf32(x[j + e]) : __float_as_uint(x[j + e]);
                    st_s128(query ? to + sw128(i, 2 * (b & 3) + j / 4) : to + 4 * j, v[0], v[1], v[2], v[3]);
                }
            }
            tc_fence_before();
            arrive(B_SCREAD + (c & 1));
            bar_sync(2, 128);
            invert(X, t);
            // T's terms: a row and 32 columns a thread
            if (c > 0) sy.wait(B_U, (c - 1) & 1);  // their last reader
            const int r = t >> 1, c0 = 32 * (t & 1);
#pragma unroll 1
            for (int x = 0; x < 32; x += 8) {
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 y = lds4(X + 4 * (LDX * r + c0 + x + 4 * e)), m = lds4(gt + GT_BETA + 4 * (c0 + x + 4 * e));
                    float2 y0 = mul2(make_float2(y.x, y.y), make_float2(m.x, m.y)), y1 = mul2(make_float2(y.z, y.w), make_float2(m.z, m.w));
                    t0[2 * e] = round2(y0);
                    t0[2 * e + 1] = round2(y1);
                    t1[2 * e] = round2(y0);
                    t1[2 * e + 1] = round2(y1);
                    t2[2 * e] = top2(y0);
                    t2[2 * e + 1] = top2(y1);
                }
                const uint32_t at = sb + L_T + sw128(r, (c0 + x) / 8);
                st_s128(at, t0[0], t0[1], t0[2], t0[3]);
                st_s128(at + T_TERM, t1[0], t1[1], t1[2], t1[3]);
                st_s128(at + 2 * T_TERM, t2[0], t2[1], t2[2], t2[3]);
            }
            fence_proxy_async_smem();
            arrive(B_T);
            bar_sync(2, 128);  // (X has been read)
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

}  // namespace
}  // namespace delta

// bf16, K up to 128 and a multiple of 8, V a multiple of 8 (a row of each begins 16-byte aligned, as TMA wants it)
bool delta_tensor_dims(bool bf16, int K, int V) { return bf16 && K % 8 == 0 && K <= 128 && V % 8 == 0; }

cudaError_t launch_delta_tensor(const DeltaArgs& a) {
    using namespace delta;
    CUtensorMap m[4];  // q, k, v, o
    const long tokens = (long)a.B * a.T;
    if (tokens == 0 && !a.hT) return cudaSuccess;
    const void* some = a.hT;  // nothing to load: the maps are never used
    if (!make_map(m, tokens ? a.q : some, tokens ? tokens : 1, a.Hk, a.K) ||
        !make_map(m + 1, tokens ? a.k : some, tokens ? tokens : 1, a.Hk, a.K) ||
        !make_map(m + 2, tokens ? a.v : some, tokens ? tokens : 1, a.H, a.V) ||
        !make_map(m + 3, tokens ? a.o : some, tokens ? tokens : 1, a.H, a.V))
        return cudaErrorInvalidValue;
    const int vblocks = (a.V + VB - 1) / VB;
    const Params p{Gates(a), a.h0, a.hT, a.cu, a.o, a.N, a.T, a.H, a.H / a.Hk, a.K, a.V, vblocks, a.flags, a.status, hook_stall_chunk()};
    const cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    delta_chunk_kernel<<<dim3(a.H, vblocks, a.N), NTHR, SMEM_BYTES, a.stream>>>(m[0], m[1], m[2], m[3], p);
    return cudaGetLastError();
}

cudaError_t read_delta_timeouts(unsigned* count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, delta::g_delta_timeouts, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(delta::g_delta_timeouts, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace kda
