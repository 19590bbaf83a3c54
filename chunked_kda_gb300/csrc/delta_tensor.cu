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
// Roundings.  The state is a float32 output and feeds every later chunk: its operands have 24 bits.  S, R, T and
// U' are operands as three bf16 terms each (the products of R and T without the three smallest), a chunk's addition
// is summed by itself and added to S in rounded FP32, S is held in registers between chunks.  The factors 2^(G_i - G_j) of A
// and P are the hardware's powers (2^-22).  The output is bf16, and its operands have 16 bits, 2^-16 of each term: O1 reads
// S's first two terms (with the first alone an output was off by up to 1.4 times its own rounding, and no call was faster),
// O2 is formed of U's and P's first two, without the product of the second ones.  (U cut to tf32's 11 bits as it stood in
// TMEM and P rounded to them: 606 us in place of 620 for 4 x 4096 tokens, 64 heads, and the chunk's part of an output
// too small by 3.5e-4 on average, up to 2^-10 of its terms.)
//
// What is not finite must not reach back through masked zeros (0 times it is NaN).  A gate, beta or key: the rows from
// its token on are treated like rows behind the sequence, and the outputs from there on and the state are NaN.  A
// value: its place in R is cleared and noted (MARK), the channel's outputs from there on and its state are NaN.  Places of R and U
// that are finite, but too large for a bf16 term (from 3.3953e38 on), are treated the same.
//
// One CTA per unit and SM, 27 warps: 0-15 the chain (R, U' and S in turn, and the output while they wait for products),
// 16-23 the preparation of the next chunk (scores, inverse), 24 all products, 25 loads, 26 gates.  Every wait is
// bounded (a CTA that gives up lets its copies and MMAs finish, frees its TMEM and returns).  What happens rarely is
// out of line and loops are rolled: together the roles' loops have to fit the instruction caches.
// Dense calls whose units do not fill the SMs evenly are cut: an SM has the same number of chunks, and a unit's second
// part takes the state over through scratch.
//
// Times of a call, heads of 128 x 128: 4 x 4096 tokens, 64 heads 620 us (in FP32 without tensor cores 6.4 ms);
// 4096 tokens, 152 heads 358; 8192 tokens, 96 heads 687; 20480 tokens, 32 heads 1690, and as much with 4 (a unit has one
// SM).  The bytes alone are 160 us of the first.  A chunk is about 10,800 clocks of an SM.  With one term each of U and P, when
// it was 10,000, the chain (S 1350, O 1600, R 2200, U 700 and its wait, U' 1200, D 1300) and the preparation (scores
// 3300, inverse 4300, T 1200) were as long as one another, and the second terms are work of both.
// No pipe is full: the chain's order bounds it, with shared memory (ordinary loads and stores 50 % of its wavefronts, the
// tensor cores' operands beside them), issue slots (60 %) and instruction fetches, which 27 warps of six kinds share.
// The tensor cores are at 31 %, HBM at 20 %.  Tried and slower: the inverse on tensor cores (mma of tf32: 3530 clocks
// against 3130 alone), polls with a time hint, outputs stored without staging, one barrier for several roles' waits.
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

constexpr int KD = 128, VB = 128, NTHR = 864, NCH = 512, NPREP = 256, NKQ = 3, NP = 3, NG = 3, kRanked = 128;

// Barriers.  A phase's waiters see its parity alone: each barrier's next phase needs (through others) that all waiters of the
// last one have gone on.  Where that does not follow from the chain's order there is a barrier for each slot of the ring or parity.
enum { B_KQ = 0, B_V = B_KQ + NKQ, B_G, B_F = B_G + NG, B_SC = B_F + 2, B_SCREAD, B_S = B_SCREAD + 2, B_Y, B_O1, B_R, B_T, B_U, B_UD, B_D,
       B_O2, B_O2READ, B_OFREE, B_KQFREE = B_OFREE + NP, B_VFREE = B_KQFREE + NKQ, B_GFREE, B_DRAIN = B_GFREE + NG, B_NEVER, NBAR };

// shared memory: stages of k and q (by 64 channels: 64 rows of k, then of q), of v; T's terms; P and, behind its reader, the
// staged output; the third term of R and U'; the matrix of the inverse
constexpr uint32_t KQ_BYTES = 32768, PANEL = 16384, QROWS = 8192, V_BYTES = 16384, T_TERM = 8192, P_TERM = 8192;
constexpr uint32_t L_KQ = 0, L_V = L_KQ + NKQ * KQ_BYTES, L_T = L_V + V_BYTES, L_P = L_T + 3 * T_TERM, L_LO = L_P + NP * 16384;
constexpr uint32_t L_X = L_LO + 16384, LDX = 68, L_G = L_X + 64 * LDX * 4;
// a chunk's factors, one slot of a ring of NG: byte offsets of its float arrays
constexpr uint32_t GT_G = 0;      // [2][64] -G_i as integer and fraction
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
constexpr uint32_t SMEM_BYTES = L_END;
static_assert(SMEM_BYTES <= 232448, "shared memory of a block");
// TMEM columns: S's three terms; D, whose first half is O1's place; Y, then U; the first two terms of R, then of U'; scores, then O2
constexpr uint32_t TS = 0, TD = 192, TO1 = 192, TY = 320, TZ = 384, TSC = 448, TCOLS = 512;
// words of L_MISC
enum { M_TMEM = 0, M_ABORT, M_ODD, M_BAD };  // M_ODD: bit (c & 1): marks of that chunk

struct Params {
    Gates gates;
    const float* h0;
    float* hT;
    const int32_t* cu;
    void* o;
    int N, T, H, hr, K, V;
    int vblocks;
    unsigned flags;
    float* ws;       // cut units' states [unit of a sequence and head][K][V]
    unsigned* cuts;  // cut units: a ticket, then a counter for each unit (all zero); else null
    int per;         // chunks of an SM with cut units
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
    // One poll, which may sleep until the phase completes.  Without a time hint it is one instruction; with one it
    // is a loop of its own, and the polls of waiting warps were half of all instructions.
    static __device__ __forceinline__ bool come(uint32_t bar, uint32_t parity) {
        uint32_t ok;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        return ok != 0;
    }
    // Out of line: one copy, so that the roles' loops fit the instruction caches.  Gives up after about four seconds.
    static __device__ __noinline__ void wait_out(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int* status) {
        if (__all_sync(0xffffffffu, come(bar, parity))) return;
        slow_wait(bar, parity, abort_flag, status, 8000000000ll);
        __syncwarp();
    }
    static __device__ __forceinline__ void slow_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int* status, long long limit) {
        const long long begin = clock64();
#pragma unroll 1
        while (!*abort_flag) {
            // (short: what waiting warps execute, the working ones cannot)
#pragma unroll 1
            for (int n = 0; n < 64; ++n)
                if (come(bar, parity)) return;
            if (clock64() - begin > limit) Sync{0, abort_flag, status}.give_up();
        }
    }
    __device__ __forceinline__ bool aborted() const { return *abort_flag != 0u; }
    __device__ __forceinline__ bool stopped() const { return __any_sync(0xffffffffu, aborted()); }  // by a whole warp
    // A whole warp's wait.  After a wait that gave up all others return at once: the warps run through their loops
    // (their named barriers stay in step) on whatever is there, and nothing is stored.
    __device__ __forceinline__ void wait(int i, uint32_t parity) const { wait_out(bars + 8u * i, parity, abort_flag, status); }
};

__device__ __forceinline__ uint32_t lo_kq_mn(uint32_t addr) { return (addr >> 4) | ((PANEL >> 4) << 16); }  // MN-major, panels of k
__device__ __forceinline__ void tmem_st4(uint32_t t, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t t, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(t));
}
// 16 lanes x 8 columns: of each four columns, thread t has column t % 4 of lanes t / 4 and t / 4 + 8
__device__ __forceinline__ void st16x8(uint32_t t, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// 16 lanes x 16 columns, as ld16x16 has them
__device__ __forceinline__ void st16x16f(uint32_t t, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// Both floats in three bf16 terms: the first two rounded, the third cut (what is left then has at most eight bits).
// The remainder is formed by the multiply-add that takes bf16 as it lies in a half of a register: 4.6 clocks a pair, term
// and scheduler, against 6.6 with the halves unpacked and 8.6 with bits masked off (shifts and masks have half the rate).
__device__ __forceinline__ uint32_t round2(float2& x) {
    const uint32_t r = pack_bf16(x.x, x.y);
    asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %4;\n mov.b16 m, 0xBF80;\n"  // -1
        " fma.rn.f32.bf16 %0, l, m, %2;\n fma.rn.f32.bf16 %1, h, m, %3;\n}\n"
        : "=f"(x.x), "=f"(x.y)
        : "f"(x.x), "f"(x.y), "r"(r));
    return r;
}
// a + the pair of bf16 numbers in r
__device__ __forceinline__ float2 add_bf16(uint32_t r, float2 a) {
    float2 d;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %4;\n add.f32.bf16 %0, l, %2;\n add.f32.bf16 %1, h, %3;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "r"(r));
    return d;
}
__device__ __forceinline__ uint32_t top2(float2 x) { return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}\n" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void sts_pair(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }
// ... and not beyond what is rounded to bf16's largest number, so that its first term is finite
__device__ __forceinline__ bool term_finite(float x) { return (__float_as_uint(x) & 0x7fffffffu) < 0x7F7F8000u; }

// X <- (1 + X)^-1 in place, X strictly lower triangular, by 256 threads (named barrier 2).  The diagonal blocks of 16 by
// substitution, a warp a block and a column a lane, then twice the block below two inverted ones, -X22 (X21 X11).  Columns of
// that are independent of one another: a warp forms both products for its own, so that the warps meet only before and
// after the block is replaced.  The block right of the diagonal's blocks of 32 is scratch (nobody reads it as part of X).
__device__ __forceinline__ void invert(uint32_t X, int t) {
    const int w = t >> 5, l = t & 31;
    auto at = [&](int i, int c) { return X + 4u * (LDX * i + c); };
    if (w < 4) {
        const uint32_t b = at(16 * w, 16 * w);
        const int c = l & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == c ? 1.f : 0.f, y2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 a = lds4(b + 4 * (LDX * i + m));
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
            for (int i = 0; i < 16; ++i) sts(b + 4 * (LDX * i + c), x[i]);
    }
    bar_sync(2, NPREP);
    {   // 16 -> 32: four warps a pair, four columns a warp, a row and two columns a lane
        const int o = 32 * (w >> 2), i = l >> 1, c = 4 * (w & 3) + 2 * (l & 1);
        float2 y = make_float2(0.f, 0.f), z = y;
        const uint32_t left = at(o + 16 + i, o), right = at(o, o + c);
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 a = lds4(left + 4 * m);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) y = fma2(make_float2(av[e], av[e]), lds2(right + 4 * LDX * (m + e)), y);
        }
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 a = lds4(left + 64 + 4 * m);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int from = 2 * (m + e) + (l & 1);
                z = fma2(make_float2(-av[e], -av[e]), make_float2(__shfl_sync(0xffffffffu, y.x, from), __shfl_sync(0xffffffffu, y.y, from)), z);
            }
        }
        bar_sync(2, NPREP);
        sts2(left + 4 * c, z.x, z.y);
        bar_sync(2, NPREP);
    }
    {   // 32 -> 64: four columns a warp, a row a lane
        const int c = 4 * w;
        const uint32_t left = at(32 + l, 0);
        float2 y0 = make_float2(0.f, 0.f), y1 = y0, z0 = y0, z1 = y0;
#pragma unroll 4
        for (int m = c; m < 32; m += 4) {  // (rows before c of X11's columns are 0)
            const float4 a = lds4(left + 4 * m);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 r = lds4(at(m + e, c));
                y0 = fma2(make_float2(av[e], av[e]), make_float2(r.x, r.y), y0);
                y1 = fma2(make_float2(av[e], av[e]), make_float2(r.z, r.w), y1);
            }
        }
        st_s128(at(l, 32 + c), __float_as_uint(-y0.x), __float_as_uint(-y0.y), __float_as_uint(-y1.x), __float_as_uint(-y1.y));
        __syncwarp();
#pragma unroll 4
        for (int m = 0; m < 32; m += 4) {
            const float4 a = lds4(left + 128 + 4 * m);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 r = lds4(at(m + e, 32 + c));
                z0 = fma2(make_float2(av[e], av[e]), make_float2(r.x, r.y), z0);
                z1 = fma2(make_float2(av[e], av[e]), make_float2(r.z, r.w), z1);
            }
        }
        bar_sync(2, NPREP);
        st_s128(left + 4 * c, __float_as_uint(z0.x), __float_as_uint(z0.y), __float_as_uint(z1.x), __float_as_uint(z1.y));
        bar_sync(2, NPREP);
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

// Where a fragment of Y (or, vt = 0, of U) at t, of 16 channels from ch0 and 16 rows from row0, makes a place of R
// that is not finite as bf16 terms, both Y and v are cleared there, and the channel's first such row is noted.  By one warp, out of
// line: it runs where something is wrong, if ever.
__device__ __noinline__ void clear_odd(uint32_t t, uint32_t vt, uint32_t key, int ch0, int row0, int len, uint32_t marks, volatile uint32_t* flag,
                                       uint32_t bit) {
    float a[8];
    ld16x16(t, a);
    tmem_wait_ld();
    const int l = threadIdx.x & 31;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        const int ch = ch0 + 8 * ((e >> 1) & 1) + (l >> 2), row = row0 + 8 * (e >> 2) + 2 * (l & 3) + (e & 1);
        const uint32_t at = vt + ((ch >> 6) & 1) * 8192u + sw128(row, (ch >> 3) & 7) + 2 * (ch & 7);
        const float r = vt ? lds(key + 4 * row) * a[e] + __uint_as_float((uint32_t)lds16(at) << 16) : a[e];
        if (term_finite(r) || row >= len) continue;
        a[e] = 0.f;
        if (vt) sts16(at, 0);
        asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(marks + 4 * ch), "r"(row) : "memory");
        atomicOr(const_cast<uint32_t*>(flag), bit);
    }
    __syncwarp();
    st16x16f(t, a);
    tmem_wait_st();
}
// rows of a channel's staged output that are none, from its mark or the head's on
__device__ __noinline__ void nan_rows(uint32_t stage, uint32_t marks, int ch, int len, int rows) {
#pragma unroll 1
    for (int r = min(len, __float_as_int(lds(marks + 4 * ch))); r < rows; ++r)
        sts16(stage + (ch >> 6) * 8192u + sw128(r, (ch >> 3) & 7) + 2 * (ch & 7), 0x7FFF);
    sts(marks + 4 * ch, __int_as_float(C));
}

// raw gates of two tokens, `left` of them (or more) in the sequence
__device__ __noinline__ void activate(const Gates& g, Gates::Head head, int left, float& a0, float& a1, float& b0, float& b1) {
    a0 = left > 0 ? g.decay_of(a0, head) : 0.f;
    a1 = left > 1 ? g.decay_of(a1, head) : 0.f;
    b0 = left > 0 ? g.rate_of(b0) : 0.f;
    b1 = left > 1 ? g.rate_of(b1) : 0.f;
}

__global__ void __launch_bounds__(NTHR, 1)
delta_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];  // (as the operands' swizzle wants it; checked below)
    const uint32_t sb = smem_u32(smem);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L_MISC);
    const Sync sy{sb + L_BAR, misc + M_ABORT, p.status};
    if ((sb & 1023u) != 0) {
        if (threadIdx.x == 0) sy.give_up();
        return;
    }
    auto gates = [&](int c) { return sb + L_G + (uint32_t)(c % NG) * GT_BYTES; };
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), l = tid & 31;

    // ---- the unit: heads fastest, then value blocks
    int h = blockIdx.x, vb = blockIdx.y, n = blockIdx.z, unit = 0, bos, eos;
    bool first = true, last = true;  // (of its unit's pieces)
    if (p.cuts) {
        const Piece pc = cut_piece<NTHR>(p, reinterpret_cast<int*>(smem));
        unit = pc.unit;
        h = unit % p.H;
        vb = unit / p.H % p.vblocks;
        n = unit / (p.H * p.vblocks);
        first = pc.c0 == 0;
        last = pc.c1 == (p.T + C - 1) / C;
        bos = n * p.T + pc.c0 * C;
        eos = n * p.T + min(pc.c1 * C, p.T);
    } else {
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
        if (p.cu) { bos = __ldg(p.cu + n); eos = __ldg(p.cu + n + 1); }
        else      { bos = n * p.T; eos = bos + p.T; }
    }
    const int nt = __shfl_sync(0xffffffffu, (eos - bos + C - 1) / C, 0);
    const int hq = h / p.hr, vc0 = vb * VB;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int count = 1;
            if (i == B_S || i == B_R || i == B_UD || i == B_O2READ) count = NCH / 32;
            if ((i >= B_F && i < B_F + 2) || (i >= B_SCREAD && i < B_SCREAD + 2) || i == B_T) count = NPREP / 32;
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
    if (tid < 2 * C) sts(sb + L_RQ + 4 * tid, 1.f);  // (without norms)
    if (w == 24) tmem_alloc(sb + L_MISC + 4 * M_TMEM, TCOLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[M_TMEM], 0);
    auto arrive = [&](int bar) {
        __syncwarp();
        if (l == 0) mbar_arrive(sy.bar(bar));
    };

    if (w == 24) {
        // ------------------------------------------------ all products
        auto scores = [&](int c) {
            sy.wait(B_KQ + c % NKQ, (c / NKQ) & 1);
            tc_fence_after();
            if (!sy.stopped() && elect()) {
                const uint32_t a = lo_k(sb + L_KQ + (c % NKQ) * KQ_BYTES);
#pragma unroll
                for (int kk = 0; kk < KD / 16; ++kk) {
                    const uint64_t d = desc(a + (kk >> 2) * (PANEL >> 4) + (kk & 3) * 2);
                    umma_bf16(tmem + TSC, d, d, idesc_bf16(128, 64, 0, 0), kk > 0);
                }
                umma_commit(sy.bar(B_SC));
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int c = -1; c < nt; ++c) {
            const uint32_t st = sb + L_KQ + ((c + NKQ) % NKQ) * KQ_BYTES;
            if (c >= 0) {
                if (c == p.stall_chunk) Sync::slow_wait(sy.bar(B_NEVER), 0, sy.abort_flag, sy.status, 200000);
                sy.wait(B_S, c & 1);  // S's terms; D of the last chunk has been taken
                if (sy.stopped()) break;
                tc_fence_after();
                if (elect()) {
#pragma unroll 1
                    for (int x = 0; x < 5; ++x) {  // Y from S's terms 2, 1, 0, then O1 from terms 1, 0
                        const uint32_t to = tmem + (x < 3 ? TY : TO1), from = tmem + TS + 64 * (x < 3 ? 2 - x : 4 - x);
                        const uint32_t r = lo_k(st + (x < 3 ? 0 : QROWS));
#pragma unroll
                        for (int kk = 0; kk < KD / 16; ++kk)
                            umma_bf16_ta(to, from + 8 * kk, desc(r + (kk >> 2) * (PANEL >> 4) + (kk & 3) * 2), idesc_bf16(128, 64, 0, 0),
                                         (x != 0 && x != 3) || kk > 0);
                        if (x == 2 || x == 4) umma_commit(sy.bar(x == 2 ? B_Y : B_O1));
                    }
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
                mbar_arrive(sy.bar(B_VFREE));  // (v has been read into R, the last chunk's output has been formed)
                if (c > 0) mbar_arrive(sy.bar(B_GFREE + (c - 1) % NG));
                const uint32_t T = lo_k(sb + L_T), lo = lo_mn(sb + L_LO);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // R's third term
                    umma_bf16(tmem + TY, desc(lo + kk * 128), desc(T + kk * 2), idesc_bf16(128, 64, 1, 0), kk > 0);
#pragma unroll 1
                for (int x = 0; x < 5; ++x) {  // T's terms 2, 1, 1, 0, 0 with R's 0, 1, 0, 1, 0
                    const uint32_t t = (0x00112u >> (4 * x)) & 15u, r = (0x01010u >> (4 * x)) & 15u;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tmem + TY, tmem + TZ + 32 * r + 8 * kk, desc(T + t * (T_TERM >> 4) + kk * 2), idesc_bf16(128, 64, 0, 0), 1);
                }
                umma_commit(sy.bar(B_U));
            }
            __syncwarp();
            sy.wait(B_UD, c & 1);  // (and O1, scaled, lies in O2's place)
            if (sy.stopped()) break;
            tc_fence_after();
            if (elect()) {
                const uint32_t k = lo_kq_mn(st), lo = lo_mn(sb + L_LO), P = lo_k(sb + L_P + (c % NP) * 16384);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(tmem + TD, desc(lo + kk * 128), desc(k + kk * 128), idesc_bf16(128, KD, 1, 1), kk > 0);
#pragma unroll 1
                for (int t = 1; t >= 0; --t)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tmem + TD, tmem + TZ + 32 * t + 8 * kk, desc(k + kk * 128), idesc_bf16(128, KD, 0, 1), 1);
                umma_commit(sy.bar(B_D));
                umma_commit(sy.bar(B_KQFREE + c % NKQ));
#pragma unroll 1
                for (int x = 0; x < 3; ++x) {  // P's terms 1, 0, 0 with U's 0, 1, 0
                    const uint32_t u = x == 1 ? 8 : 0, pt = P + (x == 0 ? P_TERM >> 4 : 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tmem + TSC, tmem + TY + 16 * kk + u, desc(pt + kk * 2), idesc_bf16(128, 64, 0, 0), 1);
                }
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
    } else if (w == 25) {
        // ------------------------------------------------ loads
        auto load_kq = [&](int c) {
            if (elect()) {
                const uint32_t to = sb + L_KQ + (c % NKQ) * KQ_BYTES, full = sy.bar(B_KQ + c % NKQ);
                mbar_arrive_expect_tx(full, KQ_BYTES);
#pragma unroll 1
                for (int x = 0; x < KD / 64; ++x) {
                    tma_load_3d(to + x * PANEL, &tm_k, 64 * x, hq, bos + c * C, full);
                    tma_load_3d(to + x * PANEL + QROWS, &tm_q, 64 * x, hq, bos + c * C, full);
                }
            }
            __syncwarp();
        };
        int kq = 0, v = 0;  // loads that have been issued
#pragma unroll 1
        for (int c = -NKQ; kq < nt || v < nt; ++c) {  // in chunk c: v's stage is free in its middle, k's and q's behind it
            if (c >= -1 && v < nt) {
                if (c >= 0) sy.wait(B_VFREE, c & 1);
                if (sy.stopped()) break;
                if (elect()) {
                    mbar_arrive_expect_tx(sy.bar(B_V), V_BYTES);
#pragma unroll 1
                    for (int x = 0; x < VB / 64; ++x) tma_load_3d(sb + L_V + x * 8192, &tm_v, vc0 + 64 * x, h, bos + v * C, sy.bar(B_V));
                }
                __syncwarp();
                ++v;
            }
            if (kq < nt) {
                if (c >= 0) sy.wait(B_KQFREE + c % NKQ, (c / NKQ) & 1);
                if (sy.stopped()) break;
                load_kq(kq++);
            }
        }
        if (sy.stopped()) {  // leave no copy in flight behind
            if (elect()) {
                for (int x = max(0, kq - NKQ); x < kq; ++x) mbar_wait(sy.bar(B_KQ + x % NKQ), (x / NKQ) & 1);
                if (v > 0) mbar_wait(sy.bar(B_V), (v - 1) & 1);
            }
            __syncwarp();
        }
    } else if (w == 26) {
        // ------------------------------------------------ gates: a chunk's decays and rates, two tokens a lane
        const Gates::Head head = p.gates.head(h);
        const float scale = rsqrtf((float)p.K);
        float ra[2] = {}, rb[2] = {};  // as they lie in memory, asked for a chunk before they are used
#pragma unroll 1
        for (int c = -1; c < nt; ++c) {
            float a0 = ra[0], a1 = ra[1], b0 = rb[0], b1 = rb[1];
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const int t = bos + (c + 1) * C + 2 * l + e;
                const float x = t < eos ? p.gates.raw_decay(t, h) : 0.f, y = t < eos ? p.gates.raw_rate(t, h) : 0.f;
                ra[0] = ra[1];
                rb[0] = rb[1];
                ra[1] = x;
                rb[1] = y;
            }
            if (c < 0) continue;
            const uint32_t gt = gates(c);
            const int left = eos - (bos + c * C);
            if (p.gates.raw || p.gates.logits) activate(p.gates, head, left - 2 * l, a0, a1, b0, b1);
            const float none = __int_as_float(0x7fffffff);
            const int bad = first_nan(a0 < 3e38f && finite(b0) ? 0.f : none, a1 < 3e38f && finite(b1) ? 0.f : none);
            // (sums as pair_sums forms them, with one copy of the conversion)
            long long g = 0, g1 = 0;
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                g1 = fixed(e ? a1 : a0);
                g += g1;
            }
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, g, m);
                if (l >= m) g += y;
            }
            int Il, Fl;
            parts(g, Il, Fl);
            const int Im = __shfl_sync(0xffffffffu, Il, l | 7), Fm = __shfl_sync(0xffffffffu, Fl, l | 7);
            Il = __shfl_sync(0xffffffffu, Il, 31);
            Fl = __shfl_sync(0xffffffffu, Fl, 31);
            if (c >= NG) sy.wait(B_GFREE + c % NG, (c / NG - 1) & 1);
            g -= g1;
#pragma unroll 1
            for (int i = 2 * l; i < 2 * l + 2; ++i, g += g1) {
                int I, F;
                parts(g, I, F);
                const uint32_t to = gt + 4 * i;
                sts(to + GT_G, -(float)I);
                sts(to + GT_G + 256, (float)F * (-1.f / 16777216.f));
                sts(to + GT_COL, pow2_fast(Im - I, Fm - F));
                sts(to + GT_BETA, i < bad ? (i & 1 ? b1 : b0) : 0.f);
                float r;
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {  // 2^(G_l - G_i), then 2^G_i
                    r = pow2(e ? I : Il - I, e ? F : Fl - F);
                    if (e == 0) sts(to + GT_UPD, i < bad ? r : 0.f);
                }
                sts(to + GT_ROW, scale * r);
                sts(to + GT_KEY, -r);
                if (i == C - 1) {
                    sts(gt + GT_LAST, r);
                    sts(gt + GT_LEN, __int_as_float(min(bad, left)));
                }
            }
            arrive(B_G + c % NG);
        }
    } else if (w < 16) {
        // ------------------------------------------------ the chain: R, U' and S, value channels on lanes; the output
        // A warp has 32 key channels of 32 lanes of S, and of the chunk's matrices 16 lanes x 32 rows.
        const int qd = w & 3, part = w >> 2, y16 = 16 * (part & 1), row0 = 32 * (part >> 1);
        const uint32_t lane = (uint32_t)(32 * qd) << 16, lane16 = lane + ((uint32_t)y16 << 16);
        const int vl = 32 * qd + l;
        const bool mine = vc0 + vl < p.V;
        const int rows = p.K - 32 * part;  // of this warp's key channels
        float S[32];
        const size_t state = ((size_t)n * p.H + h) * (size_t)p.K * p.V + (size_t)(32 * part) * p.V + vc0 + vl;
        if (!first) {  // a cut unit's second piece: it began later than the first, so this wait is short
            bool come = false;
            // (a poll takes half a microsecond or more, a chunk six: enough for a whole unit)
            for (int i = 0; i < (1 << 20) + p.T && !(come = ld_acquire_gpu(p.cuts + 1 + unit) == NCH / 32); ++i)
                if (sy.aborted()) break;
            if (!__all_sync(0xffffffffu, come) && l == 0 && !sy.aborted()) sy.give_up();
            __syncwarp();
        }
        {
            const float* src = first ? p.h0 : p.ws;
            const float* from = src + state;
#pragma unroll
            for (int j = 0; j < 32; ++j, from += p.V) S[j] = src && mine && j < rows ? *from : 0.f;
        }
        // Fragments: a lane's row of the four 8 x 8 blocks of a load is channels + 0, + 8, rows + 0, + 8 (sixteen rows further
        // it is 2048 bytes more: the swizzle repeats)
        const int lrow = row0 + (l & 7) + ((l >> 4) << 3), lpiece = 4 * (qd & 1) + (y16 >> 3) + ((l >> 3) & 1);
        const uint32_t frag = (qd >> 1) * 8192u + sw128(lrow, lpiece);
        const uint32_t tf = tmem + lane16 + row0;                 // the warp's fragments of Y, U, O1, O2
        const uint32_t tz = tmem + TZ + lane16 + row0 / 2;        // ... of the terms of R and U'
        const uint32_t pair = 4 * (row0 + 2 * (l & 3));           // a lane's first two rows' factors
        // The terms of sixteen rows' fragments (x[2 G + 0 / 1]: rows 8 G + 2 (l % 4) of channels l / 4 / + 8).  The first ones by
        // themselves: what they leave is finite where a number and its first term are.
        auto first_terms = [](float2 (&x)[4], uint32_t (&t)[4]) {
            float2 odd = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] = round2(x[e]);
                odd = fma2(x[e], make_float2(0.f, 0.f), odd);
            }
            return __any_sync(0xffffffffu, odd.x != 0.f || odd.y != 0.f) != 0;  // something is not
        };
        auto write_fragments = [&](int r, const uint32_t (&first)[4], float2 (&x)[4]) {
            uint32_t t[4];
            st16x8(tz + r / 2, first);
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = round2(x[e]);
            st16x8(tz + r / 2 + 32, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = top2(x[e]);
            stmatrix4_t(sb + L_LO + frag + 128 * r, t);
        };
        auto marked = [&](int b) { return ((misc[M_ODD] >> b) & 1u) != 0u; };
        // One warp polls, the others wait at a named barrier: polls take issue slots from the warps that work.
        auto together = [&] {
            bar_sync(1, NCH);
            tc_fence_after();
        };
        uint32_t gt = sb + L_G, gp = gt, po = 0;  // this chunk's factors, the last one's; the last one's place of P
#pragma unroll 1
        for (int c = 0;; ++c) {
            const uint32_t b = c & 1, pb = b ^ 1;
            // ---- S behind chunk c - 1, its terms for chunk c
            float gl = 1.f;
            if (c > 0) {
                gl = lds(gp + GT_LAST);
                if (marked(pb)) gl += nan_if(__float_as_int(lds(sb + L_MARK + 512 * pb + 4 * vl)) < C);
                if (w == 0) sy.wait(B_D, pb);
                together();
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
                if (c > 0) {
                    float d[8];
                    tmem_ld8(tmem + TD + lane + 32 * part + x, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float2 s = fma2(make_float2(gl, gl), make_float2(S[x + j], S[x + j + 1]), make_float2(d[j], d[j + 1]));
                        S[x + j] = s.x;
                        S[x + j + 1] = s.y;
                    }
                }
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 y = make_float2(S[x + 2 * j], S[x + 2 * j + 1]);
                    t0[j] = round2(y);
                    t1[j] = round2(y);
                    t2[j] = top2(y);
                }
                const uint32_t at = tmem + TS + lane + 16 * part + x / 2;
                tmem_st4(at, t0);
                tmem_st4(at + 64, t1);
                tmem_st4(at + 128, t2);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(B_S);
            if (c > 0) {
                // ---- chunk c - 1's output, through P's place
                const int t0 = bos + (c - 1) * C, n_rows = min(C, eos - t0), len = __float_as_int(lds(gp + GT_LEN));
                const uint32_t rq = sb + L_RQ + 256 * pb + pair, stage = sb + L_P + po;
                if (w == 0) sy.wait(B_O2, pb);
                together();
                float o[16];
                ld16x32(tf + TSC, o);
                float2 m[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) m[g] = lds2(rq + 32 * g);
                const bool odd = len < n_rows || marked(pb);
                tmem_wait_ld();
                tc_fence_before();
                arrive(B_O2READ);
                uint32_t r[8];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 y0 = mul2(m[g], make_float2(o[4 * g], o[4 * g + 1])), y1 = mul2(m[g], make_float2(o[4 * g + 2], o[4 * g + 3]));
                    r[2 * g] = pack_bf16(y0.x, y0.y);
                    r[2 * g + 1] = pack_bf16(y1.x, y1.y);
                }
                stmatrix4_t(stage + frag, r);
                stmatrix4_t(stage + frag + 2048, r + 4);
                if (odd) {
                    bar_sync(1, NCH);  // (a channel's rows are two warps')
                    if (w < 4) nan_rows(stage, sb + L_MARK + 512 * pb, vl, len, n_rows);
                    bar_sync(1, NCH);
                    if (tid == 0) atomicAnd(const_cast<uint32_t*>(misc + M_ODD), ~(1u << pb));
                }
                fence_proxy_async_smem();
                bar_sync(1, NCH);
                if (!sy.aborted()) {
                    if (n_rows == C) {
                        if (tid == 0) {
#pragma unroll
                            for (int x = 0; x < VB / 64; ++x)
                                if (vc0 + 64 * x < p.V) tma_store_3d(&tm_o, stage + x * 8192, vc0 + 64 * x, h, t0);
                            bulk_commit();
                        }
                    } else {  // the sequence's last rows
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + ((size_t)t0 * p.H + h) * p.V + vc0;
#pragma unroll 1
                        for (int x = tid; x < n_rows * (VB / 8); x += NCH) {
                            const int row = x / (VB / 8), ch = x % (VB / 8);
                            uint32_t v[4];
                            ld_s128(stage + (ch >> 3) * 8192u + sw128(row, ch & 7), v);
                            if (vc0 + 8 * ch < p.V) *reinterpret_cast<uint4*>(out + (size_t)row * p.H * p.V + 8 * ch) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                __syncwarp();
                po = po == (NP - 1) * 16384 ? 0 : po + 16384;
            }
            if (c == nt) break;
            // ---- R
            if (w == 0) {
                sy.wait(B_F + b, (c >> 1) & 1);
                sy.wait(B_V, b);
                sy.wait(B_Y, b);
            }
            together();
            const int len = __float_as_int(lds(gt + GT_LEN));
            if (len < C) {  // rows that do not count, for D
                const uint32_t kt = sb + L_KQ + (c % NKQ) * KQ_BYTES;
#pragma unroll 1
                for (int x = tid; x < C * (KD / 8); x += NCH)
                    if ((x & 63) >= len) st_s128(kt + (x >> 9) * PANEL + sw128(x & 63, (x >> 6) & 7), 0, 0, 0, 0);
            }
            const uint32_t vt = sb + L_V;
#pragma unroll 1
            for (int r = 0; r < 32; r += 16) {
                float2 x[4];
                uint32_t first[4];
#pragma unroll 1
                for (int again = 0; again < 2; ++again) {
                    float a[8];
                    uint32_t v[4];
                    ld16x16(tf + TY + r, a);
                    ldmatrix4_t(vt + frag + 128 * r, v);
                    const uint32_t key = gt + GT_KEY + pair + 4 * r;
                    const float2 f[2] = {lds2(key), lds2(key + 32)};
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = add_bf16(v[e], mul2(f[e >> 1], make_float2(a[2 * e], a[2 * e + 1])));
                        if (len < C) {
                            const int j = row0 + r + 8 * (e >> 1) + 2 * (l & 3);
                            if (j >= len) x[e].x = 0.f;
                            if (j + 1 >= len) x[e].y = 0.f;
                        }
                    }
                    if (!first_terms(x, first)) break;
                    clear_odd(tf + TY + r, vt, gt + GT_KEY, 32 * qd + y16, row0 + r, len, sb + L_MARK + 512 * b, misc + M_ODD, 1u << b);
                }
                write_fragments(r, first, x);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(B_R);
            if (c > 0 && tid == 0) {  // the staged output has left
                bulk_wait_read();
                mbar_arrive(sy.bar(B_OFREE + (c - 1) % NP));
            }
            __syncwarp();
            // ---- O1 with its rows' factors, where O2 will be added to it
            if (w == 0) {
                if (c == 0) sy.wait(B_SCREAD, 0);
                if (c + 1 < nt) sy.wait(B_SCREAD + pb, ((c + 1) >> 1) & 1);
                sy.wait(B_O1, b);
            }
            together();
#pragma unroll 1
            for (int r = 0; r < 32; r += 16) {
                float o[8];
                ld16x16(tf + TO1 + r, o);
                const uint32_t row = gt + GT_ROW + pair + 4 * r;
                const float2 f[2] = {lds2(row), lds2(row + 32)};
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 s = mul2(f[e >> 1], make_float2(o[2 * e], o[2 * e + 1]));
                    o[2 * e] = s.x;
                    o[2 * e + 1] = s.y;
                }
                st16x16f(tf + TSC + r, o);
            }
            // ---- U'
            if (w == 0) sy.wait(B_U, b);
            together();
#pragma unroll 1
            for (int r = 0; r < 32; r += 16) {
                float2 x[4], u[4];
                uint32_t t[4];
#pragma unroll 1
                for (int again = 0; again < 2; ++again) {
                    float a[8];
                    ld16x16(tf + TY + r, a);
                    const uint32_t upd = gt + GT_UPD + pair + 4 * r;
                    const float2 f[2] = {lds2(upd), lds2(upd + 32)};
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u[e] = make_float2(a[2 * e], a[2 * e + 1]);
                        x[e] = mul2(f[e >> 1], u[e]);
                    }
                    if (!first_terms(u, t)) break;
                    clear_odd(tf + TY + r, 0, 0, 32 * qd + y16, row0 + r, C, sb + L_MARK + 512 * b, misc + M_ODD, 1u << b);
                }
                // U's two terms for O2, where its sixteen columns were
                st16x8(tf + TY + r, t);
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = pack_bf16(u[e].x, u[e].y);
                st16x8(tf + TY + r + 8, t);
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = round2(x[e]);
                write_fragments(r, t, x);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(B_UD);
            gp = gt;
            gt = gt == sb + L_G + (NG - 1) * GT_BYTES ? sb + L_G : gt + GT_BYTES;
        }
        if (tid == 0) bulk_wait();
        float* dst = last ? p.hT : p.ws;
        if (dst && mine && !sy.aborted()) {
            float* to = dst + state;
#pragma unroll
            for (int j = 0; j < 32; ++j, to += p.V)
                if (j < rows) *to = S[j];
        }
        __syncwarp();
        if (!last && l == 0) red_release_gpu(p.cuts + 1 + unit, 1u);
    } else {
        // ------------------------------------------------ preparation: T and P of a chunk
        // A warp has 32 rows of the scores, of keys or of queries, and 32 of their columns.
        const int t = tid - NCH, i = 32 * (w & 1) + l, c0 = 32 * ((w - 16) >> 2);
        const bool query = (w & 2) != 0, hi = (w & 1) != 0;
        const uint32_t sc = tmem + TSC + ((uint32_t)(32 * (w & 3)) << 16) + c0, X = sb + L_X;
        const float scale = rsqrtf((float)p.K);
        const bool qnorm = (p.flags & KDA_FLAG_Q_L2NORM) != 0, knorm = (p.flags & KDA_FLAG_K_L2NORM) != 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const uint32_t gt = gates(c), P = sb + L_P + (c % NP) * 16384;
            if (w == 16) {
                sy.wait(B_G + c % NG, (c / NG) & 1);
                if (c >= NP) sy.wait(B_OFREE + c % NP, (c / NP - 1) & 1);  // P's place
                sy.wait(B_SC, c & 1);
            }
            bar_sync(2, NPREP);
            tc_fence_after();
            const bool some = hi || c0 == 0;  // (else the block lies right of the diagonal)
            float x[32];
            if (some) {
                ld32(sc, x);
                tmem_wait_ld();
            }
            tc_fence_before();
            arrive(B_SCREAD + (c & 1));
            const float gi = -lds(gt + GT_G + 4 * i), gf = -lds(gt + GT_G + 256 + 4 * i);
            float rk = 1.f;
            if (qnorm || knorm) {  // the rows' norms, half a row a thread
                const uint32_t row = sb + L_KQ + (c % NKQ) * KQ_BYTES + (query ? QROWS : 0) + (c0 >> 5) * PANEL;
                const bool on = query ? qnorm : knorm;
                const float n2 = on ? row_square(row, i) : 0.f;
                if (c0 > 0) sts(X + 4 * (LDX * i + (query ? 66 : 65)), n2);
                bar_sync(2, NPREP);
                if (c0 == 0) {
                    const float sum = n2 + lds(X + 4 * (LDX * i + (query ? 66 : 65)));
                    // (NaN behind the sequence, too, perhaps: what it is a factor of does not count)
                    sts(query ? sb + L_RQ + 256 * (c & 1) + 4 * i : X + 4 * (LDX * i + 64), on ? row_norm(sum) : 1.f);
                }
                bar_sync(2, NPREP);
                rk = lds(X + 4 * (LDX * i + 64));
                if (knorm && !query && c0 == 0) {  // a key's norm is a factor of its column, too
                    sts(gt + GT_G + 256 + 4 * i, log2f(rk) - gf);
                    sts(gt + GT_COL + 4 * i, lds(gt + GT_COL + 4 * i) * rk / lds(X + 4 * (LDX * (i | 15) + 64)));
                }
                bar_sync(2, NPREP);
            }
            const int full = __float_as_int(lds(gt + GT_LEN));
            // A's rows (lanes with keys) in X, P's rows (with queries) as two bf16 terms: the score times
            // f 2^(G_i - G_j), 0 where j > last.  Left of the row's 32 the factor parts into the row's and the column's,
            // both <= 1; within them each is formed by itself.
            const int last = i < full ? i - (query ? 0 : 1) : -1;
            const float f = last < 0 ? 0.f : query ? scale : lds(gt + GT_BETA + 4 * i) * rk;
            float2 odd = make_float2(0.f, 0.f);
            const float r0 = ex2_fast((gi + lds(gt + GT_G + 4 * 15)) + (gf + lds(gt + GT_G + 256 + 4 * 15)));
            const float r1 = ex2_fast((gi + lds(gt + GT_G + 4 * 31)) + (gf + lds(gt + GT_G + 256 + 4 * 31)));
            const uint32_t to = query ? P + 128 * i : X + 4 * (LDX * i + c0), turn = (i & 7) << 4 ^ 2 * c0;  // (P's 16-byte pieces at ^ turn)
            const bool left = hi && c0 == 0;
            const uint32_t gs = gt + 4 * c0;
            float4 gj = lds4(gs + (left ? GT_COL : GT_G)), fj = lds4(gs + GT_G + 256);
            // (the factors of the next columns are asked for before these are stored: the order in which they stand is kept)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const int j = c0 + e;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 g = gj, f4 = fj;
                if (e < 28) {
                    gj = lds4(gs + (left ? GT_COL : GT_G) + 4 * (e + 4));
                    fj = lds4(gs + GT_G + 256 + 4 * (e + 4));
                }
                if (some) {
                    float2 e0, e1;
                    if (left) {  // (with the key's norm of the column j | 15, which the others' are given by)
                        const float r = e < 16 ? r0 : r1;
                        e0 = mul2(make_float2(r, r), make_float2(g.x, g.y));
                        e1 = mul2(make_float2(r, r), make_float2(g.z, g.w));
                    } else {
                        const float2 g0 = add2(add2(make_float2(gi, gi), make_float2(g.x, g.y)), add2(make_float2(gf, gf), make_float2(f4.x, f4.y)));
                        const float2 g1 = add2(add2(make_float2(gi, gi), make_float2(g.z, g.w)), add2(make_float2(gf, gf), make_float2(f4.z, f4.w)));
                        e0 = make_float2(ex2_fast(g0.x), ex2_fast(g0.y));
                        e1 = make_float2(ex2_fast(g1.x), ex2_fast(g1.y));
                    }
                    e0 = mul2(mul2(make_float2(f, f), make_float2(x[e], x[e + 1])), e0);
                    e1 = mul2(mul2(make_float2(f, f), make_float2(x[e + 2], x[e + 3])), e1);
                    y.x = j <= last ? e0.x : 0.f;
                    y.y = j + 1 <= last ? e0.y : 0.f;
                    y.z = j + 2 <= last ? e1.x : 0.f;
                    y.w = j + 3 <= last ? e1.y : 0.f;
                    odd = fma2(make_float2(y.x, y.y), make_float2(0.f, 0.f), odd);
                    odd = fma2(make_float2(y.z, y.w), make_float2(0.f, 0.f), odd);
                }
                if (query) {
                    float2 ya = make_float2(y.x, y.y), yb = make_float2(y.z, y.w);
                    const uint32_t at = to + (((2 * e & ~15) ^ turn) | (2 * e & 8)), a0 = round2(ya), b0 = round2(yb);
                    sts_pair(at, a0, b0);
                    sts_pair(at + P_TERM, pack_bf16(ya.x, ya.y), pack_bf16(yb.x, yb.y));
                } else if (some) st_s128(to + 4 * e, __float_as_uint(y.x), __float_as_uint(y.y), __float_as_uint(y.z), __float_as_uint(y.w));
            }
            // a row of A that is not finite: its key is not, or one before it
            const unsigned none = __ballot_sync(0xffffffffu, !query && (odd.x != 0.f || odd.y != 0.f));
            if (!query && l == 0) misc[M_BAD + 2 * (w & 1) + (c0 >> 5)] = none ? 32 * (w & 1) + __ffs(none) - 1 : C;
            bar_sync(2, NPREP);
            const int len = min(min(full, (int)min(misc[M_BAD], misc[M_BAD + 1])), (int)min(misc[M_BAD + 2], misc[M_BAD + 3]));
            if (!query && c0 == 0 && (knorm || len < full)) {
                sts(gt + GT_KEY + 4 * i, rk * lds(gt + GT_KEY + 4 * i));
                sts(gt + GT_UPD + 4 * i, i < len ? rk * lds(gt + GT_UPD + 4 * i) : 0.f);
                if (i >= len) {  // rows that do not count
                    sts(gt + GT_BETA + 4 * i, 0.f);
#pragma unroll 1
                    for (int j = 0; j < i; ++j) sts(X + 4 * (LDX * i + j), 0.f);
                }
            }
            if (t == 0) {
                sts(gt + GT_LEN, __int_as_float(len));
                if (len < min(C, eos - (bos + c * C))) sts(gt + GT_LAST, __int_as_float(0x7fffffff));
            }
            arrive(B_F + (c & 1));
            if (len < full) bar_sync(2, NPREP);
            invert(X, t);
            // T's terms: a row and 16 columns a thread
            if (c > 0) sy.wait(B_U, (c - 1) & 1);  // their last reader
            const int r = t & 63, cc = 16 * (t >> 6);
#pragma unroll 1
            for (int x = cc; x < cc + 16; x += 8) {
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = x + 4 * e;
                    const float4 y = lds4(X + 4 * (LDX * r + j)), m = lds4(gt + GT_BETA + 4 * j);
                    float2 y0 = mul2(make_float2(y.x, y.y), make_float2(m.x, m.y)), y1 = mul2(make_float2(y.z, y.w), make_float2(m.z, m.w));
                    if (j > (r | 31)) y0 = y1 = make_float2(0.f, 0.f);  // (right of the diagonal's blocks of 32: nothing is there)
                    t0[2 * e] = round2(y0);
                    t0[2 * e + 1] = round2(y1);
                    t1[2 * e] = round2(y0);
                    t1[2 * e + 1] = round2(y1);
                    t2[2 * e] = top2(y0);
                    t2[2 * e + 1] = top2(y1);
                }
                const uint32_t at = sb + L_T + sw128(r, x / 8);
                st_s128(at, t0[0], t0[1], t0[2], t0[3]);
                st_s128(at + T_TERM, t1[0], t1[1], t1[2], t1[3]);
                st_s128(at + 2 * T_TERM, t2[0], t2[1], t2[2], t2[3]);
            }
            fence_proxy_async_smem();
            arrive(B_T);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 24) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

}  // namespace
}  // namespace delta

// bf16, K up to 128 and a multiple of 8, V a multiple of 8 (a row of each begins 16-byte aligned, as TMA wants it)
bool delta_tensor_dims(bool bf16, int K, int V) { return bf16 && K % 8 == 0 && K <= 128 && V % 8 == 0; }

namespace delta {
namespace {
// Chunks that cuts cost an SM (a state's way through memory, another piece's start).  us cut / whole, heads of 128: 240 units of 8
// chunks (13 an SM for the 16 of two waves) 110/111, 160 of 4 (5 for 8) 55/64, 256 of 16 (27 for 32) 188/196, 256 of 64 (108 for 128)
// 621/700, 160 of 64 (68 for 128) 401/692.
constexpr int kCutCost = 3;
struct Plan {
    int per, pieces;
    size_t states, counters;
};
Plan plan(int B, int T, int H, int K, int V, bool packed) {
    Plan pl{0, 0, 0, 0};
    const int vblocks = (V + VB - 1) / VB;
    if (packed || (pl.per = plan_cuts(B, T, H, vblocks, kCutCost)) == 0) return pl;
    pl.pieces = count_pieces(T, B * H * vblocks, pl.per);
    pl.states = ((size_t)B * H * K * V * sizeof(float) + 255) / 256 * 256;
    pl.counters = ((size_t)(B * H * vblocks + 1) * sizeof(unsigned) + 255) / 256 * 256;
    return pl;
}
}  // namespace
}  // namespace delta

size_t delta_tensor_workspace_bytes(int B, int T, int H, int K, int V, bool packed) {
    const delta::Plan pl = delta::plan(B, T, H, K, V, packed);
    return pl.states + pl.counters;
}

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
    const Plan pl = plan(a.B, a.T, a.H, a.K, a.V, a.cu != nullptr);
    unsigned* cuts = pl.per ? (unsigned*)((char*)a.ws + pl.states) : nullptr;
    const Params p{Gates(a), a.h0, a.hT, a.cu, a.o, a.N, a.T, a.H, a.H / a.Hk, a.K, a.V, vblocks, a.flags, (float*)a.ws, cuts, pl.per, a.status, hook_stall_chunk()};
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e == cudaSuccess && pl.per) e = cudaMemsetAsync(cuts, 0, pl.counters, a.stream);
    if (e != cudaSuccess) return e;
    delta_chunk_kernel<<<pl.per ? dim3(pl.pieces) : dim3(a.H, vblocks, a.N), NTHR, SMEM_BYTES, a.stream>>>(m[0], m[1], m[2], m[3], p);
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
