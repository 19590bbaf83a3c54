// Linear attention with a decay for each head in chunks of 64 tokens, bf16 inputs, on the tensor
// cores (tcgen05 with TMEM accumulators, TMA loads).
//
// Per chunk of a (sequence, head, block of value channels), G_i the decay's sum in log2 units up to
// and including row i, l the last row, s = 1/sqrt(K):
//   P[i][j] = 2^(G_i - G_j) (q_i . k_j)  for j <= i, else 0                     (bf16 operand)
//   o_i     = s (2^G_i S^T q_i + sum_j P[i][j] v_j)
//   S      <- 2^G_l S + sum_j k_j (2^(G_l - G_j) v_j)^T                         (FP32)
// as four products, value channels (M = 128) on TMEM lanes:
//   QK [i, j] = q k^T;   O1^T [v, i] = S^T q^T;   O2^T [v, i] = v^T P^T;   D^T [v, c] = vd^T k, added to S^T.
// The stored state is S 2^-E, E from kTop = 32 down to 0.  Where the decay is slow, E' = E + G_l and the
// values carry 2^(G_l - G_j - E') = 2^-(E + G_j): what is stored is only added to, and S is rounded once
// less.  Before E falls below 0 the stored state is scaled with the addition (factor 2^(E + G_l - kTop)) and
// E starts again at kTop.  So what is stored is never larger than S, and nothing overflows that FP32 holds;
// the price is at the other end, where values below 2^-85 lose low bits.
//
// q, k and v enter the products as they are; O1's row factor s 2^(E + G_i) is applied to the FP32
// results.  The decay is a number per row, so no anchors are needed: G_i - G_j <= 0 is formed as a
// difference of an integer and of a fraction part (integer sums), exact whatever the sums.
//
// A masked score is 0, and 0 times a value that is not finite is NaN: such values are taken out of the tile
// before P meets them, and their channel's outputs are NaN from their token on (the first row of each
// channel is noted, GT_MARK).  The state has them as they are.
//
// Roundings: for a bf16 output P and the copy of S that O1 reads are bf16 (each adds the output's own rounding
// once more; both in quadrature keep o's error within 1.45 of one rounding).  A caller who wants more asks for a
// float32 output: there both are three bf16 terms (24 bits), S's one after another through the copy's place
// (kFine; 4 x 4096 tokens, 64 heads: 427 us).  The state is a float32 output and
// feeds every later chunk, so the scaled values vd are three bf16 terms (24 bits), and a chunk's additions are
// summed by themselves and then added to S in rounded FP32: the tensor cores cut, not round, what they add to an
// accumulator, and S as that accumulator leaned to zero by 1.3e-6 for each chunk of its memory (9e-6 at a fixed
// decay of -0.0023, 3.6e-4 after 32768 tokens with hardly any).  Now the cut is one of a chunk's own sum, the
// smallest term first: S is off by 1e-7 at -0.0023 and by 3e-7 to 1e-6 after 32768 tokens with hardly any decay,
// whatever their signs.  That costs a read of the sum and a read and write of S a chunk (4 x 4096 tokens, 64 heads:
// 218 us against 203).
//
// What bounds it is shared memory's 128 bytes a clock next to HBM, and the order of a chunk's steps through TMEM: per
// chunk at K = V = 128 the loads write 48 KB, the products read 150 KB, the warps and the stores about 75 KB.  That is
// why two terms of the scaled values are operands that lie in TMEM, straight from registers (there is no column left
// for the third); scaled keys in shared memory cost 48 KB of writes and 48 KB of reads more a chunk.
// 4 x 4096 tokens, 64 heads, the final state written: 1.09 GB in 218 us with cut units, 5.0 TB/s; 20480 packed tokens
// with states, 32 heads: 0.74 GB in 147 us, 5.0 TB/s; one sequence of 32767 tokens, 16 heads, cut into segments (k
// and v read twice): 180 us.  A head of 256 key channels is two of 128 whose FP32 outputs are written, read back and
// added (8 x 2048 tokens, 32 heads, 256 x 256: 735 us, of which 194 for the addition, against 7266 in FP32).
//
// One CTA per unit and SM, 28 warps: 0-3 P, 4-11 state, 12-15 output, 16-23 scaled values, 24 the output's
// products, 25 decay factors, 26 the state's products, 27 loads and scores.  Every wait is bounded (a CTA
// that gives up lets its copies and MMAs finish, frees its TMEM and returns).  The roles' loops are kept
// rolled and short: together they have to fit the instruction caches (unrolled, "no instruction" was 40 %
// of all stalls and a chunk took twice as long).
#include <cudaTypedefs.h>

#include "common.cuh"
#include "decay_gates.cuh"
#include "kda_internal.h"
#include "sm100.cuh"

namespace kda {
namespace decay {

using namespace sm100;

__device__ unsigned int g_decay_timeouts = 0;

constexpr int C = 64, NTHR = 896, NS = 3, NG = 8, kAhead = 1, kRanked = 128, kMaxCuts = 4096, kCutCost = 8, kTop = 32;

// barriers
enum { B_FULL = 0, B_FREE = B_FULL + NS, B_QK = B_FREE + NS, B_P, B_D = B_P + NS, B_DREAD, B_SBF, B_VD, B_STATE, B_VFREE, B_INTER, B_O,
       B_OFREE = B_O + 2, B_DRAIN, B_DRAIN2, B_DRAIN3, B_NEVER, NBAR };

// The decay factors of a chunk, one slot of a ring of NG (written when the chunk is loaded, read
// last by its output warps, at most NS + 3 chunks later): byte offsets of its float arrays.
constexpr uint32_t GT_G = 0;       // [64][2] G_i as integer and fraction
constexpr uint32_t GT_ROW = 512;   // [64] s 2^(E + G_i)
constexpr uint32_t GT_KEY = 768;   // [64] 2^(G_l - G_j - E'), the values' factors
constexpr uint32_t GT_COL = 1024;  // [64] 2^(G_m - G_j), m the last of j's 16 rows
constexpr uint32_t GT_LAST = 1280; // the stored state's factor before this chunk's product, 1: none
constexpr uint32_t GT_OUT = 1284;  // 2^E'
constexpr uint32_t GT_MARK = 1296; // [128] bytes: each channel's first row with a value that is not finite, 64: none
constexpr uint32_t GT_BYTES = 1424;

// kFine: P and the state that the queries read in three bf16 terms each (24 bits), for a float32 output
template <int KD, int VB, bool kFine = false>
struct Layout {
    static constexpr uint32_t QB = C * KD * 2, VBYTES = C * VB * 2, STAGE = 2 * QB + VBYTES;
    static constexpr uint32_t LO = NS * STAGE, P = LO + (KD == 128 ? (kFine ? 1 : 2) * VBYTES : 0), O = P + 2 * C * C * 2, G = O + (kFine ? 4 * C * C * 2 : VBYTES);
    static constexpr uint32_t BAR = G + NG * GT_BYTES, MISC = (BAR + 8 * NBAR + 15) / 16 * 16, END = MISC + 16;
    // P's term and buffer: the second and third terms have the place of the staged output
    __host__ __device__ static constexpr uint32_t term(int t, int b) { return t == 0 ? P + b * (C * C * 2) : O + (2 * b + t - 1) * (C * C * 2); }
    // an A operand of 64 value channels is read as 128: up to 8 KB behind its tile
    static constexpr uint32_t BYTES = END + 1024 + 64;
};
// TMEM columns: S^T; its bf16 copy; the terms of the scaled values; what a chunk adds to kN key channels of S^T; QK;
// O1; O2.  With 128 key channels all 512 are taken: a state product is formed in two passes of 64, and the values'
// third term lies in shared memory, in two places by turns (kSmemTerm).
template <int KD, bool kStates>
struct Tmem {
    static constexpr int kN = kStates ? KD : 64;
    static constexpr bool kSmemTerm = KD == 128 && !kStates;
    static constexpr uint32_t S = 0, SB = 128, VD = 192, D = KD == 64 ? 64 : kStates ? 288 : 256, QK = KD == 64 ? 288 : 320;
    static constexpr uint32_t O1 = 384, O2 = 448, COLS = 512;
};

struct Params {
    const float* decay;
    int decay_stride;  // floats between tokens (H, or 0 for one decay per head)
    const float* h0;
    float* hT;
    const int32_t* cu;
    void* o;
    int N, T, H, hr, K, V;
    int vblocks;
    int k0;         // this launch's first key channel (a head of 256 takes two launches of 128)
    int seg;        // tokens of a segment (a multiple of C), 0: whole sequences
    float* ws;      // segment states [slot][h][K][V]
    float* wdec;    // segment decays [slot][h]
    unsigned* cuts; // cut units: a ticket, then a counter for each unit (all zero); else null
    int per;        // chunks of an SM with cut units
    int* status;
    int stall_chunk;
};

struct Sync {
    uint32_t bars;
    volatile uint32_t* abort_flag;
    int* status;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
    __device__ __forceinline__ void give_up() const {
        atomicAdd(&g_decay_timeouts, 1u);
        if (status) atomicOr(status, 1);
        *abort_flag = 1u;
    }
    // (out of line: one copy, so that the loops stay in the instruction caches)
    __device__ __noinline__ void slow_wait(int i, uint32_t parity, uint32_t limit) const {
        if (!*abort_flag && !mbar_wait_unless(bar(i), parity, abort_flag, limit)) give_up();
    }
    __device__ __forceinline__ bool aborted() const { return *abort_flag != 0u; }
    // A whole warp's wait, the same answer in every lane: false when a wait has given up and this
    // one's phase has not come.
    __device__ __forceinline__ bool warp_wait(int i, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
        slow_wait(i, parity, 1u << 22);
        return __all_sync(0xffffffffu, !aborted());
    }
};

// A product's operand in shared memory: the descriptor's low word changes with the address (16-byte
// units), its high word (stride 1024 bytes between groups of 8 rows, 128-byte swizzle) does not.
__device__ __forceinline__ uint32_t lo_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }               // K-major
__device__ __forceinline__ uint32_t lo_mn(uint32_t addr) { return (addr >> 4) | ((8192u >> 4) << 16); }    // MN-major, 64 apart
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)DESC_HI << 32) | lo; }
// True in one lane of a converged warp.  The products are issued inside a branch on this: there
// their descriptors stay in uniform registers and a product of 128 x 64 x 16 issues in 31 to 48
// clocks, its own time; in a branch on the lane number, or each predicated, it took 50 to 85.
__device__ __forceinline__ uint32_t elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p;
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the issued stores have read their shared memory / are complete
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ float lds(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 lds2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts2(uint32_t a, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint16_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint16_t v) { asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory"); }
__device__ __forceinline__ void ld_s128(uint32_t a, uint32_t* v) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void ld32(uint32_t t, float* v) {
    tmem_ld16(t, v);
    tmem_ld16(t + 16, v + 16);
}
// 16 lanes x 32 columns: thread t gets lanes t / 4 and t / 4 + 8 and of each eight columns the pair
// 2 (t % 4), 2 (t % 4) + 1: v[4 g + 0..1] the first lane's, v[4 g + 2..3] the second's
__device__ __forceinline__ void ld16x32(uint32_t t, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void ld16x16(uint32_t t, float* v) {  // the same for 16 columns
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// two FP32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}\n" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// four 8 x 8 matrices of 16-bit elements, each stored transposed; lane i holds the address of
// (transposed) row i % 8 of matrix i / 8
__device__ __forceinline__ void stmatrix4_t(uint32_t a, const uint32_t* r) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

// four 8 x 8 matrices of 16-bit elements, each transposed on the way (addresses as above)
__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// 16 lanes x 16 columns: of each four columns, thread t has column t % 4 of lanes t / 4 and t / 4 + 8
__device__ __forceinline__ void st16x16(uint32_t t, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t a, const uint32_t* r) {  // as they are
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

// The upper bf16 halves of two floats as a pair, and what they leave.  Cutting three times gives a
// float's 24 significant bits as three bf16 terms exactly: 8 + 8 + 8 (a cut leaves a remainder that
// the next term holds, as a rounding would, without a conversion).
__device__ __forceinline__ uint32_t cut(float2& x) {
    const uint32_t top = 0xFFFF0000u, a = __float_as_uint(x.x), b = __float_as_uint(x.y);
    x = fma2(make_float2(__uint_as_float(a & top), __uint_as_float(b & top)), make_float2(-1.f, -1.f), x);
    return __byte_perm(a, b, 0x7632);
}

// both floats in three terms
__device__ __forceinline__ void split(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = cut(x);
    mid = cut(x);
    lo = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// Values that are not finite in the `len` rows of a tile of VB channels: cleared, and each channel's first of them
// noted.  (By one warp, out of line and rolled: it runs where something is wrong, if ever.)
template <int VB>
__device__ __noinline__ void hide_odd(uint32_t tile, int len, uint32_t marks) {
#pragma unroll 1
    for (int ch = threadIdx.x & 31; ch < VB; ch += 32) {
        int first = C;
#pragma unroll 1
        for (int r = len - 1; r >= 0; --r) {
            const uint32_t at = tile + (ch >> 6) * 8192u + sw128(r, (ch >> 3) & 7) + 2 * (ch & 7);
            if ((lds16(at) & 0x7F80) != 0x7F80) continue;
            sts16(at, 0);
            first = r;
        }
        sts8(marks + ch, first);
    }
    fence_proxy_async_smem();
    __syncwarp();
}
// ... and a noted channel's outputs (one channel a lane) in a tile of bf16 rows, where bit 0 says that there are notes
__device__ __noinline__ void nan_rows(uint32_t tile, uint32_t marks, int ch, uint32_t odd) {
    __syncwarp();  // (a warp's 32 channels have been stored by all its lanes)
    if (odd & 1u)
#pragma unroll 1
        for (int r = (int)lds8(marks + ch); r < C; ++r) sts16(tile + (ch >> 6) * 8192u + sw128(r, (ch >> 3) & 7) + 2 * (ch & 7), 0x7FFF);
}

// Whole sequences of one length, more units than SMs, the last wave part-empty: the units' chunks are
// laid end to end and shared out evenly, `per` (at least a unit's nt) an SM, so a unit that does not fit into what
// is left of an SM is cut.  Its part on the next SM, which is that SM's first work, is the earlier one in time;
// the part at this SM's end runs per - nt chunks or more after the other's end and finds its state there.
// Blocks take the pieces in the order of their starts (a ticket, so that whoever waits began later than what it waits for):
// the SMs' first pieces, then the whole units, then the cut units' second pieces, the longest first (their SMs
// are free first).  4 x 4096 tokens, 64 heads (256 units): 218 us against 225 with whole
// units; 5 x 4096, 64 heads (320): 264 against 331; 2 x 16384, 80 heads (160): 479 against 841.
struct Piece {
    int unit, c0, c1;
};
__device__ __forceinline__ Piece cut_piece(const Params& p, int* scratch) {
    const int tid = threadIdx.x, nt = (p.T + C - 1) / C, units = p.N * p.H * p.vblocks;
    const int W = units * nt, firsts = (W + p.per - 1) / p.per;
    if (tid == 0) scratch[0] = (int)atomicAdd(p.cuts, 1u);
    for (int m = tid; m < firsts; m += NTHR) scratch[2 + m] = (int)((long)m * p.per % nt);
    __syncthreads();
    const int i = scratch[0];
    Piece pc;
    if (i < firsts) {
        const int at = i * p.per;
        pc.unit = at / nt;
        pc.c0 = 0;
        pc.c1 = (pc.unit + 1) * nt - at;
    } else if (i < units) {
        // the (i - firsts)-th unit without a multiple of per in it: of the units up to u, ceil((u + 1) nt / per) have one
        int lo = 0, hi = units - 1;
        while (lo < hi) {
            const int u = (lo + hi) / 2;
            if (u + 1 - ((u + 1) * nt + p.per - 1) / p.per > i - firsts) hi = u;
            else lo = u + 1;
        }
        pc = {lo, 0, nt};
    } else {
        for (int m = tid; m < firsts; m += NTHR) {
            const int mine = scratch[2 + m];
            int rank = 0;
            for (int j = 0; j < firsts; ++j) rank += scratch[2 + j] > mine || (scratch[2 + j] == mine && j < m);
            if (rank == i - units) scratch[1] = m;
        }
        __syncthreads();
        const int m = scratch[1], at = m * p.per;
        pc.unit = at / nt;
        pc.c0 = nt - at % nt;
        pc.c1 = nt;
    }
    fence_proxy_async_smem();  // (a stage's place)
    __syncthreads();
    return pc;
}

// kStates: only the state a segment adds (no queries, no output), for the segments' scan.
template <int KD, int VB, typename OT, bool kStates, bool kFine = false>
__global__ void __launch_bounds__(NTHR, 1)
decay_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, Params p) {
    using L = Layout<KD, VB, kFine>;
    using M = Tmem<KD, kStates>;
    constexpr int kTerms = kFine ? 3 : 1, NP = KD / M::kN;  // NP: passes of kN key channels of a state product
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L::MISC);
    const Sync sy{sb + L::BAR, misc + 2, p.status};
    // (the aligned base is not known to be shared memory: a slot's floats are read by address)
    auto gates = [&](int c) { return sb + L::G + (uint32_t)(c % NG) * GT_BYTES; };
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), l = tid & 31;

    // ---- the unit: heads fastest, then value blocks
    int h = blockIdx.x, vb = blockIdx.y, slot = blockIdx.z, unit = 0;
    int n, bos, eos;
    bool first = true, last = true;
    if (!kStates && p.cuts) {
        const Piece pc = cut_piece(p, reinterpret_cast<int*>(smem));
        unit = pc.unit;
        h = unit % p.H;
        vb = unit / p.H % p.vblocks;
        n = slot = unit / (p.H * p.vblocks);
        first = pc.c0 == 0;
        last = pc.c1 == (p.T + C - 1) / C;
        bos = n * p.T + pc.c0 * C;
        eos = n * p.T + min(pc.c1 * C, p.T);
    } else if (p.seg == 0) {
        n = slot;
        if (p.cu && p.N <= kRanked) {
            // The blocks start in order: the longest sequences first, so that none is left for the
            // end (16 sequences of 20480 tokens, 32 heads: 181 us in their own order, 157 in this)
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
            n = ranked[slot];
            fence_proxy_async_smem();  // (a stage's place)
            __syncthreads();
        }
        if (p.cu) { bos = __ldg(p.cu + n); eos = __ldg(p.cu + n + 1); }
        else      { bos = n * p.T; eos = bos + p.T; }
    } else {
        const ChunkMap cm{p.cu, p.N, p.T, p.seg};
        int t0, len, b0, e0;
        cm.map_first(slot, n, t0, len, b0, e0);
        if (n < 0) return;
        first = t0 == b0;
        last = t0 + len >= e0;
        bos = t0;
        eos = t0 + len;
        if (kStates && last) return;  // nothing follows it
    }
    const int nt = __shfl_sync(0xffffffffu, (eos - bos + C - 1) / C, 0);
    const int hq = h / p.hr, vc0 = vb * VB;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int count = 1;
            if (i >= B_FULL && i < B_FULL + NS) count = 2;                 // the loads and the decay factors
            if (i >= B_FREE && i < B_FREE + NS) count = kStates ? 1 : 2;   // the products of both issuing warps
            if (i >= B_P && i < B_P + NS) count = 4 + 8;                   // four P warps, eight that have looked at v
            if (i == B_OFREE) count = 4;                                   // four output warps
            if (i >= B_D && i <= B_VD) count = 8;                          // eight warps
            mbar_init(sy.bar(i), count);
        }
        fence_mbar_init();
        misc[2] = misc[3] = 0;  // given up; a bit for each slot of the factors' ring that ever had notes
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_o);
    }
    if (w == 26) tmem_alloc(sb + L::MISC, M::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);

    if (w < 4) {
        // ------------------------------------------------ P = QK with the decays, bf16, K-major rows
        // A warp's 16 rows (QK's 64 rows lie on the first 16 lanes of each quarter of TMEM) in
        // fragments of 8 x 8: a thread has rows l / 4 and l / 4 + 8, and of eight columns a pair.
        if constexpr (!kStates) {
            const int r0 = 16 * w + (l >> 2), cp = 2 * (l & 3);
            const float scale = rsqrtf((float)p.K), log2_scale = -0.5f * log2f((float)p.K);
            // where a lane's row of the four stored blocks goes (columns 16 cb: piece 2 cb more)
            const int srow = 16 * w + (l & 15), spiece = l >> 4;
            for (int x = l; x < 2 * 16 * 8; x += 32) {  // the blocks right of the diagonal stay zero
                const int row = 16 * w + (x & 15), piece = (x >> 4) & 7;
                if (piece > 2 * w + 1)
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) st_s128(sb + L::term(t, x >> 7) + sw128(row, piece), 0, 0, 0, 0);
            }
#pragma unroll 1
            for (int c = 0; c < nt; ++c) {
                const int b = c & 1;
                if (!sy.warp_wait(B_FULL + c % NS, (c / NS) & 1)) break;                // the decay factors
                if (!sy.warp_wait(B_QK, c & 1)) break;
                if (c >= 2 && !sy.warp_wait(B_O + b, ((c - 2) >> 1) & 1)) break;        // this P buffer's last reader
                tc_fence_after();
                const uint32_t gt = gates(c), to = sb + L::P + b * (C * C * 2), qk = tmem + M::QK + ((uint32_t)(32 * w) << 16);
                float2 g0 = lds2(gt + GT_G + 8 * r0), g1 = lds2(gt + GT_G + 8 * (r0 + 8));
                // left of the diagonal block the factor parts into a row's and a column's, both <= 1
#pragma unroll 1
                for (int cb = 0; cb < w; ++cb) {
                    float x[8];
                    ld16x16(qk + 16 * cb, x);
                    const float2 gm = lds2(gt + GT_G + 8 * (16 * cb + 15));
                    const float f0 = scale * ex2_fast((g0.x - gm.x) + (g0.y - gm.y));
                    const float f1 = scale * ex2_fast((g1.x - gm.x) + (g1.y - gm.y));
                    tmem_wait_ld();
                    uint32_t r[4], r1[4], r2[4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float2 f = lds2(gt + GT_COL + 4 * (16 * cb + 8 * g + cp));
                        const float2 y0 = mul2(make_float2(x[4 * g], x[4 * g + 1]), mul2(f, make_float2(f0, f0)));
                        const float2 y1 = mul2(make_float2(x[4 * g + 2], x[4 * g + 3]), mul2(f, make_float2(f1, f1)));
                        if constexpr (kFine) {
                            split(y0, r[2 * g], r1[2 * g], r2[2 * g]);
                            split(y1, r[2 * g + 1], r1[2 * g + 1], r2[2 * g + 1]);
                        } else {
                            r[2 * g] = pack_bf16(y0.x, y0.y);
                            r[2 * g + 1] = pack_bf16(y1.x, y1.y);
                        }
                    }
                    stmatrix4(to + sw128(srow, 2 * cb + spiece), r);
                    if constexpr (kFine) {
                        stmatrix4(sb + L::term(1, b) + sw128(srow, 2 * cb + spiece), r1);
                        stmatrix4(sb + L::term(2, b) + sw128(srow, 2 * cb + spiece), r2);
                    }
                }
                {
                    float x[8];
                    ld16x16(qk + 16 * w, x);
                    g0.y += log2_scale;
                    g1.y += log2_scale;
                    tmem_wait_ld();
                    uint32_t r[4], r1[4], r2[4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int j = 8 * g + cp, i = l >> 2;  // within the block
                        const float4 gj = lds4(gt + GT_G + 8 * (16 * w + j));
                        const float y0 = x[4 * g] * ex2_fast((g0.x - gj.x) + (g0.y - gj.y));
                        const float y1 = x[4 * g + 1] * ex2_fast((g0.x - gj.z) + (g0.y - gj.w));
                        const float y2 = x[4 * g + 2] * ex2_fast((g1.x - gj.x) + (g1.y - gj.y));
                        const float y3 = x[4 * g + 3] * ex2_fast((g1.x - gj.z) + (g1.y - gj.w));
                        if constexpr (kFine) {
                            split(make_float2(j <= i ? y0 : 0.f, j + 1 <= i ? y1 : 0.f), r[2 * g], r1[2 * g], r2[2 * g]);
                            split(make_float2(j <= i + 8 ? y2 : 0.f, j + 1 <= i + 8 ? y3 : 0.f), r[2 * g + 1], r1[2 * g + 1], r2[2 * g + 1]);
                        } else {
                            r[2 * g] = pack_bf16(j <= i ? y0 : 0.f, j + 1 <= i ? y1 : 0.f);
                            r[2 * g + 1] = pack_bf16(j <= i + 8 ? y2 : 0.f, j + 1 <= i + 8 ? y3 : 0.f);
                        }
                    }
                    stmatrix4(to + sw128(srow, 2 * w + spiece), r);
                    if constexpr (kFine) {
                        stmatrix4(sb + L::term(1, b) + sw128(srow, 2 * w + spiece), r1);
                        stmatrix4(sb + L::term(2, b) + sw128(srow, 2 * w + spiece), r2);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (l == 0) mbar_arrive(sy.bar(B_P + c % NS));
            }
        }
    } else if (w == 25) {
        // ------------------------------------------------ decay factors
        const float kScale = rsqrtf((float)p.K);
        const float* dp = p.decay + h;
        auto raw = [&](int t) { return t < eos ? __ldg(dp + (size_t)t * p.decay_stride) : 0.f; };
        float a0 = raw(bos + 2 * l), a1 = raw(bos + 2 * l + 1);
        long long E = (long long)kTop << 32, total = 0;  // the stored state's exponent; the whole segment's log2 decay
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int s = c % NS, t0 = bos + c * C;
            const float x0 = a0, x1 = a1;
            a0 = raw(t0 + C + 2 * l);
            a1 = raw(t0 + C + 2 * l + 1);
            int I[2], F[2];
            long long G[2];
            pair_sums(x0, x1, G);
            const long long Gl = __shfl_sync(0xffffffffu, G[1], 31);
            parts(G[0], I[0], F[0]);
            parts(G[1], I[1], F[1]);
            const int Il = __shfl_sync(0xffffffffu, I[1], 31), Fl = __shfl_sync(0xffffffffu, F[1], 31);
            const int Im = __shfl_sync(0xffffffffu, I[1], l | 7), Fm = __shfl_sync(0xffffffffu, F[1], l | 7);
            const int bad = first_nan(x0, x1);
            const float poison = nan_if(bad < C);  // of the state behind the chunk
            if constexpr (kStates) total = max(total + Gl, -(4000ll << 32));
            // this chunk's value and row factors, and the exponent behind it
            int Ei, Ef, ni, nf;
            parts(E, Ei, Ef);
            parts(E + Gl, ni, nf);
            const bool renew = ni < 0 || ni >= 2 * kTop;
            // the slot's last readers are done: chunk c - NS is loaded (and its FULL phase complete),
            // so the products of c - 2 NS are done, which the output warps of c - NG preceded
            if (c >= NS && !sy.warp_wait(B_FULL + s, ((c / NS) - 1) & 1)) break;
            const uint32_t gt = gates(c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * l + e;
                const float none = nan_if(i >= bad);
                sts2(gt + GT_G + 8 * i, (float)I[e], (float)F[e] * (1.f / 16777216.f) + none);
                const int rf = Ef + F[e];
                sts(gt + GT_ROW + 4 * i, kScale * pow2_fast(Ei + I[e] + (rf >> 24), rf & 0xFFFFFF) + none);
                sts(gt + GT_KEY + 4 * i, (renew ? pow2(Il - I[e] - kTop, Fl - F[e]) : pow2(-Ei - I[e] - (rf >> 24), -(rf & 0xFFFFFF))) + poison);
                sts(gt + GT_COL + 4 * i, pow2_fast(Im - I[e], Fm - F[e]) + nan_if((i | 15) >= bad));
            }
            if (l == 0) {
                sts(gt + GT_LAST, (renew ? pow2(ni - kTop, nf) : 1.f) + poison);
                sts(gt + GT_OUT, renew ? pow2i(kTop) : pow2(ni, nf));
            }
            E = renew ? (long long)kTop << 32 : E + Gl;
            __syncwarp();
            if (l == 0) mbar_arrive(sy.bar(B_FULL + s));
            if (kStates && c == nt - 1 && l == 0 && vb == 0) {
                int i, f;
                parts(total, i, f);
                p.wdec[(size_t)slot * p.H + h] = pow2(max(i, -300), f) + poison;
            }
        }
    } else if (w == 27) {
        // ------------------------------------------------ loads, and the scores QK
        // Both as early as they can: a chunk's loads when its stage is free, its scores when it is
        // loaded and P has been formed from the last chunk's.
        // (One copy of each in the loop: a warp that issues from several places misses in the
        // instruction caches.)
        int c = 0, nq = kStates ? nt : 0;
        uint32_t idle = 0;
        auto ready = [&](int bar, int parity, uint32_t ns) {
            return __all_sync(0xffffffffu, mbar_try_wait(sy.bar(bar), parity, ns));
        };
#pragma unroll 1
        while (c < nt || nq < nt) {
            bool moved = false;
            if (c < nt && (c < NS || ready(B_FREE + c % NS, ((c / NS) - 1) & 1, nq < nt ? 0 : 1000))) {
                if (elect()) {
                    const uint32_t st = sb + (c % NS) * L::STAGE, full = sy.bar(B_FULL + c % NS);
                    const int t0 = bos + c * C;
                    mbar_arrive_expect_tx(full, (kStates ? L::QB : 2 * L::QB) + L::VBYTES);
#pragma unroll
                    for (int x = 0; x < KD / 64; ++x) {
                        if constexpr (!kStates) tma_load_3d(st + x * 8192, &tm_q, p.k0 + 64 * x, hq, t0, full);
                        tma_load_3d(st + L::QB + x * 8192, &tm_k, p.k0 + 64 * x, hq, t0, full);
                    }
#pragma unroll
                    for (int x = 0; x < VB / 64; ++x) tma_load_3d(st + 2 * L::QB + x * 8192, &tm_v, vc0 + 64 * x, h, t0, full);
                    // The stages hold the chunks in work and one ahead, too few bytes in flight for
                    // the memory: the tiles behind them come into L2 meanwhile
                    if (c + kAhead < nt) {
#pragma unroll
                        for (int x = 0; x < KD / 64; ++x) {
                            if constexpr (!kStates) tma_prefetch_l2_3d(&tm_q, p.k0 + 64 * x, hq, t0 + kAhead * C);
                            tma_prefetch_l2_3d(&tm_k, p.k0 + 64 * x, hq, t0 + kAhead * C);
                        }
#pragma unroll
                        for (int x = 0; x < VB / 64; ++x) tma_prefetch_l2_3d(&tm_v, vc0 + 64 * x, h, t0 + kAhead * C);
                    }
                }
                __syncwarp();
                ++c;
                moved = true;
            }
            if constexpr (!kStates) {
                if (nq < c && (nq < 1 || ready(B_P + (nq - 1) % NS, ((nq - 1) / NS) & 1, 0)) &&
                    ready(B_FULL + nq % NS, (nq / NS) & 1, 200)) {
                    const uint32_t qa = lo_k(sb + (nq % NS) * L::STAGE), ka = qa + (L::QB >> 4);
                    tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int kk = 0; kk < KD / 16; ++kk) {
                            const uint32_t d = (kk >> 2) * 512 + (kk & 3) * 2;
                            umma_bf16(tmem + M::QK, desc(qa + d), desc(ka + d), idesc_bf16(64, 64, 0, 0), kk > 0);
                        }
                        umma_commit(sy.bar(B_QK));
                    }
                    __syncwarp();
                    ++nq;
                    moved = true;
                }
            }
            idle = moved ? 0 : idle + 1;
            if (idle >= (1u << 24) && l == 0) sy.give_up();
            if ((idle & 255u) == 255u && __any_sync(0xffffffffu, sy.aborted())) break;
        }
        if (__any_sync(0xffffffffu, sy.aborted())) {  // leave no copy and no MMA in flight behind
            if (elect()) {
                umma_commit(sy.bar(B_DRAIN3));
                mbar_wait(sy.bar(B_DRAIN3), 0);
                // (where a chunk's decay factors do not come any more, their arrival is made here)
                for (int x = max(0, c - NS); x < c; ++x)
                    if (!mbar_wait(sy.bar(B_FULL + x % NS), (x / NS) & 1, 1u << 12)) {
                        mbar_arrive(sy.bar(B_FULL + x % NS));
                        mbar_wait(sy.bar(B_FULL + x % NS), (x / NS) & 1);
                    }
            }
            __syncwarp();
        }
    } else if (w == 26) {
        // ------------------------------------------------ the state's products
        constexpr uint32_t id_s = idesc_bf16(128, M::kN, 0, 1);
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int s = c % NS;
            const uint32_t k = lo_mn(sb + s * L::STAGE + L::QB);
            if (c == p.stall_chunk) sy.slow_wait(B_NEVER, 0, 2000);
            if (!sy.warp_wait(B_VD, c & 1)) break;
            bool ok = true;
#pragma unroll 1
            for (int x = 0; x < NP; ++x) {
                // the state warps have read what it replaces
                if (x > 0) ok = sy.warp_wait(B_D, c & 1);
                else if (c > 0) ok = sy.warp_wait(B_DREAD, (c - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (elect()) {  // vd^T k, the smallest of the three terms of vd first: each cut is one of the sum so far
#pragma unroll
                    for (int term = 2; term >= 0; --term)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t b = desc(k + x * 512 + kk * 128);
                            if (M::kSmemTerm && term == 2) umma_bf16(tmem + M::D, desc(lo_mn(sb + L::LO + (kFine ? 0 : (c & 1) * L::VBYTES)) + kk * 128), b, idesc_bf16(128, M::kN, 1, 1), kk > 0);
                            else umma_bf16_ta(tmem + M::D, tmem + M::VD + 32 * term + 8 * kk, b, id_s, term < 2 || kk > 0);
                        }
                    umma_commit(sy.bar(B_STATE));
                    if (x + 1 == NP) umma_commit(sy.bar(B_VFREE));
                    if (x + 1 == NP && c + NS < nt) umma_commit(sy.bar(B_FREE + s));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (__any_sync(0xffffffffu, sy.aborted())) {  // let the MMAs in flight finish
            if (elect()) {
                umma_commit(sy.bar(B_DRAIN));
                mbar_wait(sy.bar(B_DRAIN), 0);
            }
            __syncwarp();
        }
    } else if (w == 24) {
        // ------------------------------------------------ the output's products
        if constexpr (!kStates) {
            constexpr uint32_t id_o1 = idesc_bf16(128, 64, 0, 0), id_o2 = idesc_bf16(128, 64, 1, 0);
#pragma unroll 1
            for (int c = 0; c < nt; ++c) {
                const int s = c % NS, b = c & 1;
                const uint32_t q = lo_k(sb + s * L::STAGE), v = lo_mn(sb + s * L::STAGE + 2 * L::QB);
                bool ok = sy.warp_wait(B_FULL + s, (c / NS) & 1);  // the queries
                if (!ok) break;
#pragma unroll 1
                for (int t = 0; t < kTerms; ++t) {  // (the terms come one after another into one place)
                    if (!(ok = sy.warp_wait(B_SBF, (kTerms * c + t) & 1))) break;
                    if (c >= 1 && t == 0 && !(ok = sy.warp_wait(B_OFREE, (c - 1) & 1))) break;  // the output warps have read the last chunk's
                    tc_fence_after();
                    if (elect()) {
#pragma unroll
                        for (int kk = 0; kk < KD / 16; ++kk)
                            umma_bf16_ta(tmem + M::O1, tmem + M::SB + 8 * kk, desc(q + (kk >> 2) * 512 + (kk & 3) * 2), id_o1, kk > 0 || t > 0);
                        umma_commit(sy.bar(B_INTER));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (!sy.warp_wait(B_P + s, (c / NS) & 1)) break;  // (v's rows behind the sequence are cleared, too)
                if ((misc[3] >> (c % NG)) & 1u) hide_odd<VB>(sb + s * L::STAGE + 2 * L::QB, min(C, eos - (bos + c * C)), gates(c) + GT_MARK);
                tc_fence_after();
                if (elect()) {
#pragma unroll
                    for (int t = 0; t < kTerms; ++t)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16(tmem + M::O2, desc(v + kk * 128), desc(lo_k(sb + L::term(t, b)) + kk * 2), id_o2, kk > 0 || t > 0);
                    umma_commit(sy.bar(B_O + b));
                    if (c + NS < nt) umma_commit(sy.bar(B_FREE + s));
                }
                __syncwarp();
            }
            if (__any_sync(0xffffffffu, sy.aborted())) {
                if (elect()) {
                    umma_commit(sy.bar(B_DRAIN2));
                    mbar_wait(sy.bar(B_DRAIN2), 0);
                }
                __syncwarp();
            }
        }
    } else if (w < 12) {
        // ------------------------------------------------ state: S^T in TMEM, lane = value channel
        const int vl = 32 * (w & 3) + l;
        const uint32_t lane = (uint32_t)(32 * (w & 3)) << 16;
        const int c0 = w < 8 ? 0 : 32;  // this warp's key channels: 32 of each 64, from c0
        const bool mine = vl < VB && vc0 + vl < p.V;
        const size_t at = (size_t)p.k0 * p.V + vc0 + vl, st = ((size_t)n * p.H + h) * (size_t)p.K * p.V + at;
        const size_t sg = ((size_t)slot * p.H + h) * (size_t)p.K * p.V + at;
        // a cut sequence's segments take their incoming states from the scan
        const bool head = p.cuts && !last;  // a cut unit's first piece: its state goes to the other
        const float* src = kStates ? nullptr : (first && last) || head ? (p.h0 ? p.h0 + st : nullptr) : p.ws + sg;
        float* dst = kStates || head ? p.ws + sg : (last && p.hT) ? p.hT + st : nullptr;
        if (!kStates && p.cuts && !first) {  // the second: it began later, so this wait is short
            bool come = false;
            // (a poll takes half a microsecond or more, a chunk two: enough for a whole unit)
            for (int i = 0; i < (1 << 20) + p.T && !(come = ld_acquire_gpu(p.cuts + 1 + unit) == 8u); ++i)
                if (sy.aborted()) break;
            if (!__all_sync(0xffffffffu, come) && l == 0 && !sy.aborted()) sy.give_up();
            __syncwarp();
        }
        auto arrive = [&](int bar) {
            tc_fence_before();
            __syncwarp();
            if (l == 0) mbar_arrive(sy.bar(bar));
        };
        auto copy = [&](int x, const float* v) {  // 32 columns of the bf16 copy
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
            tmem_st16(tmem + M::SB + lane + x / 2, r);
        };
        // the incoming state, 32 rows in flight; an empty sequence's goes straight on
#pragma unroll 1
        for (int x = c0; x < KD; x += 64) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
            if (src && mine) {
                const float* from = src + (size_t)x * p.V;
#pragma unroll
                for (int j = 0; j < 32; ++j, from += p.V) v[j] = *from;
            }
            __syncwarp();
            if (nt > 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= 1.f / (1ll << kTop);  // E = kTop
                tmem_st16(tmem + M::S + lane + x, reinterpret_cast<uint32_t*>(v));
                tmem_st16(tmem + M::S + lane + x + 16, reinterpret_cast<uint32_t*>(v) + 16);
                if (!kStates && !kFine) copy(x, v);
            } else if (dst && mine) {
                float* to = dst + (size_t)x * p.V;
#pragma unroll
                for (int j = 0; j < 32; ++j, to += p.V) *to = v[j];
            }
        }
        tmem_wait_st();
        if (!kStates && !kFine && nt > 0) arrive(B_SBF);
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            if constexpr (kFine) {
                // the copy's three terms one after another
#pragma unroll 1
                for (int t = 0; t < kTerms && ok; ++t) {
                    if (c + t > 0 && !(ok = sy.warp_wait(B_INTER, (kTerms * c + t - 1) & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int x = c0; x < KD; x += 64) {
                        float v[32];
                        uint32_t r[16];
                        ld32(tmem + M::S + lane + x, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            uint32_t r1, r2;
                            split(make_float2(v[2 * j], v[2 * j + 1]), r[j], r1, r2);
                            r[j] = t == 0 ? r[j] : t == 1 ? r1 : r2;
                        }
                        tmem_st16(tmem + M::SB + lane + x / 2, r);
                    }
                    tmem_wait_st();
                    arrive(B_SBF);
                }
                if (!ok) break;
            }
            const bool more = !kStates && !kFine && c + 1 < nt;  // a copy for the next chunk
#pragma unroll 1
            for (int x = c0; x < KD; x += 64) {
                if (x % M::kN < 64 && !(ok = sy.warp_wait(B_STATE, (NP * c + x / M::kN) & 1))) break;
                tc_fence_after();
                const float gl = lds(gates(c) + GT_LAST);  // (there since the values were scaled)
                float d[32], v[16];
                ld32(tmem + M::D + lane + x % M::kN, d);
                tmem_ld16(tmem + M::S + lane + x, v);
                tmem_wait_ld();
                if (x % M::kN + 64 >= M::kN) arrive(x + 64 >= KD ? B_DREAD : B_D);
                if (more && x == c0 && !(ok = sy.warp_wait(B_INTER, c & 1))) break;  // the copy's last reader
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                    if (y > 0) {
                        tmem_ld16(tmem + M::S + lane + x + y, v);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 t = fma2(make_float2(gl, gl), make_float2(v[j], v[j + 1]), make_float2(d[y + j], d[y + j + 1]));
                        d[y + j] = t.x;
                        d[y + j + 1] = t.y;
                    }
                    tmem_st16(tmem + M::S + lane + x + y, reinterpret_cast<uint32_t*>(d) + y);
                }
                if (more) copy(x, d);
            }
            if (!ok) break;
            tmem_wait_st();
            if (more) arrive(B_SBF);
        }
        if (nt > 0 && ok) {
            const float out = lds(gates(nt - 1) + GT_OUT);
#pragma unroll 1
            for (int x = c0; x < KD; x += 64) {
                float v[32];
                ld32(tmem + M::S + lane + x, v);
                tmem_wait_ld();
                if (dst && mine) {
                    float* to = dst + (size_t)x * p.V;  // (one address carried on, not 32 kept)
#pragma unroll
                    for (int j = 0; j < 32; ++j, to += p.V) *to = v[j] * out;
                }
                __syncwarp();
            }
            if (head && l == 0) red_release_gpu(p.cuts + 1 + unit, 1u);
        }
    } else if (w < 16) {
        // ------------------------------------------------ output rows
        if constexpr (!kStates) {
            const int vl = 32 * (w & 3) + l;
            const uint32_t lane = (uint32_t)(32 * (w & 3)) << 16;
            constexpr bool kStaged = sizeof(OT) == 2;
            // a bf16 row segment would be written 64 bytes a warp and token: it goes through shared
            // memory (the TMA layout) and leaves as one tile, or row by row at a sequence's end
            const bool mine = vl < VB;
#pragma unroll 1
            for (int c = 0; c < nt; ++c) {
                const int b = c & 1, t0 = bos + c * C, len = min(C, eos - t0);
                if (kStaged && c > 0) {
                    if (tid == 384) bulk_wait_read();
                    bar_sync(1, 128);  // (all four warps have copied their rows of the last chunk, too)
                }
                const bool ok = sy.warp_wait(B_O + b, (c >> 1) & 1);
                tc_fence_after();
                const uint32_t gt = gates(c) + GT_ROW;
                OT* dst = (OT*)p.o + ((size_t)t0 * p.H + h) * p.V + vc0;
                const size_t step = (size_t)p.H * p.V;
                auto taken = [&] {  // both buffers have been read
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (l == 0) mbar_arrive(sy.bar(B_OFREE));
                };
                if (!ok) {
                    if (!kStaged) break;
                } else if constexpr (kStaged) {
                    // pieces of 16 channels x 32 tokens: fragments of 8 x 8, stored transposed
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t at = tmem + lane + ((uint32_t)(16 * (x >> 1)) << 16) + 32 * (x & 1);
                        float o1[16], o2[16];
                        ld16x32(at + M::O1, o1);
                        ld16x32(at + M::O2, o2);
                        if (x < 3) tmem_wait_ld();
                        else taken();
                        const int ch = 4 * (w & 3) + 2 * (x >> 1) + ((l >> 3) & 1);  // the 16-byte piece of this lane's address
                        const uint32_t base = sb + L::O + (ch >> 3) * 8192u;
#pragma unroll
                        for (int g = 0; g < 4; g += 2) {
                            uint32_t r[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 f = lds2(gt + 4 * (32 * (x & 1) + 8 * (g + e) + 2 * (l & 3)));
                                const float *a1 = o1 + 4 * (g + e), *a2 = o2 + 4 * (g + e);
                                const float2 y0 = fma2(f, make_float2(a1[0], a1[1]), make_float2(a2[0], a2[1]));
                                const float2 y1 = fma2(f, make_float2(a1[2], a1[3]), make_float2(a2[2], a2[3]));
                                r[2 * e] = pack_bf16(y0.x, y0.y);
                                r[2 * e + 1] = pack_bf16(y1.x, y1.y);
                            }
                            if (32 * (w & 3) < VB)
                                stmatrix4_t(base + sw128(32 * (x & 1) + 8 * (g + (l >> 4)) + (l & 7), ch & 7), r);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        float o1[16], o2[16];
                        tmem_ld16(tmem + M::O1 + lane + 16 * x, o1);
                        tmem_ld16(tmem + M::O2 + lane + 16 * x, o2);
                        if (x < 3) tmem_wait_ld();
                        else taken();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float r = fmaf(lds(gt + 4 * (16 * x + j)), o1[j], o2[j]);
                            if (mine && 16 * x + j < len) dst[(16 * x + j) * step + vl] = to_out<OT>(r);
                        }
                    }
                }
                if constexpr (!kStaged) {
                    if ((misc[3] >> (c % NG)) & 1u) {
#pragma unroll 1
                        for (int r = mine ? (int)lds8(gates(c) + GT_MARK + vl) : C; r < len; ++r)
                            dst[r * step + vl] = to_out<OT>(__int_as_float(0x7fffffff));
                    }
                } else {
                    if (__any_sync(0xffffffffu, mine && misc[3] != 0u)) nan_rows(sb + L::O, gates(c) + GT_MARK, vl, misc[3] >> (c % NG));
                    fence_proxy_async_smem();
                    bar_sync(1, 128);
                    if (sy.aborted()) {
                        // (as the other warps: each chunk has the same barriers)
                    } else if (len == C) {
                        if (tid == 384) {
#pragma unroll
                            for (int x = 0; x < VB / 64; ++x) tma_store_3d(&tm_o, sb + L::O + x * 8192, vc0 + 64 * x, h, t0);
                            bulk_commit();
                        }
                    } else {
                        for (int x = tid - 384; x < len * (VB / 8); x += 128) {
                            const int row = x / (VB / 8), ch = x % (VB / 8);
                            uint32_t v[4];
                            ld_s128(sb + L::O + (ch >> 3) * 8192u + sw128(row, ch & 7), v);
                            *reinterpret_cast<uint4*>(dst + row * step + 8 * ch) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
            }
            if (kStaged && tid == 384) bulk_wait();
        }
    } else if (w < 24) {
        // ------------------------------------------------ scaled values, three bf16 terms
        // A warp's 32 value channels (its quarter of the lanes) x 32 rows: fragments of 8 x 8 read
        // transposed, so that a thread has a channel's pairs of consecutive rows, as the products
        // read them from TMEM.  The terms take the place of the last chunk's, so they wait for its
        // state product in registers.
        const int qd = w & 3, jh = (w - 16) >> 2;
        const bool mine = 32 * qd < VB;
        // a lane's row of the four 8 x 8 blocks of a load: channels + 0, + 8, rows + 0, + 8
        const int lrow = 32 * jh + (l & 7) + ((l >> 4) << 3), lpiece = 4 * (qd & 1) + ((l >> 3) & 1);
        const uint32_t to = tmem + M::VD + ((uint32_t)(32 * qd) << 16) + 16 * jh;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int s = c % NS, len = min(C, eos - (bos + c * C));
            const uint32_t kt = sb + s * L::STAGE + L::QB, vt = kt + L::QB, gt = gates(c) + GT_KEY;
            if (!sy.warp_wait(B_FULL + s, (c / NS) & 1)) break;
            if (len < C) {  // rows behind the sequence (another one's, or anything), for the products
                const int x0 = tid - 512;
                for (int x = x0; x < C * (VB / 8); x += 256)
                    if (((x >> 3) & 63) >= len) st_s128(vt + (x >> 9) * 8192u + sw128((x >> 3) & 63, x & 7), 0, 0, 0, 0);
                for (int x = x0; x < C * (KD / 8); x += 256)
                    if (((x >> 3) & 63) >= len) st_s128(kt + (x >> 9) * 8192u + sw128((x >> 3) & 63, x & 7), 0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            uint32_t hi[2][8];
            float2 rest[2][8], odd = make_float2(0.f, 0.f);
            if (mine) {
#pragma unroll
                for (int g = 0; g < 4; g += 2) {
                    const float2 f0 = lds2(gt + 4 * (32 * jh + 8 * g + 2 * (l & 3)));
                    const float2 f1 = lds2(gt + 4 * (32 * jh + 8 * g + 8 + 2 * (l & 3)));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // sixteen channels each
                        uint32_t r[4];
                        ldmatrix4_t(vt + (qd >> 1) * 8192u + sw128(lrow + 8 * g, lpiece + 2 * y), r);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2& x = rest[y][2 * g + e];
                            x = mul2(make_float2(bf_lo(r[e]), bf_hi(r[e])), e < 2 ? f0 : f1);
                            if (len < C) {  // (whether or not the row is cleared yet)
                                const int j = 32 * jh + 8 * g + (e < 2 ? 0 : 8) + 2 * (l & 3);
                                if (j >= len) x.x = 0.f;
                                if (j + 1 >= len) x.y = 0.f;
                            }
                            hi[y][2 * g + e] = cut(x);
                            odd = fma2(x, make_float2(0.f, 0.f), odd);
                        }
                    }
                }
                // what is not finite leaves no number: then the first term alone is the value
                if (odd.x != 0.f || odd.y != 0.f) {
                    atomicOr(const_cast<uint32_t*>(misc + 3), 1u << (c % NG));
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2& x = rest[e >> 3][e & 7];
                        if (x.x != x.x) x.x = 0.f;
                        if (x.y != x.y) x.y = 0.f;
                    }
                }
            }
            if constexpr (!kStates) {
                __syncwarp();
                if (l == 0) mbar_arrive(sy.bar(B_P + s));
            }
            // the third term has two places in shared memory, whose last reader was the product of two chunks ago
            // (one for a float32 output, which then waits like the others)
            uint32_t mid[2][8];
            const uint32_t lo = sb + L::LO + (kFine ? 0 : (c & 1) * L::VBYTES) + (qd >> 1) * 8192u;
            auto third = [&] {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        mid[y][e] = cut(rest[y][e]);
                        r[e] = __byte_perm(__float_as_uint(rest[y][e].x), __float_as_uint(rest[y][e].y), 0x7632);
                    }
#pragma unroll
                    for (int g = 0; g < 4; g += 2) stmatrix4_t(lo + sw128(lrow + 8 * g, lpiece + 2 * y), r + 2 * g);  // as the values lie there
                }
                fence_proxy_async_smem();
            };
            if (M::kSmemTerm && !kFine && mine) third();
            if (c > 0 && !sy.warp_wait(B_VFREE, (c - 1) & 1)) break;
            tc_fence_after();
            if (M::kSmemTerm && kFine && mine) third();
            if (mine) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t at = to + ((uint32_t)(16 * y) << 16);
                    st16x16(at, hi[y]);
                    if constexpr (M::kSmemTerm) {
                        st16x16(at + 32, mid[y]);
                    } else {
                        uint32_t r[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = cut(rest[y][e]);
                        st16x16(at + 32, r);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            r[e] = __byte_perm(__float_as_uint(rest[y][e].x), __float_as_uint(rest[y][e].y), 0x7632);
                        st16x16(at + 64, r);
                    }
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (l == 0) mbar_arrive(sy.bar(B_VD));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 26) {
        tc_fence_after();
        tmem_dealloc(tmem, M::COLS);
    }
}

// The segments' states in order: each segment's addition becomes its incoming state.
__global__ void __launch_bounds__(256) decay_scan_kernel(const float* __restrict__ h0, float* ws, const float* __restrict__ wdec,
                                                         ChunkMap cm, int H, int KV) {
    const int n = blockIdx.z, h = blockIdx.y, e = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (e >= KV) return;
    int bos, eos;
    if (cm.cu) { bos = __ldg(cm.cu + n); eos = __ldg(cm.cu + n + 1); }
    else       { bos = n * cm.T; eos = bos + cm.T; }
    const int ns = (eos - bos + cm.C - 1) / cm.C;
    if (ns < 2) return;
    const int s0 = cm.first_slot(n, bos);
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h0) S = *reinterpret_cast<const float4*>(h0 + ((size_t)n * H + h) * KV + e);
    // The first segment's too: the last one may write its final state over h0.  Eight additions are on
    // their way at once (9 segments of 16 heads from cold caches 5 us; one ahead of the sum 19).
    constexpr int R = 8;
    const size_t step = (size_t)H * KV;
    float* at = ws + ((size_t)s0 * H + h) * KV + e;
    const float* decay = wdec + (size_t)s0 * H + h;
    for (int s = 0; s < ns; s += R) {
        float4 add[R];
        float d[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (s + j + 1 >= ns) break;
            add[j] = *reinterpret_cast<const float4*>(at + j * step);
            d[j] = __ldg(decay + (size_t)(s + j) * H);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (s + j >= ns) break;
            *reinterpret_cast<float4*>(at + j * step) = S;
            if (s + j + 1 >= ns) break;
            S.x = fmaf(d[j], S.x, add[j].x);
            S.y = fmaf(d[j], S.y, add[j].y);
            S.z = fmaf(d[j], S.z, add[j].z);
            S.w = fmaf(d[j], S.w, add[j].w);
        }
        at += R * step;
    }
}

// A head of 256 key channels is the sum of two of 128 (scores, outputs and states all split that way):
// their FP32 outputs added and rounded once.
template <typename OT>
__global__ void __launch_bounds__(256) decay_join_kernel(const float* __restrict__ a, const float* __restrict__ b,
                                                         OT* __restrict__ o, long rows, const int32_t* end, long row4) {
    const long n4 = (end ? (long)__ldg(end) : rows) * row4;  // (rows behind a packed batch's last sequence stay as they are)
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long)gridDim.x * 256) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(a) + i), y = __ldcs(reinterpret_cast<const float4*>(b) + i);
        const float r[4] = {x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w};
        if constexpr (sizeof(OT) == 4) reinterpret_cast<float4*>(o)[i] = make_float4(r[0], r[1], r[2], r[3]);
        else reinterpret_cast<uint2*>(o)[i] = make_uint2(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]));
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* ptr = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// [tokens, H, D] bf16, box of 64 channels x 1 head x 64 tokens, 128-byte swizzle
bool make_map(CUtensorMap* m, const void* base, long tokens, int H, int D) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    const cuuint32_t box[3] = {64, 1, 64}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a segment (0: whole sequences).  One CTA per SM runs a unit (a sequence's head and
// value block) in order, so few units leave SMs idle: the time axis is then cut into segments whose
// added states come from a first pass over k and v (half of the call's bytes once more) and a scan.
// That pays when whole sequences fill less than half of the SMs, and segments stay at least four
// chunks long (a segment costs its state twice through memory, one chunk's worth of bytes).
int plan_segment(int B, int T, int H, int vblocks, int N, bool packed) {
    const int sms = planned_sm_count();
    const long units = (long)N * H * vblocks;
    if (sms <= 0 || units == 0 || 2 * units > sms) return 0;
    const long tokens = packed ? T : (long)N * T;
    long per = (tokens * H * vblocks + sms - 1) / sms;  // tokens of a unit for one CTA per SM
    per = (per + C - 1) / C * C;
    if (!packed) {  // whole segments per sequence, evenly
        const long ns = sms / units;
        per = ((T + ns - 1) / ns + C - 1) / C * C;
    }
    if (per < 4 * C) per = 4 * C;
    return 2 * per > T ? 0 : (int)per;
}

// Chunks of an SM where units are cut (0: they are not).  Cuts cost an SM about eight chunks (a state's way,
// more starts): 8 x 1024 tokens, 32 heads (27 chunks an SM for the 32 of two waves) 78 us with cuts and
// 69 without, 8 x 2048, 64 heads (108 for 128) 231 and 234.
int plan_cuts(int B, int T, int H, int vblocks) {
    const long sms = planned_sm_count(), units = (long)B * H * vblocks, nt = (T + C - 1) / C;
    if (sms <= 0 || units <= sms || units * nt > 1 << 30 || sms > kMaxCuts) return 0;
    const long waves = (units + sms - 1) / sms, per = (units * nt + sms - 1) / sms;
    return per + kCutCost <= waves * nt ? (int)per : 0;
}

struct Plan {
    int seg, slots, per, pieces;
    size_t states, counters, half, bytes;  // states handed on; counters; one of the two outputs of a head of 256; in all
};
Plan plan(int B, int T, int H, int K, int V, int N, bool packed) {
    Plan pl{0, N, 0, 0, 0, 0, 0, 0};
    const int vblocks = V > 128 ? 2 : 1;
    pl.seg = plan_segment(B, T, H, vblocks, N, packed);
    if (pl.seg) {
        pl.slots = packed ? T / pl.seg + N + 1 : N * ((T + pl.seg - 1) / pl.seg);
        pl.states = (size_t)pl.slots * H * K * V * sizeof(float);
        pl.bytes = pl.states + ((size_t)pl.slots * H * sizeof(float) + 255) / 256 * 256;
    }
    if (!packed && !pl.seg && (pl.per = plan_cuts(B, T, H, vblocks)) > 0) {
        const int nt = (T + C - 1) / C, units = B * H * vblocks, firsts = (units * nt + pl.per - 1) / pl.per;
        pl.pieces = units;
        for (int m = 0; m < firsts; ++m) pl.pieces += (long)m * pl.per % nt != 0;
        pl.states = (size_t)N * H * K * V * sizeof(float);
        pl.counters = ((size_t)(units + 1) * sizeof(unsigned) + 255) / 256 * 256;
        pl.bytes = pl.states + pl.counters;
    }
    if (K == 256) {
        pl.half = ((size_t)B * T * H * V * sizeof(float) + 255) / 256 * 256;
        pl.bytes += 2 * pl.half;
    }
    return pl;
}

template <typename Kernel>
cudaError_t launch(Kernel kern, uint32_t bytes, dim3 grid, cudaStream_t stream, const CUtensorMap (&m)[4], const Params& p) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, NTHR, bytes, stream>>>(m[0], m[1], m[2], m[3], p);
    return cudaGetLastError();
}

template <int KD, int VB, typename OT>
cudaError_t run(const DecayArgs& a) {
    using L = Layout<KD, VB>;
    constexpr bool kFine = sizeof(OT) == 4;  // a float32 output is worth 24 bits of its operands
    constexpr uint32_t kBytes = Layout<KD, VB, kFine>::BYTES;
    CUtensorMap m[4];  // q, k, v, o (a stand-in for a float32 o, which leaves by plain stores)
    const long tokens = (long)a.B * a.T;
    if (tokens == 0 && !a.hT) return cudaSuccess;
    const void* some = a.hT;  // nothing to load: the maps are never used
    if (!make_map(m, tokens ? a.q : some, tokens ? tokens : 1, a.Hk, a.K) ||
        !make_map(m + 1, tokens ? a.k : some, tokens ? tokens : 1, a.Hk, a.K) ||
        !make_map(m + 2, tokens ? a.v : some, tokens ? tokens : 1, a.H, a.V) ||
        !make_map(m + 3, tokens && !a.o_f32 ? a.o : tokens ? a.v : some, tokens ? tokens : 1, a.H, a.V))
        return cudaErrorInvalidValue;
    const Plan pl = plan(a.B, a.T, a.H, a.K, a.V, a.N, a.cu != nullptr);
    char* ws = (char*)a.ws;
    const int vblocks = (a.V + VB - 1) / VB;
    Params p{a.decay, a.per_token ? a.H : 0, a.h0, a.hT, a.cu, a.o, a.N, a.T, a.H, a.H / a.Hk, a.K, a.V, vblocks, 0, pl.seg,
             (float*)ws, (float*)(ws + pl.states), nullptr, pl.per, a.status, hook_stall_chunk()};
    dim3 grid(a.H, vblocks, pl.slots);
    cudaError_t e;
    if (pl.per) {
        p.cuts = (unsigned*)(ws + pl.states);
        grid = dim3(pl.pieces);
    }
    auto clear = [&] { return pl.per ? cudaMemsetAsync(p.cuts, 0, pl.counters, a.stream) : cudaSuccess; };
    if (pl.seg) {
        for (p.k0 = 0; p.k0 < a.K; p.k0 += KD)
            if ((e = launch(decay_chunk_kernel<KD, VB, __nv_bfloat16, true>, L::BYTES, grid, a.stream, m, p)) != cudaSuccess)
                return e;
        const int KV = a.K * a.V;
        decay_scan_kernel<<<dim3((KV / 4 + 255) / 256, a.H, a.N), 256, 0, a.stream>>>(
            a.h0, p.ws, p.wdec, ChunkMap{a.cu, a.N, a.T, pl.seg}, a.H, KV);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    p.k0 = 0;
    if (a.K == KD) {
        if ((e = clear()) != cudaSuccess) return e;
        return launch(decay_chunk_kernel<KD, VB, OT, false, kFine>, kBytes, grid, a.stream, m, p);
    }
    if constexpr (KD < 128) return cudaErrorInvalidValue;  // (a head of 256 is two of 128)
    else {
        float* half = (float*)(ws + pl.bytes - 2 * pl.half);
        for (; p.k0 < a.K; p.k0 += KD) {
            p.o = p.k0 == 0 ? half : half + pl.half / sizeof(float);
            if ((e = clear()) != cudaSuccess) return e;
            if ((e = launch(decay_chunk_kernel<KD, VB, float, false, kFine>, kBytes, grid, a.stream, m, p)) != cudaSuccess) return e;
        }
        if (tokens == 0) return cudaSuccess;
        decay_join_kernel<OT><<<8 * max(1, planned_sm_count()), 256, 0, a.stream>>>(
            half, half + pl.half / sizeof(float), (OT*)a.o, tokens, a.cu ? a.cu + a.N : nullptr, (long)a.H * a.V / 4);
        return cudaGetLastError();
    }
}

template <typename OT>
cudaError_t run_dims(const DecayArgs& a) {
    if (a.K == 64) return a.V == 64 ? run<64, 64, OT>(a) : run<64, 128, OT>(a);
    return a.V == 64 ? run<128, 64, OT>(a) : run<128, 128, OT>(a);  // (K = 256 in two halves)
}

}  // namespace decay

bool decay_tensor_dims(bool bf16, int K, int V) {
    return bf16 && (K == 64 || K == 128 || K == 256) && (V == 64 || V == 128 || V == 256);
}

size_t decay_tensor_workspace_bytes(int B, int T, int H, int K, int V, int N, bool packed) {
    return decay::plan(B, T, H, K, V, N, packed).bytes;
}

cudaError_t launch_decay_tensor(const DecayArgs& a) {
    return a.o_f32 ? decay::run_dims<float>(a) : decay::run_dims<__nv_bfloat16>(a);
}

cudaError_t read_decay_timeouts(unsigned* count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, decay::g_decay_timeouts, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(decay::g_decay_timeouts, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace kda
