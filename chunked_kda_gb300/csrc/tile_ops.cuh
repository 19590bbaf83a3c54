// What the chunked kernels of the per-head recurrences (decay_tensor.cu, delta_tensor.cu) share: operand descriptors,
// fragments of TMEM and shared-memory tiles, bf16 terms of floats, and the tensor maps of their inputs.
#pragma once

#include <cudaTypedefs.h>

#include "kda_internal.h"
#include "sm100.cuh"

namespace kda {
namespace decay {

using namespace sm100;

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

// Whole sequences of one length, more units than SMs, the last wave part-empty: the units' chunks are
// laid end to end and shared out evenly, `per` (at least a unit's nt) an SM, so a unit that does not fit into what
// is left of an SM is cut.  Its part on the next SM, which is that SM's first work, is the earlier one in time;
// the part at this SM's end runs per - nt chunks or more after the other's end and finds its state there.
// Blocks take the pieces in the order of their starts (a ticket, so that whoever waits began later than what it waits for):
// the SMs' first pieces, then the whole units, then the cut units' second pieces, the longest first (their SMs
// are free first).
constexpr int C = 64, kMaxCuts = 4096;  // tokens of a chunk; SMs that a plan is made for, at most

struct Piece {
    int unit, c0, c1;
};
// p: T, N, H, vblocks, per, and cuts, whose first word is the ticket; scratch: kMaxCuts + 2 words of shared memory
template <int NTHR, typename Params>
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

// ------------------------------------------------------------------ host side
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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
inline bool make_map(CUtensorMap* m, const void* base, long tokens, int H, int D) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    const cuuint32_t box[3] = {64, 1, 64}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Chunks of an SM where units are cut (0: they are not).  `cost`: chunks that cuts cost an SM.
inline int plan_cuts(int B, int T, int H, int vblocks, int cost) {
    const long sms = planned_sm_count(), units = (long)B * H * vblocks, nt = (T + C - 1) / C;
    if (sms <= 0 || units <= sms || units * nt > 1 << 30 || sms > kMaxCuts) return 0;
    const long waves = (units + sms - 1) / sms, per = (units * nt + sms - 1) / sms;
    return per + cost <= waves * nt ? (int)per : 0;
}

// the blocks of a launch with cut units
inline int count_pieces(int T, int units, int per) {
    const int nt = (T + C - 1) / C, firsts = (units * nt + per - 1) / per;
    int pieces = units;
    for (int m = 0; m < firsts; ++m) pieces += (long)m * per % nt != 0;
    return pieces;
}

}  // namespace decay
}  // namespace kda
