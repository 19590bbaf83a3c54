// Linear attention with a decay for each head in chunks of 64 tokens, in FP32 without tensor cores:
// float32 inputs (whose 24 bits the tensor cores' operand types do not hold) and head sizes that the
// tensor-core kernel has no instance for.
//
// Three launches, all chunks at once but for the scan:
//   1. each chunk's addition to the state, A = sum_j 2^(G_l - G_j) k_j v_j^T, and its decay 2^G_l;
//   2. the scan over a sequence's chunks: the addition's place takes the next chunk's incoming state;
//   3. each chunk's output, o_i = s (2^G_i S^T q_i + sum_{j <= i} 2^(G_i - G_j) (q_i . k_j) v_j).
// Scratch holds the additions of chunks that another one follows, at most a state for each 64 tokens however many
// sequences there are (4096 single tokens of 32 heads of 128 x 128: 135 MB): a first chunk reads the initial state, a
// last one's addition is made in the final state.  Where that is the initial state, which the outputs still read,
// the last additions are a fourth launch behind the outputs.
// The products are 64 x 64 tiles, 256 threads with 4 x 4 results each, operands in shared memory with
// the summed index outermost, so that a thread takes its four rows and its four columns as one vector
// each.  16384 tokens, 8 heads of 128 x 128 take 567 us (additions 165, scan 62, outputs 322), where the bytes would
// take 40: 98 k operations a token and head keep the FP32 pipe busy for 40 % of that and shared memory (two vectors
// for 16 multiply-adds) for 69 %; the largest stalls are its latency and that of loads, none of which is in flight
// during a product.
#include "common.cuh"
#include "decay_gates.cuh"
#include "kda_internal.h"

namespace kda {
namespace decay {
namespace {

constexpr int C = 64, NT = 256, LD = 68;  // LD: row stride of a 64-wide shared tile, 16-byte aligned

struct SimtArgs {
    const float* decay;
    int decay_stride;
    const float* h0;
    float* hT;
    ChunkMap cm;
    int H, hr, K, V;
    float* ws;    // [place][h][K][V]
    float* wdec;  // [slot][h]
    // the place of the first chunk of sequence n (its c-th chunk's is c further).  Packed: a sequence of m + 1
    // chunks needs m, and floor(eos / C) - floor(bos / C) >= m.
    __device__ size_t place(int n, int bos) const { return cm.cu ? bos / C : (size_t)n * (cm.n_slots() / cm.N - 1); }
    __device__ bool in_place() const { return hT && hT == h0; }
};

// the chunk's G as integer and fraction, and the first token without one, by warp 0 (a barrier follows)
__device__ __forceinline__ void chunk_gates(const SimtArgs& p, int h, int t0, int len, int (*sI)[C]) {
    if (threadIdx.x < 32) {
        const int l = threadIdx.x;
        auto a = [&](int i) { return i < len ? __ldg(p.decay + (size_t)(t0 + i) * p.decay_stride + h) : 0.f; };
        int I[2], F[2];
        const float a0 = a(2 * l), a1 = a(2 * l + 1);
        long long G[2];
        pair_sums(a0, a1, G);
        parts(G[0], I[0], F[0]);
        parts(G[1], I[1], F[1]);
        const int first = first_nan(a0, a1);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sI[0][2 * l + e] = I[e];
            sI[1][2 * l + e] = F[e];
        }
        if (l == 0) sI[2][0] = first;
    }
    __syncthreads();
}

// four consecutive elements of a row of n, the first at c (0 behind the row)
template <typename T>
__device__ __forceinline__ void load4(const T* row, int c, int n, float (&r)[4]) {
    if (n % 4 == 0) {
        if (c >= n) {
            r[0] = r[1] = r[2] = r[3] = 0.f;
        } else if constexpr (sizeof(T) == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(row + c));
            r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + c));
            r[0] = sm100::bf_lo(v.x); r[1] = sm100::bf_hi(v.x); r[2] = sm100::bf_lo(v.y); r[3] = sm100::bf_hi(v.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = c + e < n ? to_f32(row[c + e]) : 0.f;
    }
}
// [64 rows][nc channels from c0] of q or k, transposed: lanes are rows, so that the stores meet no bank twice
template <typename T>
__device__ __forceinline__ void load_transposed(const T* base, size_t stride, int len, int c0, int nc, int n, float* out) {
    for (int x = threadIdx.x; x < C * (nc / 4); x += NT) {
        const int i = x & 63, c = 4 * (x >> 6);
        float r[4] = {0.f, 0.f, 0.f, 0.f};
        if (i < len) load4(base + i * stride, c0 + c, n, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(c + e) * LD + i] = r[e];
    }
}
// [rows][64 columns from c0], as it is, each row times its factor
template <typename T>
__device__ __forceinline__ void load_rows(const T* base, size_t stride, int rows, int len, int c0, int n, const float* f, float* out) {
    for (int x = threadIdx.x; x < rows * 16; x += NT) {
        const int j = x >> 4, c = 4 * (x & 15);
        float r[4] = {0.f, 0.f, 0.f, 0.f};
        if (j < len) load4(base + j * stride, c0 + c, n, r);
        const float g = f ? f[j] : 1.f;
        *reinterpret_cast<float4*>(out + j * LD + c) = f && j >= len ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                                     : make_float4(r[0] * g, r[1] * g, r[2] * g, r[3] * g);
    }
}

// [32 rows from j0][64 columns from c0] of v.  A masked score is 0, and 0 times a value that is not finite is NaN:
// such values are left out, and the first row of each column that has one is noted.
template <typename T>
__device__ __forceinline__ void load_values(const T* base, size_t stride, int j0, int len, int c0, int n, int* first, float* out) {
    for (int x = threadIdx.x; x < 32 * 16; x += NT) {
        const int j = j0 + (x >> 4), c = 4 * (x & 15);
        float r[4] = {0.f, 0.f, 0.f, 0.f};
        if (j < len) load4(base + j * stride, c0 + c, n, r);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (!(fabsf(r[e]) < __int_as_float(0x7f800000))) {
                r[e] = 0.f;
                atomicMin(first + c + e, j);
            }
        *reinterpret_cast<float4*>(out + (x >> 4) * LD + c) = make_float4(r[0], r[1], r[2], r[3]);
    }
}

// acc[i][j] += sum_{x < n} A[x][4 ti + i] B[x][4 tj + j]
__device__ __forceinline__ void tile_product(const float* A, const float* B, int n, int ti, int tj, float (&acc)[4][4]) {
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
        const float4 a = *reinterpret_cast<const float4*>(A + x * LD + 4 * ti);
        const float4 b = *reinterpret_cast<const float4*>(B + x * LD + 4 * tj);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
}

// grid (slots, H, K blocks x V blocks of 64).  kLast: the last chunks alone, a slot for each sequence, onto their
// decayed incoming states (which may be the initial ones, in place).
template <typename T, bool kLast>
__global__ void __launch_bounds__(NT) decay_add_kernel(const T* __restrict__ k, const T* __restrict__ v, SimtArgs p) {
    __shared__ __align__(16) float sk[C * LD], sv[C * LD];
    __shared__ float sf[C];
    __shared__ int sI[3][C];
    int n, t0, len, bos, eos;
    if constexpr (kLast) {
        n = blockIdx.x;
        if (p.cm.cu) { bos = __ldg(p.cm.cu + n); eos = __ldg(p.cm.cu + n + 1); }
        else         { bos = n * p.cm.T; eos = bos + p.cm.T; }
        if (bos == eos) return;  // its state is where it was
        t0 = bos + (eos - bos - 1) / C * C;
        len = eos - t0;
    } else {
        if (!p.cm.map_first(blockIdx.x, n, t0, len, bos, eos)) return;
        if (t0 + len >= eos && (!p.hT || p.in_place())) return;
    }
    const bool last = t0 + len >= eos;
    const int h = blockIdx.y, nkb = (p.K + 63) / 64, c0 = 64 * (blockIdx.z % nkb), d0 = 64 * (blockIdx.z / nkb);
    const int tid = threadIdx.x;
    chunk_gates(p, h, t0, len, sI);
    const float poison = nan_if(sI[2][0] < C);
    const int Hk = p.H / p.hr, hq = h / p.hr;
    if (tid < C) sf[tid] = pow2(sI[0][C - 1] - sI[0][tid], sI[1][C - 1] - sI[1][tid]) + poison;
    __syncthreads();
    load_rows(k + ((size_t)t0 * Hk + hq) * p.K, (size_t)Hk * p.K, C, len, c0, p.K, sf, sk);
    load_rows(v + ((size_t)t0 * p.H + h) * p.V, (size_t)p.H * p.V, C, len, d0, p.V, nullptr, sv);
    __syncthreads();
    const int ti = tid >> 4, tj = tid & 15;
    float acc[4][4] = {};
    tile_product(sk, sv, C, ti, tj, acc);
    const size_t KV = (size_t)p.K * p.V, at = p.place(n, bos) + (t0 - bos) / C;
    float* out = last ? p.hT + ((size_t)n * p.H + h) * KV : p.ws + (at * p.H + h) * KV;
    const float* in = !kLast ? nullptr : t0 == bos ? out : p.ws + ((at - 1) * p.H + h) * KV;
    const float decay = pow2(max(sI[0][C - 1], -300), sI[1][C - 1]) + poison;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + 4 * ti + i, d = d0 + 4 * tj + j;
            if (c >= p.K || d >= p.V) continue;
            const size_t e = (size_t)c * p.V + d;
            out[e] = kLast ? fmaf(decay, in[e], acc[i][j]) : acc[i][j];
        }
    if (!kLast && tid == 0 && blockIdx.z == 0) p.wdec[(size_t)blockIdx.x * p.H + h] = decay;
}

// grid (blocks of 256 state elements, H, sequences): the chunks' incoming states, and the final one
__global__ void __launch_bounds__(NT) decay_chunk_scan_kernel(SimtArgs p) {
    const int n = blockIdx.z, h = blockIdx.y, KV = p.K * p.V, e = blockIdx.x * NT + threadIdx.x;
    if (e >= KV) return;
    int bos, eos;
    if (p.cm.cu) { bos = __ldg(p.cm.cu + n); eos = __ldg(p.cm.cu + n + 1); }
    else         { bos = n * p.cm.T; eos = bos + p.cm.T; }
    const int ns = (eos - bos + C - 1) / C;
    const size_t st = ((size_t)n * p.H + h) * KV + e;
    float S = p.h0 ? p.h0[st] : 0.f;
    const int s0 = ns > 0 ? p.cm.first_slot(n, bos) : 0;
    float* at = p.ws + (p.place(n, bos) * p.H + h) * KV + e;
    const size_t step = (size_t)p.H * KV;
    // (eight chunks' additions are loaded before the first is used)
    constexpr int U = 8;
    for (int s = 0; s + 1 < ns; s += U) {
        float add[U], dec[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u + 1 < ns;
            add[u] = in ? at[(s + u) * step] : 0.f;
            dec[u] = in ? __ldg(p.wdec + (size_t)(s0 + s + u) * p.H + h) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u + 1 >= ns) break;
            S = fmaf(dec[u], S, add[u]);
            at[(s + u) * step] = S;
        }
    }
    if (p.hT && !p.in_place()) p.hT[st] = ns > 0 ? fmaf(__ldg(p.wdec + (size_t)(s0 + ns - 1) * p.H + h), S, p.hT[st]) : S;
}

// grid (slots, H): the chunk's output, all its value channels
template <typename T, typename OT>
__global__ void __launch_bounds__(NT) decay_out_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                       const T* __restrict__ v, OT* __restrict__ o, SimtArgs p) {
    extern __shared__ __align__(16) float sm[];
    const int Kp = (p.K + 31) / 32 * 32;
    float* sq = sm;               // [Kp][LD] q, transposed
    float* sp = sq + Kp * LD;     // [64][LD] P, transposed
    float* sx = sp + C * LD;      // [32][LD] a slice of k (transposed), S or v
    __shared__ int sI[3][C], s_odd[64];
    int n, t0, len, bos, eos;
    if (!p.cm.map_first(blockIdx.x, n, t0, len, bos, eos)) return;
    const int h = blockIdx.y, tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    chunk_gates(p, h, t0, len, sI);
    const int bad = sI[2][0];
    const int Hk = p.H / p.hr, hq = h / p.hr;
    const float scale = rsqrtf((float)p.K);
    load_transposed(q + ((size_t)t0 * Hk + hq) * p.K, (size_t)Hk * p.K, len, 0, Kp, p.K, sq);
    {
        float acc[4][4] = {};
        for (int c0 = 0; c0 < Kp; c0 += 32) {
            __syncthreads();
            load_transposed(k + ((size_t)t0 * Hk + hq) * p.K, (size_t)Hk * p.K, len, c0, 32, p.K, sx);
            __syncthreads();
            tile_product(sq + c0 * LD, sx, 32, ti, tj, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 4 * ti + i, s = 4 * tj + j;
                float y = 0.f;
                if (s <= r) y = acc[i][j] * (pow2(sI[0][r] - sI[0][s], sI[1][r] - sI[1][s]) + nan_if(r >= bad));
                sp[s * LD + r] = y;
            }
    }
    const size_t KV = (size_t)p.K * p.V;
    const float* S = t0 > bos ? p.ws + ((p.place(n, bos) + (t0 - bos) / C - 1) * p.H + h) * KV
                     : p.h0 ? p.h0 + ((size_t)n * p.H + h) * KV : nullptr;
    for (int d0 = 0; d0 < p.V; d0 += 64) {
        float acc[4][4] = {};
        if (!S) __syncthreads();
        for (int c0 = 0; c0 < Kp && S; c0 += 32) {
            __syncthreads();
            load_rows(S + (size_t)c0 * p.V, p.V, 32, p.K - c0, d0, p.V, nullptr, sx);
            __syncthreads();
            tile_product(sq + c0 * LD, sx, 32, ti, tj, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = pow2(sI[0][4 * ti + i], sI[1][4 * ti + i]) + nan_if(4 * ti + i >= bad);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= f;
        }
        if (tid < 64) s_odd[tid] = C;  // (the products' barriers lie behind the last block's reads)
        for (int j0 = 0; j0 < C; j0 += 32) {
            __syncthreads();
            load_values(v + ((size_t)t0 * p.H + h) * p.V, (size_t)p.H * p.V, j0, len, d0, p.V, s_odd, sx);
            __syncthreads();
            tile_product(sp + j0 * LD, sx, 32, ti, tj, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ti + i;
            if (r >= len) continue;
            OT* dst = o + ((size_t)(t0 + r) * p.H + h) * p.V + d0 + 4 * tj;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (d0 + 4 * tj + j < p.V) dst[j] = from_f32<OT>(acc[i][j] * scale + nan_if(r >= s_odd[4 * tj + j]));
        }
    }
}

// chunks that another one follows, at most
int places(int T, int N, bool packed) { return packed ? T / C : N * max(0, (T + C - 1) / C - 1); }
size_t state_bytes(int places, int H, int K, int V) { return ((size_t)places * H * K * V * 4 + 255) / 256 * 256; }

template <typename T, typename OT>
cudaError_t run(const DecayArgs& a) {
    const ChunkMap cm{a.cu, a.N, a.T, C};
    const int slots = cm.n_slots();
    SimtArgs p{a.decay, a.per_token ? a.H : 0, a.h0, a.hT, cm, a.H, a.H / a.Hk, a.K, a.V, (float*)a.ws,
               (float*)((char*)a.ws + state_bytes(places(a.T, a.N, a.cu), a.H, a.K, a.V))};
    cudaError_t e;
    const int tiles = ((a.K + 63) / 64) * ((a.V + 63) / 64);
    if (slots > 0) {
        decay_add_kernel<T, false><<<dim3(slots, a.H, tiles), NT, 0, a.stream>>>((const T*)a.k, (const T*)a.v, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    decay_chunk_scan_kernel<<<dim3((a.K * a.V + NT - 1) / NT, a.H, a.N), NT, 0, a.stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (slots > 0) {
        auto kern = decay_out_kernel<T, OT>;
        const int bytes = ((a.K + 31) / 32 * 32 + C + 32) * LD * (int)sizeof(float);
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
        kern<<<dim3(slots, a.H), NT, bytes, a.stream>>>((const T*)a.q, (const T*)a.k, (const T*)a.v, (OT*)a.o, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (a.hT && a.hT == a.h0) {
            decay_add_kernel<T, true><<<dim3(a.N, a.H, tiles), NT, 0, a.stream>>>((const T*)a.k, (const T*)a.v, p);
            e = cudaGetLastError();
        }
    }
    return e;
}

}  // namespace
}  // namespace decay

size_t decay_simt_workspace_bytes(int B, int T, int H, int K, int V, int N, bool packed) {
    const int slots = packed ? T / decay::C + N + 1 : N * ((T + decay::C - 1) / decay::C);
    return decay::state_bytes(decay::places(T, N, packed), H, K, V) + ((size_t)slots * H * 4 + 255) / 256 * 256;
}

cudaError_t launch_decay_simt(const DecayArgs& a) {
    if (!a.qkv_bf16) return decay::run<float, float>(a);
    return a.o_f32 ? decay::run<__nv_bfloat16, float>(a) : decay::run<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace kda
