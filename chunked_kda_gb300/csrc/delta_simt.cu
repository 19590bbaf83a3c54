// The gated delta rule with a decay for each head in chunks of 64 tokens, in FP32 without tensor cores: float32
// inputs (whose 24 bits the tensor cores' operand types do not hold), float32 outputs of bf16 inputs, and head sizes
// that the tensor-core kernel does not take.
//
// G_i the decay's sum up to and including row i of a chunk, l its last row, s = 1/sqrt(K), S the incoming state:
//   A_ij = beta_i e^(G_i - G_j) k_i . k_j (j < i),   T = (1 + A)^-1 diag(beta)
//   U = T (V - diag(e^G) K S),   O = s (diag(e^G) Q S + (e^(G_i - G_j) q_i . k_j)_{j <= i} U)
//   S <- e^G_l S + K^T diag(e^(G_l - G_j)) U
// Two launches:
//   1. per chunk and head, all at once: T, the masked scores P and the rows' factors, into scratch: a row of kRow
//      floats for each token and head, so that it does not grow with the number of sequences;
//   2. per (sequence, head, block of VB value columns), chunks in order: the state in shared memory.
// The value columns are independent of one another, so with few heads narrow blocks fill the SMs.
// A masked element is 0, and 0 times a value that is not finite is NaN: the triangular products leave out what is
// masked instead, so nothing reaches back.
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

constexpr int C = 64, NT = 256, LD = 68;  // LD: row stride of a 64-wide shared tile, 16-byte aligned
// a token's row in scratch: T's row, P's row, then e^G_i / |k_i|, s e^G_i / |q_i|, e^(G_l - G_i) / |k_i| and e^G_l
// (the norms where they are asked for)
constexpr int kRow = 2 * C + 4, kFactors = 2 * C;

struct Args {
    Gates gates;
    const float* h0;
    float* hT;
    ChunkMap cm;
    int H, hr, K, V;
    unsigned flags;
    float* ws;
};

// four elements as they lie in memory
template <typename T>
struct Four {
    T e[4];
};
template <typename T>
__device__ __forceinline__ Four<T> four(const T* p) {  // aligned to the four
    Four<T> r;
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(&r) = *reinterpret_cast<const float4*>(p);
    else                          *reinterpret_cast<uint2*>(&r) = *reinterpret_cast<const uint2*>(p);
    return r;
}
template <typename T>
__device__ __forceinline__ float4 floats(const Four<T>& r) {
    return make_float4(to_f32(r.e[0]), to_f32(r.e[1]), to_f32(r.e[2]), to_f32(r.e[3]));
}
// four consecutive elements of a row of n, the first at c (0 behind the row)
template <typename T>
__device__ __forceinline__ Four<T> load4(const T* row, int c, int n) {
    Four<T> r{};
    if (n % 4 == 0) {
        if (c < n) r = four(row + c);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < n) r.e[e] = row[c + e];
    }
    return r;
}
// A thread's share (of 256 threads') of a [64 rows][NC channels from c0] tile: asked for as it lies in memory, put down transposed.  A warp
// has eight rows and sixteen channels at a time: whole sectors of few lines (a row a lane read 32 lines a load), and no
// more than two stores to a bank.
template <typename T, int NC>
struct Tile {
    static constexpr int N = NC / 16;
    static_assert(NT == 4 * C, "");
    Four<T> r[N];
    static __device__ __forceinline__ int row() { return (threadIdx.x & 7) + 8 * (threadIdx.x >> 5 & 7); }
    static __device__ __forceinline__ int channel(int x) { return 4 * (threadIdx.x >> 3 & 3) + 16 * x; }
    __device__ __forceinline__ void fetch(const T* base, size_t stride, int len, int n, int c0 = 0) {
        const int i = row();
#pragma unroll
        for (int x = 0; x < N; ++x) {
            r[x] = Four<T>{};
            if (i < len) r[x] = load4(base + i * stride, c0 + channel(x), n);
        }
    }
    template <typename S>
    __device__ __forceinline__ void put(S* out) const {  // as it is, or as floats
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(S) == sizeof(T)) out[(channel(x) + e) * LD + row()] = r[x].e[e];
                else                                  out[(channel(x) + e) * LD + row()] = to_f32(r[x].e[e]);
            }
    }
};

// X = (1 + A)^-1 of a strictly lower triangular 64 x 64 matrix whose rows from len on are 0, by all threads; Y: 32 x 33 floats between.  The diagonal
// blocks of 16 by substitution, a column a thread, then twice the block below two inverted ones: -X22 (A21 X11).
__device__ __forceinline__ void invert(const float* A, float* X, float* Y, int len) {
    const int tid = threadIdx.x;
    for (int x = tid; x < C * LD; x += NT) X[x] = 0.f;
    __syncthreads();
    if (tid < 64) {
        const int b = tid & ~15, c = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == c ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m)
                if (m >= c) y = fmaf(-A[(b + i) * LD + b + m], x[m], y);
            x[i] = i >= c ? y : 0.f;
            X[(b + i) * LD + b + c] = x[i];
        }
    }
    for (int w = 16; w < C; w *= 2) {
        for (int o = 0; o + w < len; o += 2 * w) {  // (else the block below is 0)
            __syncthreads();
            for (int x = tid; x < w * w; x += NT) {
                const int i = x / w, c = x % w;
                float y = 0.f;
                for (int m = c; m < w; ++m) y = fmaf(A[(o + w + i) * LD + o + m], X[(o + m) * LD + o + c], y);
                Y[i * 33 + c] = y;
            }
            __syncthreads();
            for (int x = tid; x < w * w; x += NT) {
                const int i = x / w, c = x % w;
                float y = 0.f;
                for (int m = 0; m <= i; ++m) y = fmaf(X[(o + w + i) * LD + o + w + m], Y[m * 33 + c], y);
                X[(o + w + i) * LD + o + c] = -y;
            }
        }
    }
    __syncthreads();
}

// grid (slots, H)
template <typename T>
__global__ void __launch_bounds__(NT) delta_prep_kernel(const T* __restrict__ q, const T* __restrict__ k, Args p) {
    __shared__ __align__(16) float sk[C * LD], sq[C * LD];  // 64 channels of k and q, transposed; then A and its inverse
    __shared__ float sy[32 * 33], s_beta[C], s_nk[C], s_nq[C];
    __shared__ int sI[2][C], s_bad;
    int n, t0, len, bos, eos;
    if (!p.cm.map(blockIdx.x, n, t0, len, bos, eos)) return;
    const int h = blockIdx.y, tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    if (tid < 32) {
        const Gates::Head head = p.gates.head(h);
        const int i0 = 2 * tid;
        const float a0 = i0 < len ? p.gates.decay(t0 + i0, h, head) : 0.f;
        const float a1 = i0 + 1 < len ? p.gates.decay(t0 + i0 + 1, h, head) : 0.f;
        long long G[2];
        pair_sums(a0, a1, G);
        const int bad = first_nan(a0, a1);
#pragma unroll
        for (int e = 0; e < 2; ++e) parts(G[e], sI[0][i0 + e], sI[1][i0 + e]);
        if (tid == 0) s_bad = bad;
    } else if (tid < 32 + C) {
        const int i = tid - 32;
        s_beta[i] = i < len ? p.gates.rate(t0 + i, h) : 0.f;
    }
    const int Hk = p.H / p.hr, hq = h / p.hr;
    const T* kb = k + ((size_t)t0 * Hk + hq) * p.K;
    const T* qb = q + ((size_t)t0 * Hk + hq) * p.K;
    float kk[4][4] = {}, qk[4][4] = {}, nq = 0.f;
    for (int c0 = 0; c0 < p.K; c0 += 64) {
        Tile<T, C> tk, tq;
        tk.fetch(kb, (size_t)Hk * p.K, len, p.K, c0);
        tq.fetch(qb, (size_t)Hk * p.K, len, p.K, c0);
        __syncthreads();
        tk.put(sk);
        tq.put(sq);
        __syncthreads();
        if (4 * ti < len)
#pragma unroll 4
        for (int c = 0; c < 64; ++c) {
            const float4 a = *reinterpret_cast<const float4*>(sk + c * LD + 4 * ti);
            const float4 b = *reinterpret_cast<const float4*>(sq + c * LD + 4 * ti);
            const float4 d = *reinterpret_cast<const float4*>(sk + c * LD + 4 * tj);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    kk[i][j] = fmaf(av[i], dv[j], kk[i][j]);
                    qk[i][j] = fmaf(bv[i], dv[j], qk[i][j]);
                }
        }
        if (tid < C && (p.flags & KDA_FLAG_Q_L2NORM))
            for (int c = 0; c < 64; ++c) nq = fmaf(sq[c * LD + tid], sq[c * LD + tid], nq);
    }
    if (tid < C) s_nq[tid] = p.flags & KDA_FLAG_Q_L2NORM ? row_norm(nq) : 1.f;
    if (ti == tj)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_nk[4 * ti + i] = p.flags & KDA_FLAG_K_L2NORM ? row_norm(kk[i][i]) : 1.f;
    __syncthreads();
    const float scale = rsqrtf((float)p.K);
    const int bad = s_bad;
    float* row0 = p.ws + ((size_t)t0 * p.H + h) * kRow;
    const size_t stride = (size_t)p.H * kRow;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ti + i;
        float out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 4 * tj + j;
            float a = 0.f, x = 0.f;
            if (c <= r) {
                const float f = s_nk[c] * pow2(sI[0][r] - sI[0][c], sI[1][r] - sI[1][c]) + nan_if(r >= bad);
                x = scale * s_nq[r] * f * qk[i][j];
                a = c < r ? s_beta[r] * s_nk[r] * f * kk[i][j] : 0.f;
            }
            sk[r * LD + c] = a;
            out[j] = x;
        }
        if (r < len) *reinterpret_cast<float4*>(row0 + r * stride + C + 4 * tj) = make_float4(out[0], out[1], out[2], out[3]);
    }
    if (tid < len) {
        const float poison = nan_if(tid >= bad), e = pow2(sI[0][tid], sI[1][tid]) + poison;
        *reinterpret_cast<float4*>(row0 + tid * stride + kFactors) =
            make_float4(e * s_nk[tid], scale * e * s_nq[tid],
                        (pow2(sI[0][C - 1] - sI[0][tid], sI[1][C - 1] - sI[1][tid]) + nan_if(bad < C)) * s_nk[tid],
                        pow2(sI[0][C - 1], sI[1][C - 1]) + nan_if(bad < C));
    }
    __syncthreads();
    invert(sk, sq, sy, len);
    for (int x = tid; x < C * 16; x += NT) {
        const int r = x >> 4, c = 4 * (x & 15);
        if (r >= len) break;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = c + j <= r ? sq[r * LD + c + j] * s_beta[c + j] : 0.f;
        *reinterpret_cast<float4*>(row0 + r * stride + c) = make_float4(y[0], y[1], y[2], y[3]);
    }
}

// [n][W] columns from a pair of shared vectors
template <int W>
__device__ __forceinline__ void lds_row(const float* p, float (&r)[W]) {
    if constexpr (W == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
    } else if constexpr (W == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        r[0] = x.x; r[1] = x.y;
    } else {
        r[0] = *p;
    }
}

// grid (V blocks, H, sequences).  Two groups of 256 threads: the first has K S, U and the state, the second Q S, P U and the
// output; a thread four rows of a chunk and W of the block's VB = 16 W columns.  Kp: K rounded up to 64, 128 or 256.  The
// next chunk is on its way into registers while this one is worked on.  o may be v, so neither is __restrict__: a block reads
// its columns of a chunk's values before it writes them, and no other block has them.
//
// Loads from shared memory bound it (70 to 73 % of their rate, of L1's 82 to 88): 16 multiply-adds take eight floats a
// thread.  W = 4 where such blocks fill the SMs, fewer where not.  Times of a call (heads of 128 x 128): float32, 4 x 4096 tokens,
// 32 heads 3.2 ms (W = 2: 4.1); 16384 tokens, 8 heads 2.9 (each chunk fetched when its turn came: 4.8); 2048 tokens, 64 heads
// 1.0, of which 0.2 the first kernel; 128 tokens, 2 heads of 64 x 64 31 us.  bf16 with float32 output, 4 x 4096 tokens, 64
// heads 6.4 ms (one group with four columns a thread 7.6, with two 9.5); of 256 x 256, 8 x 2048 tokens, 32 heads 9.7
// (11.2, 13.7).  Short chunks leave out the rows that are none (36 sequences of 7 tokens, 83 heads of 128 x 256: 0.86 ms, with
// all rows 1.96).  In FP32 multiply-adds alone the first would be 0.9 ms.
template <typename T, typename OT, int W, int Kp>
__global__ void __launch_bounds__(2 * NT) delta_chain_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                             const T* v, OT* o, Args p) {
    constexpr int VB = 16 * W;
    extern __shared__ __align__(16) float sm[];
    float* st = sm;               // [64][LD] T, transposed
    float* sp = st + C * LD;      // [64][LD] P
    float* sS = sp + C * LD;      // [Kp][VB]
    float* su = sS + Kp * VB;     // [64][VB] U
    float* sr = su + C * VB;      // [64][VB] V - diag(e^G) K S, then U with the factors of the state
    float* sf = sr + C * VB;      // [64][4] factors
    T* sk = reinterpret_cast<T*>(sf + 4 * C);  // [Kp][LD] k, transposed
    T* sq = sk + Kp * LD;                      // [Kp][LD] q
    const bool second = threadIdx.x >= NT;
    const int tid = threadIdx.x & (NT - 1), ti = tid >> 4, tj = tid & 15;
    const int v0 = blockIdx.x * VB, h = blockIdx.y, n = blockIdx.z;
    int bos, eos;
    if (p.cm.cu) { bos = __ldg(p.cm.cu + n); eos = __ldg(p.cm.cu + n + 1); }
    else         { bos = n * p.cm.T; eos = bos + p.cm.T; }
    const int Hk = p.H / p.hr, hq = h / p.hr, col = v0 + W * tj;
    const size_t state = ((size_t)n * p.H + h) * (size_t)p.K * p.V;
    constexpr int S = Kp * VB / (2 * NT);
    float s0[S];  // (all asked for before the first is put down)
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int x = threadIdx.x + 2 * NT * i, c = x / VB, d = v0 + x % VB;
        s0[i] = p.h0 && c < p.K && d < p.V ? p.h0[state + (size_t)c * p.V + d] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) sS[threadIdx.x + 2 * NT * i] = s0[i];
    const T* mine = second ? q : k;
    T* sx = second ? sq : sk;
    float* sl = second ? sp : st;
    Tile<T, Kp> tx;
    Tile<float, C> tt;
    T vr[4][W];
    float factor = 0.f;
    auto fetch = [&](int t0) {
        const int len = min(C, eos - t0);
        const float* ws = p.ws + ((size_t)t0 * p.H + h) * kRow;
        tx.fetch(mine + ((size_t)t0 * Hk + hq) * p.K, (size_t)Hk * p.K, len, p.K);
        tt.fetch(ws + (second ? C : 0), (size_t)p.H * kRow, len, C);
        if (second) {
            factor = (tid >> 2) < len ? ws[(size_t)(tid >> 2) * p.H * kRow + kFactors + (tid & 3)] : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e)
                    vr[i][e] = 4 * ti + i < len && col + e < p.V ? v[((size_t)(t0 + 4 * ti + i) * p.H + h) * p.V + col + e] : T(0.f);
        }
    };
    auto lower = [&](const float* M, const float* B, float (&r)[4][W]) {  // r_i += sum_{j <= i} M_ij B_j
#pragma unroll 2
        for (int j0 = 0; j0 < 4 * ti; j0 += 4)
#pragma unroll
            for (int j = j0; j < j0 + 4; ++j) {
                const float4 a = *reinterpret_cast<const float4*>(M + j * LD + 4 * ti);
                float b[W];
                lds_row<W>(B + j * VB + W * tj, b);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    r[0][e] = fmaf(a.x, b[e], r[0][e]);
                    r[1][e] = fmaf(a.y, b[e], r[1][e]);
                    r[2][e] = fmaf(a.z, b[e], r[2][e]);
                    r[3][e] = fmaf(a.w, b[e], r[3][e]);
                }
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float b[W];
            lds_row<W>(B + (4 * ti + j) * VB + W * tj, b);
#pragma unroll
            for (int i = j; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e) r[i][e] = fmaf(M[(4 * ti + j) * LD + 4 * ti + i], b[e], r[i][e]);
        }
    };
    if (bos < eos) fetch(bos);
    for (int t0 = bos; t0 < eos; t0 += C) {
        const int len = min(C, eos - t0);
        tx.put(sx);
        tt.put(sl);
        if (second) sf[tid] = factor;
        float vv[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) vv[i][e] = second ? 0.f : to_f32(vr[i][e]);
        if (t0 + C < eos) fetch(t0 + C);
        __syncthreads();
        float y[4][W] = {};  // K S or Q S
        const bool rows = 4 * ti < len;  // (short chunks: the other warps have nothing to do)
        if (rows)
#pragma unroll 8
        for (int c = 0; c < Kp; ++c) {
            const float4 a = floats(four(sx + c * LD + 4 * ti));
            float s[W];
            lds_row<W>(sS + c * VB + W * tj, s);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                y[0][e] = fmaf(a.x, s[e], y[0][e]);
                y[1][e] = fmaf(a.y, s[e], y[1][e]);
                y[2][e] = fmaf(a.z, s[e], y[2][e]);
                y[3][e] = fmaf(a.w, s[e], y[3][e]);
            }
        }
        if (second) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e) y[i][e] *= sf[4 * (4 * ti + i) + 1];
            __syncthreads();  // (sr below has been read, su and sr written)
            if (rows) lower(sp, su, y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (4 * ti + i < len && col + e < p.V)
                        o[((size_t)(t0 + 4 * ti + i) * p.H + h) * p.V + col + e] = from_f32<OT>(y[i][e]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    sr[(4 * ti + i) * VB + W * tj + e] = fmaf(-sf[4 * (4 * ti + i)], y[i][e], vv[i][e]);
                    y[i][e] = 0.f;
                }
            bar_sync(1, NT);
            if (rows) lower(st, sr, y);
            bar_sync(1, NT);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    su[(4 * ti + i) * VB + W * tj + e] = y[i][e];
                    sr[(4 * ti + i) * VB + W * tj + e] = 4 * ti + i < len ? y[i][e] * sf[4 * (4 * ti + i) + 2] : 0.f;
                }
            __syncthreads();  // (the second group has read the state)
            const float last = sf[3];
            for (int c0 = 4 * ti; c0 < Kp; c0 += 64) {
                float add[4][W] = {};
#pragma unroll 2
                for (int j = 0; j < len; j += 4) {
                    float u[4][W];
#pragma unroll
                    for (int x = 0; x < 4; ++x) lds_row<W>(sr + (j + x) * VB + W * tj, u[x]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 a = floats(four(sk + (c0 + i) * LD + j));
#pragma unroll
                        for (int e = 0; e < W; ++e) {
                            add[i][e] = fmaf(a.x, u[0][e], add[i][e]);
                            add[i][e] = fmaf(a.y, u[1][e], add[i][e]);
                            add[i][e] = fmaf(a.z, u[2][e], add[i][e]);
                            add[i][e] = fmaf(a.w, u[3][e], add[i][e]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        float* s = sS + (c0 + i) * VB + W * tj + e;
                        *s = fmaf(last, *s, add[i][e]);
                    }
            }
        }
        __syncthreads();
    }
    if (!p.hT) return;
    __syncthreads();  // (an empty sequence's state passes through)
    for (int x = threadIdx.x; x < Kp * VB; x += 2 * NT) {
        const int c = x / VB, d = v0 + x % VB;
        if (c < p.K && d < p.V) p.hT[state + (size_t)c * p.V + d] = sS[x];
    }
}

template <typename T, typename OT, int W, int Kp>
cudaError_t run_chain_k(const DeltaArgs& a, const Args& p) {
    constexpr int VB = 16 * W, bytes = 2 * Kp * LD * (int)sizeof(T) + (2 * C * LD + Kp * VB + 2 * C * VB + 4 * C) * (int)sizeof(float);
    auto kern = delta_chain_kernel<T, OT, W, Kp>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<dim3((a.V + VB - 1) / VB, a.H, a.N), 2 * NT, bytes, a.stream>>>((const T*)a.q, (const T*)a.k, (const T*)a.v, (OT*)a.o, p);
    return cudaGetLastError();
}
template <typename T, typename OT, int W>
cudaError_t run_chain(const DeltaArgs& a, const Args& p) {
    if (a.K <= 64) return run_chain_k<T, OT, W, 64>(a, p);
    if (a.K <= 128) return run_chain_k<T, OT, W, 128>(a, p);
    // (four columns a thread do not fit shared memory with keys of 256 floats)
    return run_chain_k<T, OT, sizeof(T) == 4 ? W < 2 ? W : 2 : W, 256>(a, p);
}

template <typename T, typename OT>
cudaError_t run(const DeltaArgs& a) {
    const ChunkMap cm{a.cu, a.N, a.T, C};
    const Args p{Gates(a), a.h0, a.hT, cm, a.H, a.H / a.Hk, a.K, a.V, a.flags, (float*)a.ws};
    if (a.T > 0) {
        delta_prep_kernel<T><<<dim3(cm.n_slots(), a.H), NT, 0, a.stream>>>((const T*)a.q, (const T*)a.k, p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    int dev = 0, sms = 1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long units = (long)a.N * a.H;
    if (units * ((a.V + 63) / 64) >= sms) return run_chain<T, OT, 4>(a, p);
    return units * ((a.V + 31) / 32) >= sms ? run_chain<T, OT, 2>(a, p) : run_chain<T, OT, 1>(a, p);
}

}  // namespace
}  // namespace delta

size_t delta_simt_workspace_bytes(int B, int T, int H) {
    return ((size_t)B * T * H * delta::kRow * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_delta_simt(const DeltaArgs& a) {
    if (a.N == 0) return cudaSuccess;
    if (!a.qkv_bf16) return delta::run<float, float>(a);
    return a.o_f32 ? delta::run<__nv_bfloat16, float>(a) : delta::run<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace kda
