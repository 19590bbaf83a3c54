// The gated delta rule with a decay for each head, token by token (decode, short prompts).
//
// Per (sequence, head), state S (K x V, rows = key channels) in FP32, g = e^a:
//   u = beta (v - g S^T k);   o = (g S^T q + (q . k) u) / sqrt(K);   S = g S + k u^T,
// the rule's decay, correction and read-out with the new state's read-out written out, so that one pass over
// the old state gives both products.
//
// Memory bounds it: the state goes in and out once.  Two kernels, the second for what does not fit the first:
//
// Rows of whole vectors (V a multiple of 4): a block has a (sequence, head) and all rows of as many value columns as make
// 64 KB, in shared memory, which one copy brings and takes away: a bulk copy where that is the whole state, else a
// tensor map's box (a bulk copy for each row took twice the time: 256 sequences of one token, 32 heads of 128 x 256 454 us,
// with boxes 317).  192 KB an SM are under way without a register.  A thread has four columns and every
// (4 threads / columns)-th row; the products are joined through shared memory.  (The state in registers, with the rows split over
// eight warps whose sums meet at a barrier before the first store: 377 us for 512 sequences of one token, 32 heads of 128 x 128;
// without the barrier, a warp with 16 columns of all rows: 424, its rows' pieces of 64 bytes are too short.)  That call
// moves 2.16 GB in 317 us, 6.8 TB/s, as a plain copy does; heads of 256 x 256 are at 98 % of it, 96 x 96 97, 64 x 64 91,
// 234 x 128 89.  Each further token costs a pass over shared memory (4 tokens: 736 us), so that from about eight on the
// chunked kernels are faster (64 sequences of 16 tokens, bf16: 358, chunked 173).
//
// V not a multiple of 4: the same with two columns or one a thread, where a state fits shared memory whole (128 x 126: 99 % of
// a copy's rate, 100 x 253 82, 99 x 77 75).  Larger ones (K from 212 on): a warp has eight columns with all rows in registers, sixteen
// pairs of lanes with 16 rows each (rows and columns beyond K and V masked), joined by shuffles; its rows begin at any
// four bytes, and single loads are what bounds it (236 x 253: 27 %).
#include "common.cuh"
#include "delta_gates.cuh"
#include "kda_internal.h"
#include "sm100.cuh"
#include "tile_ops.cuh"

namespace kda {
namespace delta {
namespace {

using namespace sm100;

__device__ unsigned int g_token_timeouts = 0;

constexpr int kTile = 16384;   // floats of a block's state, at most
constexpr int kWhole = 54000;  // ... where rows are not whole vectors, so that a state cannot be parted

template <int E>
struct alignas(4 * E) Columns {
    float e[E];
};

// o may be v, so neither is __restrict__: all reads of a token's values are in front of the barrier behind which one thread
// writes its output there.
// BV: columns of a block, E those of a thread.  All of V: a block's rows lie side by side; else they come and go by the
// tensor maps.
template <typename InT, typename OutT, int NT, int E>
__global__ void __launch_bounds__(NT, 768 / NT) delta_token_kernel(
    const __grid_constant__ CUtensorMap tm_in, const __grid_constant__ CUtensorMap tm_out, const InT* __restrict__ q,
    const InT* __restrict__ k, const InT* v, Gates gates, unsigned flags, const float* h0, float* hT,
    const int32_t* __restrict__ cu, int T, int H, int hr, int K, int V, int BV, OutT* o, int* status, bool stall) {
    constexpr int kPart = E * NT;  // partial S^T k, then S^T q, a row of a block's columns for each group of threads
    extern __shared__ __align__(128) float sm[];  // the partial products, [K][BV] the state
    __shared__ float s_q[256], s_k[256], s_dot[3][NT / 32];
    __shared__ __align__(8) uint64_t s_bar[2];  // the state's, and one that nothing completes
    float* part = sm;
    const int tid = threadIdx.x, v0 = blockIdx.x * BV, h = blockIdx.y, n = blockIdx.z, cols = min(BV, V - v0);
    const uint32_t bar = smem_u32(s_bar);
    const size_t st = ((size_t)n * H + h) * (size_t)K * V + v0;
    // a whole state may begin and end inside a bulk copy's 16 bytes: its first and last floats go one by one
    const int off = E == 4 ? 0 : (int)(st & 3), edge = min((4 - off) & 3, K * BV), body = (K * BV - edge) & ~3, end = K * BV - edge - body;
    float* state = sm + 2 * kPart + off;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 8, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    const bool whole = BV == V;
    if (h0) {
        if (tid == 0) {
            mbar_arrive_expect_tx(bar, 4u * body);  // (a box's columns behind V count, too)
            if (!whole) tma_load_3d(smem_u32(state), &tm_in, v0, 0, n * H + h, bar);
            else if (body > 0) bulk_load(smem_u32(state + edge), h0 + st + edge, 4u * body, bar);
        }
        __syncwarp();
        if (tid < edge) state[tid] = h0[st + tid];
        if (tid < end) state[edge + body + tid] = h0[st + edge + body + tid];
    } else {
        for (int x = tid; x < K * BV; x += NT) state[x] = 0.f;
    }
    long bos, eos;
    if (cu) { bos = __ldg(cu + n); eos = __ldg(cu + n + 1); }
    else    { bos = (long)n * T; eos = bos + T; }
    const int pieces = BV / E, groups = NT / pieces, piece = tid % pieces, group = tid / pieces;
    const bool on = group < groups && E * piece < cols;
    const int Hq = H / hr, hq = h / hr;
    const Gates::Head head = gates.head(h);
    const float scale = rsqrtf((float)K);
    bool waiting = h0 != nullptr;
    // The state is there for the whole block, or (true) a wait has given up: then the block waits for the copy once more, so
    // that none is in flight when it ends, and ends without a store (hT may be the only place that still holds the state).
    auto gave_up = [&] {
        waiting = false;
        if (!__syncthreads_or(!(stall ? mbar_wait(bar + 8, 0, 256) : mbar_wait(bar, 0)))) return false;
        mbar_wait(bar, 0);
        if (tid == 0) {
            atomicAdd(&g_token_timeouts, 1u);
            if (status) atomicOr(status, KDA_DEVICE_WAIT_GAVE_UP);
        }
        return true;
    };
    Columns<E>* S = reinterpret_cast<Columns<E>*>(state) + piece;
    for (long t = bos; t < eos; ++t) {
        const size_t qk = ((size_t)t * Hq + hq) * K, vo = ((size_t)t * H + h) * V + v0 + E * piece;
        float qv[256 / NT], kv[256 / NT];
#pragma unroll
        for (int x = 0; x < 256 / NT; ++x) {
            const int r = tid + x * NT;
            qv[x] = r < K ? to_f32(q[qk + r]) : 0.f;
            kv[x] = r < K ? to_f32(k[qk + r]) : 0.f;
        }
        float u[E] = {};
        if (on)
#pragma unroll
            for (int j = 0; j < E; ++j) u[j] = to_f32(v[vo + j]);
        const float dec = expf(gates.decay(t, h, head)), rate = gates.rate(t, h);
        float dots[3] = {};
#pragma unroll
        for (int x = 0; x < 256 / NT; ++x) {
            dots[0] = fmaf(qv[x], qv[x], dots[0]);
            dots[1] = fmaf(kv[x], kv[x], dots[1]);
            dots[2] = fmaf(qv[x], kv[x], dots[2]);
            s_q[tid + x * NT] = qv[x];
            s_k[tid + x * NT] = kv[x];
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) dots[e] += __shfl_xor_sync(0xffffffffu, dots[e], m);
            if ((tid & 31) == 0) s_dot[e][tid >> 5] = dots[e];
        }
        if (!waiting) __syncthreads();
        else if (gave_up()) return;
        Columns<E> y{}, z{};
        if (on) {
#pragma unroll 4
            for (int r = group; r < K; r += groups) {
                const Columns<E> s = S[r * pieces];
                const float a = s_k[r], b = s_q[r];
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    y.e[j] = fmaf(s.e[j], a, y.e[j]);
                    z.e[j] = fmaf(s.e[j], b, z.e[j]);
                }
            }
            reinterpret_cast<Columns<E>*>(part)[tid] = y;
            reinterpret_cast<Columns<E>*>(part + kPart)[tid] = z;
        }
        __syncthreads();
        if (on) {
            float d[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 3; ++e)
#pragma unroll
                for (int x = 0; x < NT / 32; ++x) d[e] += s_dot[e][x];
            const float nq = flags & KDA_FLAG_Q_L2NORM ? row_norm(d[0]) : 1.f;
            const float nk = flags & KDA_FLAG_K_L2NORM ? row_norm(d[1]) : 1.f;
            auto total = [&](const float* from) {
                Columns<E> s{};
#pragma unroll 4
                for (int g = 0; g < groups; ++g) {
                    const Columns<E> x = reinterpret_cast<const Columns<E>*>(from)[g * pieces + piece];
#pragma unroll
                    for (int j = 0; j < E; ++j) s.e[j] += x.e[j];
                }
                return s;
            };
            y = total(part);
            const float g = dec * nk;
#pragma unroll
            for (int j = 0; j < E; ++j) u[j] = rate * (u[j] - g * y.e[j]);
            if (group == t % groups) {  // (each group's turn)
                z = total(part + kPart);
                const float f = scale * nq, c = nk * d[2];
#pragma unroll
                for (int j = 0; j < E; ++j) o[vo + j] = from_f32<OutT>(f * fmaf(c, u[j], dec * z.e[j]));
            }
#pragma unroll
            for (int j = 0; j < E; ++j) u[j] *= nk;
#pragma unroll 4
            for (int r = group; r < K; r += groups) {
                Columns<E> s = S[r * pieces];
                const float a = s_k[r];
#pragma unroll
                for (int j = 0; j < E; ++j) s.e[j] = fmaf(s.e[j], dec, a * u[j]);
                S[r * pieces] = s;
            }
        }
        __syncthreads();
    }
    if ((waiting && gave_up()) || !hT) return;
    fence_proxy_async_smem();
    __syncthreads();
    // (this block has read its part of h0 and no other touches it: hT may be h0)
    if (tid == 0) {
        if (!whole) decay::tma_store_3d(&tm_out, smem_u32(state), v0, 0, n * H + h);
        else if (body > 0) bulk_store(hT + st + edge, smem_u32(state + edge), 4u * body);
        decay::bulk_commit();
        decay::bulk_wait_read();
    }
    if (tid < edge) hT[st + tid] = state[tid];
    if (tid < end) hT[st + edge + body + tid] = state[edge + body + tid];
}

constexpr int RG = 16, R = 16, COLS = 128 / RG;  // groups of lanes, rows of a lane, columns of a warp
template <typename InT, typename OutT>
__global__ void __launch_bounds__(256, 2) delta_recurrent_kernel(
    const InT* __restrict__ q, const InT* __restrict__ k, const InT* v, Gates gates, unsigned flags,
    const float* h0, float* hT, const int32_t* __restrict__ cu, int T, int H, int hr, int K, int V, int vblocks, long units,
    OutT* o) {
    const int lane = threadIdx.x & 31, rg = lane / (32 / RG);
    const long unit = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= units) return;
    const int vb = (int)(unit % vblocks), h = (int)(unit / vblocks % H), n = (int)(unit / vblocks / H);
    long bos, eos;
    if (cu) { bos = __ldg(cu + n); eos = __ldg(cu + n + 1); }
    else    { bos = (long)n * T; eos = bos + T; }

    const int row0 = R * rg, col = vb * COLS + 4 * (lane % (32 / RG));
    const size_t st = ((size_t)n * H + h) * (size_t)K * V + (size_t)row0 * V + col;
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) S[r][j] = 0.f;
        if (!h0) continue;
        const float* src = h0 + st + (size_t)r * V;
        if (row0 + r < K) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < V) S[r][j] = src[j];
        }
    }
    const float scale = rsqrtf((float)K);
    const int Hq = H / hr, hq = h / hr;
    const Gates::Head head = gates.head(h);
    for (long t = bos; t < eos; ++t) {
        const size_t qk = ((size_t)t * Hq + hq) * K + row0, vo = ((size_t)t * H + h) * V + col;
        const float dec = expf(gates.decay(t, h, head)), rate = gates.rate(t, h);
        float kr[R], u[4], y[4] = {}, z[4] = {}, qq = 0.f, kk = 0.f, qk_dot = 0.f;  // y = S^T k, z = S^T q
#pragma unroll
        for (int r = 0; r < R; ++r) kr[r] = row0 + r < K ? to_f32(k[qk + r]) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = col + j < V ? to_f32(v[vo + j]) : 0.f;
#pragma unroll
        for (int half = 0; half < R; half += 8) {
            float qr[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) qr[r] = row0 + half + r < K ? to_f32(q[qk + half + r]) : 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float kv = kr[half + r];
                qq = fmaf(qr[r], qr[r], qq);
                kk = fmaf(kv, kv, kk);
                qk_dot = fmaf(qr[r], kv, qk_dot);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[j] = fmaf(S[half + r][j], kv, y[j]);
                    z[j] = fmaf(S[half + r][j], qr[r], z[j]);
                }
            }
        }
#pragma unroll
        for (int m = 16; m >= 32 / RG; m >>= 1) {
            qq += __shfl_xor_sync(0xffffffffu, qq, m);
            kk += __shfl_xor_sync(0xffffffffu, kk, m);
            qk_dot += __shfl_xor_sync(0xffffffffu, qk_dot, m);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] += __shfl_xor_sync(0xffffffffu, y[j], m);
                z[j] += __shfl_xor_sync(0xffffffffu, z[j], m);
            }
        }
        const float nq = flags & KDA_FLAG_Q_L2NORM ? row_norm(qq) : 1.f;
        const float nk = flags & KDA_FLAG_K_L2NORM ? row_norm(kk) : 1.f;
        const float fs = scale * nq;
        __syncwarp();  // (every lane has its values)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = rate * (u[j] - dec * nk * y[j]);
            if (rg == 0 && col + j < V) o[vo + j] = from_f32<OutT>(fs * fmaf(nk * qk_dot, u[j], dec * z[j]));
            u[j] *= nk;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[r][j] = fmaf(S[r][j], dec, kr[r] * u[j]);
    }
    // this lane has read its part of h0 above and no other touches it: hT may be h0
    if (!hT) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float* dst = hT + st + (size_t)r * V;
        if (row0 + r < K) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < V) dst[j] = S[r][j];
        }
    }
}

template <typename InT, typename OutT>
cudaError_t launch_r(const DeltaArgs& a) {
    const int vblocks = (a.V + COLS - 1) / COLS;
    const long units = (long)a.N * a.H * vblocks;
    const long blocks = (units + 7) / 8;
    if (blocks > 0x7fffffffl) return cudaErrorInvalidValue;
    delta_recurrent_kernel<InT, OutT><<<(unsigned)blocks, 256, 0, a.stream>>>((const InT*)a.q, (const InT*)a.k, (const InT*)a.v, Gates(a), a.flags, a.h0, a.hT,
                                                 a.cu, a.T, a.H, a.H / a.Hk, a.K, a.V, vblocks, units, (OutT*)a.o);
    return cudaGetLastError();
}

// states [N H][K][V], boxes of BV columns of one
bool state_map(CUtensorMap* m, const float* base, const DeltaArgs& a, int BV) {
    auto fn = decay::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.V, (cuuint64_t)a.K, (cuuint64_t)a.N * a.H};
    const cuuint64_t strides[2] = {(cuuint64_t)a.V * 4, (cuuint64_t)a.K * a.V * 4};
    const cuuint32_t box[3] = {(cuuint32_t)BV, (cuuint32_t)a.K, 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <typename InT, typename OutT, int NT, int E = 4>
cudaError_t launch_token(const DeltaArgs& a, int BV) {
    auto kern = delta_token_kernel<InT, OutT, NT, E>;
    const int bytes = (a.K * BV + 2 * E * NT + (E == 4 ? 0 : 4)) * (int)sizeof(float);
    // the kernel's limit is what the largest call wants (a column block of a tile is up to four columns more), whatever this one
    // does: it is the function's, and another host thread's call may be between its own and the launch
    constexpr int most = ((E == 4 ? kTile + 4 * 256 : kWhole + 4) + 2 * E * NT) * (int)sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    CUtensorMap in{}, out{};
    if (BV < a.V && ((a.h0 && !state_map(&in, a.h0, a, BV)) || (a.hT && !state_map(&out, a.hT, a, BV)))) return cudaErrorInvalidValue;
    kern<<<dim3((a.V + BV - 1) / BV, a.H, a.N), NT, bytes, a.stream>>>(in, out, (const InT*)a.q, (const InT*)a.k, (const InT*)a.v, Gates(a),
                                                                     a.flags, a.h0, a.hT, a.cu, a.T, a.H, a.H / a.Hk, a.K, a.V, BV, (OutT*)a.o,
                                                                     a.status, hook_stall_chunk() == 0);
    return cudaGetLastError();
}

template <typename InT, typename OutT>
cudaError_t launch_k(const DeltaArgs& a) {
    if (a.V % 4 == 0) {
        const int blocks = (a.K * a.V + kTile - 1) / kTile, BV = ((a.V + blocks - 1) / blocks + 3) / 4 * 4, bytes = 4 * a.K * BV;
        // threads for a tile: 192 KB of states an SM are under way with three blocks of 64 KB, six of 32, eleven of 16
        // (512 tokens, 32 heads of 64 x 64: 183 us with 256 threads)
        return bytes > 40960 ? launch_token<InT, OutT, 256>(a, BV) : bytes > 16384 ? launch_token<InT, OutT, 128>(a, BV) : launch_token<InT, OutT, 64>(a, BV);
    }
    // a state that one bulk copy can take (512 tokens, 32 heads of 128 x 126: 312 us, by single loads 850)
    if (a.K * a.V <= kWhole) {
        const bool small = a.K * a.V <= 10240;
        if (a.V % 2 == 0) return small ? launch_token<InT, OutT, 128, 2>(a, a.V) : launch_token<InT, OutT, 256, 2>(a, a.V);
        return small && a.V <= 128 ? launch_token<InT, OutT, 128, 1>(a, a.V) : launch_token<InT, OutT, 256, 1>(a, a.V);
    }
    return launch_r<InT, OutT>(a);
}

}  // namespace
}  // namespace delta

cudaError_t launch_delta_recurrent(const DeltaArgs& a) {
    if (a.N == 0) return cudaSuccess;
    if (!a.qkv_bf16) return delta::launch_k<float, float>(a);
    return a.o_f32 ? delta::launch_k<__nv_bfloat16, float>(a) : delta::launch_k<__nv_bfloat16, __nv_bfloat16>(a);
}

cudaError_t read_token_timeouts(unsigned* count, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(count, delta::g_token_timeouts, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(delta::g_token_timeouts, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace kda
