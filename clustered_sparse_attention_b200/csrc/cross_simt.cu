// cross_simt.cu -- dense cross attention and its backward pass in fp32
// arithmetic on the FMA pipe.
//
// Forward: s_ij = scale q_i.k_j over the keys j < k_len, an online softmax
// (running maximum m, sum l), o_i = sum_j e^{s_ij - m} v_j / l and
// lse_i = m + log l.  Backward: p_ij = e^{s_ij - lse_i},
// ds_ij = p_ij (do_i.v_j - delta_i), dq_i = scale sum_j ds_ij k_j,
// dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij do_i.
//
// 64 x 64 score tiles, groups of 128 threads in an 8 x 16 grid, 8 x 4 scores and
// 8 x D/16 outputs a thread: 16 shared-memory wavefronts per 128 FMA
// instructions of a warp (4 x 4 scores a thread need 24, and kept the shared
// memory pipe 70 % busy with the FMA pipe at 46 %; packed FMA pairs measured no
// faster).  Rows of the shared tiles
// are D + 4 floats (16-byte units an odd number apart) and a thread's rows are
// ty, ty + 8, ..., so that neither the 16 column threads nor the two row threads
// of a warp meet in a bank.  The backward
// kernels' four tiles leave room for one CTA per SM; two groups share it, one
// for the scores and one for do.v (then dV and dK, or the halves of dQ's
// columns), which hides twice the latency of one group.
//
// Bound by issue: with two warps a scheduler the FMA pipe runs at 0.47 (dQ) and 0.51
// (dK, dV) of its rate and 0.8 of all instructions are FMAs.  Gradients of 2,049 x 257
// keys, 8 heads, d = 128: 203 us with dQ from the dK/dV kernel (27 TFLOP/s; a library
// chain of the same five products takes 256), 277 with a dQ kernel (see
// cross_dq_part_floats).
#include <math.h>

#include "common.cuh"
#include "cross.h"
#include "launchers.h"
#include "tc_ptx.cuh"

namespace svgear {
namespace {

constexpr int M = kCrossSimtM, N = kCrossSimtN;
constexpr int kThreads = 128;
constexpr int kGradThreads = 256;   // two groups
constexpr int R = 8;                // rows of a thread

// Starts the copy of rows [n0, n0 + 64) of head (b, h) to fp32 rows of D + 4,
// zeros from n_end on (part of the thread's next cp.async group).
template <int D>
__device__ __forceinline__ void copy_tile(float* s, const svgear_tokens& t, int b, int h, int n0, int n_end) {
    constexpr int CH = D / 4;
    for (int i = threadIdx.x; i < 64 * CH; i += blockDim.x) {
        const int r = i / CH, c = (i - r * CH) * 4;
        const bool in = n0 + r < n_end;
        const float* src = row_ptr<const float>(t, b, h, in ? n0 + r : 0) + c;
        tc::cp_async16(tc::smem_u32(s + r * (D + 4) + c), src, in ? 16u : 0u);
    }
}

// acc[i][j] = A[ty + 8 i] . B[tx + 16 j], j < J (the others 0)
template <int D, int J>
__device__ __forceinline__ void dot_columns(const float* A, const float* Bm, int ty, int tx,
                                            float (&acc)[R][4]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 a[R], c[J];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 8 * i) * (D + 4) + k);
#pragma unroll
        for (int j = 0; j < J; ++j) c[j] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * j) * (D + 4) + k);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                acc[i][j] = fmaf(a[i].x, c[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, c[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, c[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, c[j].w, acc[i][j]);
            }
    }
}
// The same for a tile of `valid` keys: one with at most 16 skips the rest.
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* Bm, int valid, int ty, int tx,
                                         float (&acc)[R][4]) {
    if (valid <= 16) dot_columns<D, 1>(A, Bm, ty, tx, acc);
    else dot_columns<D, 4>(A, Bm, ty, tx, acc);
}

// A product with a tile's weights is summed on its own and then added to the
// running sum: n terms then take chains of 64 and n / 64 additions.  In one chain of
// n the error of equal terms does not cancel (O over 75,600 equal keys: off by 9e-4,
// now by 2e-7, and the sum of the weights by 2e-5), and it saves one addition in 64.
template <int C>
__device__ __forceinline__ void clear(float (&x)[R][C]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c) x[i][c] = 0.f;
}
template <int C>
__device__ __forceinline__ void add(float (&acc)[R][C], const float (&x)[R][C]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c] += x[i][c];
}

// acc[i][4 c + e] = sum_n W[ty + 8 i][n] X[n][64 c + 4 tx + e]; W rows of N + 4,
// X rows of D + 4, n < valid (weights past it are 0); C columns (a multiple of
// 64, or 32: then two per thread)
template <int D, int C = D>
__device__ __forceinline__ void tile_product(const float* W, const float* X, int valid, int ty, int tx,
                                             float (&acc)[R][C / 16]) {
    clear(acc);
#pragma unroll 2
    for (int n = 0; n < min(N, valid); n += 4) {
        float4 w[R];
#pragma unroll
        for (int i = 0; i < R; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty + 8 * i) * (N + 4) + n);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float* row = X + (n + q) * (D + 4);
            float x[C / 16];
            if constexpr (C == 32) {
                const float2 v = *reinterpret_cast<const float2*>(row + 2 * tx);
                x[0] = v.x;
                x[1] = v.y;
            } else {
#pragma unroll
                for (int c = 0; c < C / 64; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(row + 64 * c + 4 * tx);
                    x[4 * c] = v.x;
                    x[4 * c + 1] = v.y;
                    x[4 * c + 2] = v.z;
                    x[4 * c + 3] = v.w;
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float wi = q == 0 ? w[i].x : q == 1 ? w[i].y : q == 2 ? w[i].z : w[i].w;
#pragma unroll
                for (int c = 0; c < C / 16; ++c) acc[i][c] = fmaf(wi, x[c], acc[i][c]);
            }
        }
    }
}

// acc[i][4 c + e] = sum_q W[q][8 ty + i] X[q][64 c + 4 tx + e] (W transposed)
template <int D>
__device__ __forceinline__ void tile_product_t(const float* W, const float* X, int ty, int tx,
                                               float (&acc)[R][D / 16]) {
    clear(acc);
#pragma unroll 4
    for (int q = 0; q < M; ++q) {
        const float4 w = *reinterpret_cast<const float4*>(W + q * (N + 4) + 8 * ty);
        const float4 y = *reinterpret_cast<const float4*>(W + q * (N + 4) + 8 * ty + 4);
        const float wi[R] = {w.x, w.y, w.z, w.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(X + q * (D + 4) + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                acc[i][4 * c] = fmaf(wi[i], x.x, acc[i][4 * c]);
                acc[i][4 * c + 1] = fmaf(wi[i], x.y, acc[i][4 * c + 1]);
                acc[i][4 * c + 2] = fmaf(wi[i], x.z, acc[i][4 * c + 2]);
                acc[i][4 * c + 3] = fmaf(wi[i], x.w, acc[i][4 * c + 3]);
            }
        }
    }
}

__device__ __forceinline__ float row_max16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a);
    u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
}

// The device status words: no kernel of this file waits, so one of them clears the
// words (a memset of its own costs a small call 2 us).
__device__ __forceinline__ void clear_status(const CrossArgs& a) {
    if ((blockIdx.x | blockIdx.y) == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
cross_fwd_kernel(CrossArgs a, int splits, int tiles_per_split, float* __restrict__ o_part,
                 float* __restrict__ lse_part) {
    extern __shared__ float sm[];
    float* sQ = sm;
    float* sK = sQ + M * (D + 4);
    float* sV = sK + N * (D + 4);
    float* sP = sV + N * (D + 4);
    const int qt = blockIdx.x / splits, sp = blockIdx.x - qt * splits;
    clear_status(a);
    const int b = blockIdx.y / a.Hq, h = blockIdx.y - b * a.Hq, hk = h / a.G;
    const int q0 = qt * M, keys = cross_keys(a, b);
    const int t0 = sp * tiles_per_split, t1 = min((keys + N - 1) / N, t0 + tiles_per_split);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;

    copy_tile<D>(sQ, a.Q, b, h, q0, a.Nq);
    float m[R], l[R], o[R][D / 16];
    clear(o);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
        __syncthreads();
        copy_tile<D>(sK, a.K, b, hk, t * N, keys);
        tc::cp_async_commit();
        copy_tile<D>(sV, a.V, b, hk, t * N, keys);   // arrives beside the scores
        tc::cp_async_commit();
        tc::cp_async_wait<1>();
        __syncthreads();
        float s[R][4];
        dot_tile<D>(sQ, sK, keys - t * N, ty, tx, s);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = t * N + tx + 16 * j < keys ? s[i][j] * a.scale : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            const float mn = fmaxf(m[i], row_max16(mx));
            const float mu = mn == -INFINITY ? 0.f : mn;   // every score -inf so far
            const float alpha = expf(m[i] - mu);
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= alpha;
            float lt = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = expf(s[i][j] - mu);
                lt += p;
                sP[(ty + 8 * i) * (N + 4) + tx + 16 * j] = p;
            }
            l[i] = fmaf(l[i], alpha, lt);
        }
        tc::cp_async_wait<0>();
        __syncthreads();
        float x[R][D / 16];
        tile_product<D>(sP, sV, keys - t * N, ty, tx, x);
        add(o, x);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float sum = row_sum16(l[i]);
        const int row = q0 + ty + 8 * i;
        if (row >= a.Nq) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;   // no key: o = 0, lse = -inf
        const float lse = sum == 0.f ? -INFINITY : m[i] + logf(sum);
        const size_t r = (size_t)blockIdx.y * a.Nq + row;
        if (splits > 1) {
            const size_t rp = (size_t)sp * a.B * a.Hq * a.Nq + r;
            if (tx == 0) lse_part[rp] = lse;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                store4(o_part + rp * D + 64 * c + 4 * tx,
                       make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
                                   o[i][4 * c + 3] * inv));
        } else {
            if (tx == 0) a.lse[r] = lse;
            float* dst = row_ptr<float>(a.O, b, h, row);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                store4(dst + 64 * c + 4 * tx,
                       make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
                                   o[i][4 * c + 3] * inv));
        }
    }
}

// One warp per row: o = sum_s e^{lse_s - lse} o_s, lse = log sum_s e^{lse_s},
// in split order.
template <typename T, int D>
__global__ void __launch_bounds__(256)
cross_join_kernel(CrossArgs a, int splits, const float* __restrict__ o_part,
                  const float* __restrict__ lse_part) {
    const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int lane = threadIdx.x & 31;
    float mx = -INFINITY;
    for (int s = 0; s < splits; ++s) mx = fmaxf(mx, lse_part[s * rows + r]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float ls = lse_part[s * rows + r];
        if (ls == -INFINITY) continue;   // a split past the batch's keys
        const float w = expf(ls - mu);
        sum += w;
        const float* p = o_part + (s * rows + r) * D;
        if constexpr (D == 128) {
            const float4 x = *reinterpret_cast<const float4*>(p + 4 * lane);
            o[0] = fmaf(w, x.x, o[0]); o[1] = fmaf(w, x.y, o[1]);
            o[2] = fmaf(w, x.z, o[2]); o[3] = fmaf(w, x.w, o[3]);
        } else {
            const float2 x = *reinterpret_cast<const float2*>(p + 2 * lane);
            o[0] = fmaf(w, x.x, o[0]); o[1] = fmaf(w, x.y, o[1]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t bh = r / a.Nq;
    const int b = (int)(bh / a.Hq), h = (int)(bh - (int64_t)b * a.Hq);
    T* dst = row_ptr<T>(a.O, b, h, r - bh * a.Nq);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dst[D / 32 * lane + c] = Elem<T>::to(o[c] * inv);
    if (lane == 0) a.lse[r] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// p of one 64 x 64 tile from its scores, into W
__device__ __forceinline__ void put_weights(const float (&s)[R][4], const float* lse, float* W, int ty, int tx,
                                            int k0, int keys, float scale) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            W[(ty + 8 * i) * (N + 4) + tx + 16 * j] =
                k0 + tx + 16 * j < keys ? expf(s[i][j] * scale - lse[ty + 8 * i]) : 0.f;
}
// ds = p (dp - delta) of the same tile, p from W, into G (which may be W)
__device__ __forceinline__ void put_score_grads(const float (&dp)[R][4], const float* delta, const float* W,
                                                float* G, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = (ty + 8 * i) * (N + 4) + tx + 16 * j;
            G[x] = W[x] * (dp[i][j] - delta[ty + 8 * i]);
        }
}

// a thread's columns of a row of C, as tile_product() has them, times f
template <int C>
__device__ __forceinline__ void store_half(float* dst, const float (&x)[C / 16], float f, int tx) {
    if constexpr (C == 64)
        store4(dst + 4 * tx, make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f));
    else
        *reinterpret_cast<float2*>(dst + 2 * tx) = make_float2(x[0] * f, x[1] * f);
}

template <int D>
__global__ void __launch_bounds__(kGradThreads) cross_dq_kernel(CrossArgs a) {
    constexpr int C = D / 2;   // dQ columns of a group
    extern __shared__ float sm[];
    float* sQ = sm;
    float* sG = sQ + M * (D + 4);
    float* sKV = sG + M * (D + 4);                 // K and V of two tiles
    float* sS = sKV + 4 * N * (D + 4);
    __shared__ float s_lse[M], s_delta[M];
    const int b = blockIdx.y / a.Hq, h = blockIdx.y - b * a.Hq, hk = h / a.G;
    const int q0 = blockIdx.x * M, keys = cross_keys(a, b);
    const int grp = threadIdx.x >> 7, ty = (threadIdx.x >> 4) & 7, tx = threadIdx.x & 15;
    copy_tile<D>(sQ, a.Q, b, h, q0, a.Nq);
    copy_tile<D>(sG, a.dO, b, h, q0, a.Nq);
    copy_tile<D>(sKV, a.K, b, hk, 0, keys);
    copy_tile<D>(sKV + N * (D + 4), a.V, b, hk, 0, keys);
    tc::cp_async_commit();
    if (threadIdx.x < M) {
        const int row = q0 + threadIdx.x;
        const size_t r = (size_t)blockIdx.y * a.Nq + row;
        s_lse[threadIdx.x] = row < a.Nq ? a.lse[r] : INFINITY;   // past the end: p = 0
        s_delta[threadIdx.x] = row < a.Nq ? a.delta[r] : 0.f;
    }
    float dq[R][C / 16];
    clear(dq);
    for (int t = 0; t * N < keys; ++t) {
        float* sK = sKV + (t & 1) * 2 * N * (D + 4);
        float* sV = sK + N * (D + 4);
        tc::cp_async_wait<0>();
        __syncthreads();
        if ((t + 1) * N < keys) {   // the next tile arrives beside this one's arithmetic
            float* next = sKV + ((t + 1) & 1) * 2 * N * (D + 4);
            copy_tile<D>(next, a.K, b, hk, (t + 1) * N, keys);
            copy_tile<D>(next + N * (D + 4), a.V, b, hk, (t + 1) * N, keys);
        }
        tc::cp_async_commit();
        float s[R][4];
        dot_tile<D>(grp ? sG : sQ, grp ? sV : sK, keys - t * N, ty, tx, s);
        if (grp == 0) put_weights(s, s_lse, sS, ty, tx, t * N, keys, a.scale);
        __syncthreads();
        if (grp == 1) put_score_grads(s, s_delta, sS, sS, ty, tx);
        __syncthreads();
        float x[R][C / 16];
        tile_product<D, C>(sS, sK + grp * C, keys - t * N, ty, tx, x);
        add(dq, x);
    }
    tc::cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = q0 + ty + 8 * i;
        if (row >= a.Nq) continue;
        store_half<C>(row_ptr<float>(a.dQ, b, h, row) + grp * C, dq[i], a.scale, tx);
    }
}

// DQ: also the key tile's part of dQ, half its columns a group.
template <int D, bool DQ>
__global__ void __launch_bounds__(kGradThreads) cross_dkv_kernel(CrossArgs a, float* __restrict__ part) {
    extern __shared__ float sm[];
    float* sQ2 = sm;                               // Q of two tiles
    float* sG = sQ2 + 2 * M * (D + 4);
    float* sK = sG + M * (D + 4);
    float* sV = sK + N * (D + 4);
    float* sP = sV + N * (D + 4);
    float* sS = sP + M * (N + 4);
    __shared__ float s_lse[M], s_delta[M];
    const int grp = threadIdx.x >> 7, ty = (threadIdx.x >> 4) & 7, tx = threadIdx.x & 15;
    const int qtiles = (a.Nq + M - 1) / M;
    const int64_t per = (int64_t)a.G * qtiles;
    const int64_t total = kv_total_units<N>(a) * per;
    const int64_t end = kv_range(total, blockIdx.x + 1, gridDim.x);
    KvCursor cur;
    kv_cursor_start<N>(a, cur);
    for (int64_t it = kv_range(total, blockIdx.x, gridDim.x); it < end;) {
        const int64_t u = it / per;
        const int64_t first = it - u * per, last = min(per, first + (end - it));
        const KvUnit k = kv_unit<N>(a, cur, u);
        __syncthreads();
        copy_tile<D>(sK, a.K, k.b, k.h, k.kt * N, k.keys);
        copy_tile<D>(sV, a.V, k.b, k.h, k.kt * N, k.keys);
        const int valid = k.keys - k.kt * N;
        auto copy_q = [&](int64_t x) {
            const int g = (int)(x / qtiles);
            copy_tile<D>(sQ2 + (x & 1) * M * (D + 4), a.Q, k.b, k.h * a.G + g, (int)(x - (int64_t)g * qtiles) * M, a.Nq);
        };
        copy_q(first);
        tc::cp_async_commit();
        float acc[R][D / 16];   // group 0: dV, group 1: dK
        clear(acc);
        for (int64_t x = first; x < last; ++x) {
            const int g = (int)(x / qtiles), q0 = (int)(x - (int64_t)g * qtiles) * M;
            const int h = k.h * a.G + g;
            const float* sQ = sQ2 + (x & 1) * M * (D + 4);
            __syncthreads();
            copy_tile<D>(sG, a.dO, k.b, h, q0, a.Nq);
            tc::cp_async_commit();
            if (x + 1 < last) copy_q(x + 1);   // arrives beside this tile's arithmetic
            tc::cp_async_commit();
            if (threadIdx.x < M) {
                const int row = q0 + threadIdx.x;
                const size_t r = ((size_t)k.b * a.Hq + h) * a.Nq + row;
                s_lse[threadIdx.x] = row < a.Nq ? a.lse[r] : INFINITY;
                s_delta[threadIdx.x] = row < a.Nq ? a.delta[r] : 0.f;
            }
            tc::cp_async_wait<1>();
            __syncthreads();
            float s[R][4];
            dot_tile<D>(grp ? sG : sQ, grp ? sV : sK, valid, ty, tx, s);
            if (grp == 0) put_weights(s, s_lse, sP, ty, tx, k.kt * N, k.keys, a.scale);
            __syncthreads();
            float y[R][D / 16];
            if (grp == 0) {
                if (8 * ty < valid) {   // rows past the keys are not written
                    tile_product_t<D>(sP, sG, ty, tx, y);
                    add(acc, y);
                }
                if constexpr (DQ) asm volatile("bar.sync 2, 256;" ::: "memory");   // ds from group 1
            } else {
                put_score_grads(s, s_delta, sP, sS, ty, tx);
                asm volatile("bar.sync 1, 128;" ::: "memory");   // group 1
                if constexpr (DQ) asm volatile("bar.arrive 2, 256;" ::: "memory");
                if (8 * ty < valid) {
                    tile_product_t<D>(sS, sQ, ty, tx, y);
                    add(acc, y);
                }
            }
            if constexpr (DQ) {
                constexpr int C = D / 2;
                float dq[R][C / 16];
                tile_product<D, C>(sS, sK + grp * C, valid, ty, tx, dq);
                float* pq = a.dq_part + (((size_t)k.kt * a.B + k.b) * a.Hq + h) * a.Nq * D + grp * C;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int row = q0 + ty + 8 * i;
                    if (row < a.Nq) store_half<C>(pq + (size_t)row * D, dq[i], 1.f, tx);
                }
            }
        }
        const bool whole = first == 0 && last == per;
        float* pk = part + (((size_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * 2 + (1 - grp)) * N * D;
        const float f = grp ? a.scale : 1.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = 8 * ty + i, row = k.kt * N + r;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int col = 64 * c + 4 * tx;
                const float4 v = make_float4(acc[i][4 * c] * f, acc[i][4 * c + 1] * f, acc[i][4 * c + 2] * f,
                                             acc[i][4 * c + 3] * f);
                if (!whole)
                    store4(pk + r * D + col, v);
                else if (row < k.keys)
                    store4(row_ptr<float>(grp ? a.dK : a.dV, k.b, k.h, row) + col, v);
            }
        }
        it += last - first;
        tc::cp_async_wait<0>();
    }
}

// dQ from its key tiles' parts, in their order (none: zeros); 16 bytes a thread, bound by
// the parts' bytes (mostly in L2).
template <int D>
__global__ void __launch_bounds__(256) cross_dq_join_kernel(CrossArgs a) {
    const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / (D / 4);
    if (r >= rows) return;
    const int col = (int)(i % (D / 4)) * 4;
    const int bh = (int)(r / a.Nq), b = bh / a.Hq, h = bh - b * a.Hq;
    const int nt = (cross_keys(a, b) + N - 1) / N;
    float4 p[kCrossDqTiles];   // every load before the first use
#pragma unroll
    for (int t = 0; t < kCrossDqTiles; ++t)
        if (t < nt) p[t] = *reinterpret_cast<const float4*>(a.dq_part + (t * rows + r) * D + col);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kCrossDqTiles; ++t)
        if (t < nt) {
            v.x += p[t].x; v.y += p[t].y; v.z += p[t].z; v.w += p[t].w;
        }
    store4(row_ptr<float>(a.dQ, b, h, r - (int64_t)bh * a.Nq) + col,
           make_float4(v.x * a.scale, v.y * a.scale, v.z * a.scale, v.w * a.scale));
}

// Joins the partial sums of units cut between CTAs (in CTA order) and writes
// zeros for the keys past k_len.  One CTA per 16 rows of a key tile of one
// (b, key/value head): blockIdx.x = 16-row group, blockIdx.y = b * Hkv + h.
// Bound by latency: the ranges' arithmetic, then a part's loads at a time (one float4 a
// thread at a time took 25 us for two batches of 40 heads where this takes 16).
constexpr int kJoinRows = 16;
template <typename T, int D, int BN>
__global__ void __launch_bounds__(256)
cross_dkv_join_kernel(CrossArgs a, int qrows, int ctas, const float* __restrict__ part) {
    const int row0 = blockIdx.x * kJoinRows, kt = row0 / BN;
    const int b = blockIdx.y / a.Hkv, h = blockIdx.y - b * a.Hkv;
    const int keys = cross_keys(a, b), nt = (keys + BN - 1) / BN;
    const int rows = min(kJoinRows, a.Nk - row0);
    __shared__ int s_first, s_last;
    __shared__ bool s_empties;   // some CTAs have no iteration
    if (threadIdx.x < 32 && kt < nt) {
        const int64_t per = (int64_t)a.G * ((a.Nq + qrows - 1) / qrows);
        int64_t before = 0;   // units of the batches before b
        if (!a.k_len) {
            before = (int64_t)b * a.Hkv * nt;
        } else {
            for (int x = threadIdx.x; x < b; x += 32) before += (cross_keys(a, x) + BN - 1) / BN;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
            before *= a.Hkv;
        }
        const int64_t total = kv_total_units<BN>(a) * per;
        if (threadIdx.x < 2) {
            // the CTAs whose ranges hold the unit's first and last iteration
            const int64_t s = (before + (int64_t)h * nt + kt) * per, e = s + per - 1;
            auto holder = [&](int64_t it) {
                int c = min(ctas - 1, (int)((double)it / (double)total * ctas));
                while (c > 0 && kv_range(total, c, ctas) > it) --c;
                while (c + 1 < ctas && kv_range(total, c + 1, ctas) <= it) ++c;
                return c;
            };
            const int c = holder(threadIdx.x == 0 ? s : e);
            if (threadIdx.x == 0) {
                s_first = c;
                s_empties = total < ctas;
            } else {
                s_last = c;
            }
        }
    }
    __syncthreads();
    const bool direct = kt < nt && s_first == s_last;   // written by its CTA
    if (direct && row0 + rows <= keys) return;
    // a thread's sums side by side, so that a part's loads are in flight together
    constexpr int CH = D / 4, V = 2 * kJoinRows * CH / 256;
    const float* src[V];
    float4 v[V];
#pragma unroll
    for (int x = 0; x < V; ++x) {
        const int i = threadIdx.x + 256 * x, r = i / CH % kJoinRows, col = i % CH * 4;
        src[x] = part + ((size_t)(i / (kJoinRows * CH)) * BN + row0 - kt * BN + r) * D + col;
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (!direct && kt < nt) {
        const int64_t total = s_empties ? kv_total_units<BN>(a) * a.G * ((a.Nq + qrows - 1) / qrows) : 0;
        for (int c = s_first; c <= s_last; ++c) {
            if (s_empties && kv_range(total, c, ctas) == kv_range(total, c + 1, ctas)) continue;
            const size_t at = ((size_t)c * 2 + (c == s_first ? 1 : 0)) * 2 * BN * D;
            float4 p[V];
#pragma unroll
            for (int x = 0; x < V; ++x) p[x] = *reinterpret_cast<const float4*>(src[x] + at);
#pragma unroll
            for (int x = 0; x < V; ++x) {
                v[x].x += p[x].x; v[x].y += p[x].y; v[x].z += p[x].z; v[x].w += p[x].w;
            }
        }
    }
#pragma unroll
    for (int x = 0; x < V; ++x) {
        const int i = threadIdx.x + 256 * x, row = row0 + i / CH % kJoinRows;
        if (row >= a.Nk || (direct && row < keys)) continue;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);   // (parts hold anything past the keys)
        store4(row_ptr<T>(i / (kJoinRows * CH) ? a.dV : a.dK, b, h, row) + i % CH * 4, row < keys ? v[x] : z);
    }
}

constexpr int kHeldUnits = 2;   // units of cross_delta_held_kernel per thread, 256 apart

__device__ __forceinline__ void store_chunk(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// delta_i = do_i . o_i in fp32, 16 bytes of the row per lane.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_delta_kernel(CrossArgs a) {
    constexpr int C = Elem<T>::kPerChunk, LR = D / C;   // lanes per row: 8, 16 or 32
    clear_status(a);
    const uint32_t rows = (uint32_t)((int64_t)a.B * a.Hq * a.Nq);
    const uint64_t r64 = ((uint64_t)blockIdx.x * 256 + threadIdx.x) / LR;
    const bool in = r64 < rows;
    const uint32_t r = in ? (uint32_t)r64 : rows - 1;
    const int c = (threadIdx.x % LR) * C;
    const uint32_t bh = r / (uint32_t)a.Nq, n = r - bh * (uint32_t)a.Nq;
    const int b = (int)(bh / (uint32_t)a.Hq), h = (int)(bh - (uint32_t)b * (uint32_t)a.Hq);
    float g[C], o[C];
    Elem<T>::load(row_ptr<const T>(a.dO, b, h, n) + c, g);
    Elem<T>::load(row_ptr<const T>(a.O, b, h, n) + c, o);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < C; ++e) s = fmaf(g[e], o[e], s);
#pragma unroll
    for (int x = LR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (in && c == 0) a.delta[r] = s;
}

// The same with o from its 8-bit codes, and q unpacked from its own into qx
// [B][Hq][Nq][D]: 16 elements per lane and unit (16 bytes of codes), the loads of a
// thread's units up front.  One chunk of 8 elements a lane took 45 us for 2 x 3,600 x
// 40 x 128 bf16 (223 MB), this 33: the measured copy rate.
template <typename T, int D>
__global__ void __launch_bounds__(256)
cross_delta_held_kernel(CrossArgs a, HeldTokens qh, HeldTokens oh, T* __restrict__ qx) {
    constexpr int P = 16, LR = D / P, U = kHeldUnits, C = Elem<T>::kPerChunk;
    clear_status(a);
    const uint32_t rows = (uint32_t)((int64_t)a.B * a.Hq * a.Nq);
    const uint64_t i0 = (uint64_t)blockIdx.x * (256 * U) + threadIdx.x;
    const int c = (int)(i0 % LR) * P;
    uint4 g[U][P / C], oc[U], qc[U];
    uint32_t oe[U], qe[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t r64 = (i0 + 256 * u) / LR;
        const uint32_t r = r64 < rows ? (uint32_t)r64 : rows - 1;
        const uint32_t bh = r / (uint32_t)a.Nq, n = r - bh * (uint32_t)a.Nq;
        const int b = (int)(bh / (uint32_t)a.Hq), h = (int)(bh - (uint32_t)b * (uint32_t)a.Hq);
        const T* src = row_ptr<const T>(a.dO, b, h, n) + c;
        const size_t i = (size_t)r * D + c;
        oc[u] = __ldg(reinterpret_cast<const uint4*>(oh.codes + i));
        qc[u] = __ldg(reinterpret_cast<const uint4*>(qh.codes + i));
        oe[u] = __ldg(oh.exps + i / 32);
        qe[u] = __ldg(qh.exps + i / 32);
#pragma unroll
        for (int k = 0; k < P / C; ++k) g[u][k] = Elem<T>::load_raw(src + k * C);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t r64 = (i0 + 256 * u) / LR;
        const float ostep = held_step(oe[u]), qstep = held_step(qe[u]);
        const uint32_t ow[4] = {oc[u].x, oc[u].y, oc[u].z, oc[u].w};
        const uint32_t qw[4] = {qc[u].x, qc[u].y, qc[u].z, qc[u].w};
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < P / C; ++k) {
            float x[C], q[C];
            Elem<T>::unpack(g[u][k], x);
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const int y = k * C + e;
                s = fmaf(x[e], (float)(int8_t)(ow[y / 4] >> (8 * (y % 4))) * ostep, s);
                q[e] = (float)(int8_t)(qw[y / 4] >> (8 * (y % 4))) * qstep;
            }
            if (r64 < rows) store_chunk(qx + r64 * D + c + k * C, q);
        }
#pragma unroll
        for (int x = LR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (r64 < rows && c == 0) a.delta[r64] = s;
    }
}

template <typename F>
int set_smem(F* fn, size_t bytes) {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess
               ? SVGEAR_OK
               : SVGEAR_ERR_CUDA;
}

template <int D>
int fwd(const CrossArgs& a, CrossSplit sp, float* o_part, float* lse_part, cudaStream_t st) {
    const size_t smem = sizeof(float) * (3 * 64 * (D + 4) + M * (N + 4));
    if (int s = set_smem(cross_fwd_kernel<D>, smem)) return s;
    cross_fwd_kernel<D><<<dim3((unsigned)ceil_div(a.Nq, M) * sp.splits, a.B * a.Hq), kThreads, smem, st>>>(
        a, sp.splits, sp.tiles, o_part, lse_part);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <typename T, int D>
int join(const CrossArgs& a, int splits, const float* o_part, const float* lse_part, cudaStream_t st) {
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    cross_join_kernel<T, D><<<ceil_div(rows, 8), 256, 0, st>>>(a, splits, o_part, lse_part);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <typename T, int D>
int delta(const CrossArgs& a, const HeldTokens* q, const HeldTokens* o, void* qx, cudaStream_t st) {
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    if (q)
        cross_delta_held_kernel<T, D><<<ceil_div(rows * (D / 16), 256 * kHeldUnits), 256, 0, st>>>(
            a, *q, *o, static_cast<T*>(qx));
    else
        cross_delta_kernel<T, D><<<ceil_div(rows * (D / Elem<T>::kPerChunk), 256), 256, 0, st>>>(a);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <int D>
int dq(const CrossArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * (6 * 64 * (D + 4) + M * (N + 4));
    if (int s = set_smem(cross_dq_kernel<D>, smem)) return s;
    cross_dq_kernel<D><<<dim3(ceil_div(a.Nq, M), a.B * a.Hq), kGradThreads, smem, st>>>(a);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <int D>
int dq_join(const CrossArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    cross_dq_join_kernel<D><<<ceil_div(rows * (D / 4), 256), 256, 0, st>>>(a);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <int D, bool DQ>
int dkv(const CrossArgs& a, int ctas, float* part, cudaStream_t st) {
    const size_t smem = sizeof(float) * (5 * 64 * (D + 4) + 2 * M * (N + 4));
    if (int s = set_smem(cross_dkv_kernel<D, DQ>, smem)) return s;
    cross_dkv_kernel<D, DQ><<<ctas, kGradThreads, smem, st>>>(a, part);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <typename T, int D>
int dkv_join(const CrossArgs& a, int rows, int ctas, const float* part, cudaStream_t st) {
    constexpr int BN = sizeof(T) == 4 ? kCrossSimtN : kCrossTcN;
    cross_dkv_join_kernel<T, D, BN><<<dim3(ceil_div(a.Nk, kJoinRows), a.B * a.Hkv), 256, 0, st>>>(a, rows, ctas, part);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

}  // namespace

using bf16 = __nv_bfloat16;
#define SVGEAR_PICK(f, ...)                                                             \
    (dtype == SVGEAR_F32 ? (a.D == 128 ? f<float, 128>(__VA_ARGS__) : f<float, 64>(__VA_ARGS__)) \
                         : (a.D == 128 ? f<bf16, 128>(__VA_ARGS__) : f<bf16, 64>(__VA_ARGS__)))

int launch_cross_simt(const CrossArgs& a, CrossSplit sp, float* o_part, float* lse_part,
                      cudaStream_t st) {
    return a.D == 128 ? fwd<128>(a, sp, o_part, lse_part, st)
                      : fwd<64>(a, sp, o_part, lse_part, st);
}
int launch_cross_join(const CrossArgs& a, int dtype, int splits, const float* o_part,
                      const float* lse_part, cudaStream_t st) {
    return SVGEAR_PICK(join, a, splits, o_part, lse_part, st);
}
int launch_cross_delta(const CrossArgs& a, int dtype, const HeldTokens* q, const HeldTokens* o,
                       void* qx, cudaStream_t st) {
    return SVGEAR_PICK(delta, a, q, o, qx, st);
}
int launch_cross_dkv_join(const CrossArgs& a, int dtype, int rows, int ctas, const float* part,
                          cudaStream_t st) {
    return SVGEAR_PICK(dkv_join, a, rows, ctas, part, st);
}
int launch_cross_backward_simt(const CrossArgs& a, int ctas, float* part, cudaStream_t st) {
    int s;
    if (a.dq_part) {
        s = a.D == 128 ? dkv<128, true>(a, ctas, part, st) : dkv<64, true>(a, ctas, part, st);
        if (s) return s;
        s = a.D == 128 ? dq_join<128>(a, st) : dq_join<64>(a, st);
    } else {
        s = a.D == 128 ? dq<128>(a, st) : dq<64>(a, st);
        if (s) return s;
        s = a.D == 128 ? dkv<128, false>(a, ctas, part, st) : dkv<64, false>(a, ctas, part, st);
    }
    if (s) return s;
    return launch_cross_dkv_join(a, SVGEAR_F32, M, ctas, part, st);
}

}  // namespace svgear
