// cross.h -- shared declarations of the dense cross attention and the 8-bit
// activation checkpoints (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "svgear.h"

namespace svgear {

// One call of the cross attention or its backward pass, after validation.
struct CrossArgs {
    svgear_tokens Q, K, V, O, dO, dQ, dK, dV;   // element strides; unused ones zero
    const int32_t* k_len;                       // [B] or NULL
    float* lse;                                 // [B][Hq][Nq]
    float* delta;                               // [B][Hq][Nq] do.o (workspace)
    float* dq_part;                             // fp32 backward: see cross_dq_part_floats
    int* status;                                // device status words, where a kernel clears them
    int B, Hq, Hkv, G, Nq, Nk, D;
    float scale;
};

#ifdef __CUDACC__
// Keys that take part in batch b: k_len clamped to [0, Nk].
__device__ __forceinline__ int cross_keys(const CrossArgs& a, int b) {
    return a.k_len ? min(max(__ldg(a.k_len + b), 0), a.Nk) : a.Nk;
}
template <typename T>
__device__ __forceinline__ T* row_ptr(const svgear_tokens& t, int b, int h, int64_t n) {
    return static_cast<T*>(t.data) + b * t.stride_b + h * t.stride_h + n * t.stride_n;
}

// 2^(e - 127) of a checkpoint group's exponent byte; 255: the group held a
// value that was not finite.
__device__ __forceinline__ float held_step(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FC00000u : e == 0u ? 0x00400000u : e << 23);
}

// The dK/dV pass covers the iterations (key tile, query head, query tile) of
// every valid key tile, in that order, cut into `ctas` equal ranges, so that
// every CTA does the same number of them whatever the key counts are.  A unit
// is one key tile of one (b, key/value head); it has `per` = G * (query tiles)
// iterations.  A unit whose range lies in one CTA is written by that CTA; the
// others leave fp32 partial sums (slot 0: the piece does not start the unit;
// slot 1: it does), added in CTA order by a second kernel.
struct KvUnit { int b, h, kt, keys; };   // keys: valid keys of the batch

struct KvCursor {
    int b;             // batch holding the current unit
    int64_t base;      // units before batch b
    int64_t units_b;   // units of batch b
    int nt;            // key tiles of batch b
};

template <int BN>
__device__ __forceinline__ int64_t kv_total_units(const CrossArgs& a) {
    if (!a.k_len) return (int64_t)a.B * a.Hkv * ((a.Nk + BN - 1) / BN);
    int64_t n = 0;   // every lane of the calling warp takes part
    for (int b = threadIdx.x & 31; b < a.B; b += 32) n += (cross_keys(a, b) + BN - 1) / BN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n * a.Hkv;
}
template <int BN>
__device__ __forceinline__ void kv_cursor_start(const CrossArgs& a, KvCursor& c) {
    c.b = 0;
    c.base = 0;
    c.nt = (cross_keys(a, 0) + BN - 1) / BN;
    c.units_b = (int64_t)a.Hkv * c.nt;
}
// The unit u (not before the cursor's batch).
template <int BN>
__device__ __forceinline__ KvUnit kv_unit(const CrossArgs& a, KvCursor& c, int64_t u) {
    while (u >= c.base + c.units_b && c.b + 1 < a.B) {
        c.base += c.units_b;
        ++c.b;
        c.nt = (cross_keys(a, c.b) + BN - 1) / BN;
        c.units_b = (int64_t)a.Hkv * c.nt;
    }
    const int r = (int)(u - c.base);
    KvUnit k;
    k.b = c.b;
    k.h = r / c.nt;
    k.kt = r - k.h * c.nt;
    k.keys = cross_keys(a, c.b);
    return k;
}
// First iteration of CTA c's range, of `total` iterations over `ctas`.
__device__ __forceinline__ int64_t kv_range(int64_t total, int c, int ctas) {
    return total / ctas * c + (total % ctas) * c / ctas;
}
#endif

// Rows per CTA and keys per tile of the SIMT kernels.
constexpr int kCrossSimtM = 64, kCrossSimtN = 64;
// fp32 backward: the dK/dV kernel leaves each key tile's part of dQ ([key tile][B][Hq]
// [Nq][d]) for a join, so that the scores are computed once for all three gradients (five
// products instead of seven; gradients of 2,049 x 257 keys, 8 heads, d = 128: 203 us,
// without 277).  Writing and reading a part costs some 1.6 us of an SM where the two
// products cost 9, so parts are faster at any number of tiles and what limits them is
// the workspace: at most kCrossDqTiles times dQ, and kCrossDqBytes.  Past that (0) dQ
// has a kernel of its own.  Measured past the limits, with a build without them: 8 heads,
// 2,049 x 1,024, d = 128 641 us with 16 parts (147 MB of workspace) against 887 (19 MB);
// 25,200 x 512 3.85 ms with 807 MB against 5.00 ms with 19 MB.
constexpr int kCrossDqTiles = 8;
constexpr long long kCrossDqBytes = 512ll << 20;
inline size_t cross_dq_part_floats(const svgear_cross_dims& d) {
    const long long tiles = (d.Nk + (long long)kCrossSimtN - 1) / kCrossSimtN;
    if (d.dtype != SVGEAR_F32 || tiles > kCrossDqTiles) return 0;
    const long long n = tiles * d.B * d.Hq * d.Nq * d.d;
    return n * (long long)sizeof(float) <= kCrossDqBytes ? (size_t)n : 0;
}
// Keys per tile of the tensor-core kernels.
constexpr int kCrossTcN = 128;

// How a forward call is cut: few (head, row tile) items over many keys are
// split along the keys, each split leaving a partial O and lse for the join.
struct CrossSplit {
    int splits;      // 1: no partials
    int tiles;       // key tiles per split
};
// items: CTAs without a split; slots: CTAs the GPU runs at a time.
CrossSplit cross_split(long long items, int key_tiles, int slots, int min_tiles);

// The GPU's streaming multiprocessors (B200): workspaces and grids of the
// persistent kernels are sized for them.
constexpr int kSms = 148;

int launch_cross_simt(const CrossArgs& a, CrossSplit sp, float* o_part, float* lse_part,
                      cudaStream_t st);   // fp32
// cross_sm100.cu (bf16): the partial results a call leaves (1: none), and the
// call; err: device status words.
int cross_sm100_parts(int B, int Hq, int Nq, int Nk);
int launch_cross_sm100(const CrossArgs& a, float* o_part, float* lse_part, int* err, cudaStream_t st);
int launch_cross_join(const CrossArgs& a, int dtype, int splits, const float* o_part,
                      const float* lse_part, cudaStream_t st);

// Backward: delta = do.o per row; with codes, o (and q, unpacked into qx) are
// read from 8-bit checkpoints.
struct HeldTokens {
    const int8_t* codes;    // [B][H][N][d]
    const uint8_t* exps;    // [B][H][N][d / 32]
};
int launch_cross_delta(const CrossArgs& a, int dtype, const HeldTokens* q, const HeldTokens* o,
                       void* qx, cudaStream_t st);
int launch_cross_backward_simt(const CrossArgs& a, int ctas, float* part, cudaStream_t st);   // fp32
int launch_cross_backward_sm100(const CrossArgs& a, float* part, int* err, cudaStream_t st);  // bf16
// Joins the parts of the dK/dV pass (see above); keys: rows of a key tile
// (kCrossSimtN for fp32, kCrossTcN for bf16), rows: of a query tile.
int launch_cross_dkv_join(const CrossArgs& a, int dtype, int rows, int ctas, const float* part,
                          cudaStream_t st);

int launch_checkpoint_save(svgear_tokens X, svgear_dims dims, int8_t* codes, uint8_t* exps,
                           cudaStream_t st);
int launch_checkpoint_load(const int8_t* codes, const uint8_t* exps, svgear_dims dims,
                           svgear_tokens X, cudaStream_t st);

}  // namespace svgear
