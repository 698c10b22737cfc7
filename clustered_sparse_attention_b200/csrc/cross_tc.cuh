// cross_tc.cuh -- what the tcgen05 kernels of the cross attention share: their PTX
// wrappers and waits beside those of tc_ptx.cuh and tc_wait.cuh, tensor maps of
// strided token views and the copy of a key tile whose rows past the batch's key
// count must read as zeros.
#pragma once

#include <atomic>

#include "common.cuh"
#include "cross.h"
#include "ctx_cache.h"
#include "tc_ptx.cuh"
#include "tc_wait.cuh"
#include "tma_host.h"

namespace svgear {

namespace tc {

// 4-D tile load of the tensor map's box at (x, y, z, w).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
// The same box brought into L2 only.
__device__ __forceinline__ void tma_prefetch_4d(const void* tmap, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// Writes the tensor map's box from shared memory to (x, y, z, w); rows past the
// tensor are left out.  Part of the issuing thread's current bulk group.
__device__ __forceinline__ void tma_store_4d(const void* tmap, uint32_t src, int x, int y, int z,
                                             int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until this thread's bulk groups have read shared memory.
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The first four steps of mma_bf16_ts_k128.
__device__ __forceinline__ void mma_bf16_ts_k64(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 t;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.u32 t, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(1u)
        : "memory");
}

// As mma_bf16_ts_k128 with the A operand in two runs of 32 columns, the second
// 64 columns after the first (each run 64 K elements).
__device__ __forceinline__ void mma_bf16_ts_2k64(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 t;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.u32 t, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 64;\n\tadd.s64 b, %2, 512;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 72;\n\tadd.s64 b, %2, 640;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 80;\n\tadd.s64 b, %2, 768;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t"
        "add.u32 t, %1, 88;\n\tadd.s64 b, %2, 896;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, q;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(1u)
        : "memory");
}

// As wait_bar, for loops whose waits last a few thousand cycles and whose
// latency counts: the abort flags and the clock are read every 1024 polls (some
// 30,000 cycles).  Reading the status word and %globaltimer takes long enough
// that a barrier completed meanwhile goes unseen on the critical path (cross
// attention forward, 75,600 x 512 keys: 930 us with a look every 64 polls, 873
// with this).
// The slow look, one copy for all waits of a kernel (inlined, it made up a third
// of its code).  Returns true to go on polling; *t0 is the first look's time.
static __device__ __noinline__ bool poll_look(uint64_t* t0, volatile int* abort_flag, int* err, int where,
                                              uint32_t it) {
    if (*abort_flag || *(volatile int*)err) {
        *abort_flag = 1;
        return false;
    }
    const uint64_t now = global_timer_ns();
    if (*t0 == 0) *t0 = now;
    if (now - *t0 > kWaitTimeoutNs || it >= kMaxSpins) {
        *abort_flag = 1;
        if (atomicCAS(err, 0, SVGEAR_ERR_TIMEOUT) == 0) {
            err[1] = where;
            err[2] = (int)(blockIdx.y * 65536 + blockIdx.x);
        }
        return false;
    }
    return true;
}
__device__ __forceinline__ bool poll_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         int* err, int where) {
    const uint32_t b = smem_u32(bar);
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(b, parity)) return true;
        if ((it & 1023) == 0 && !poll_look(&t0, abort_flag, err, where, it)) return false;
    }
}
// For a whole warp: every lane polls (one shared-memory access for all, and no
// divergence to undo), and all get the same answer.
__device__ __forceinline__ bool warp_poll_bar(uint64_t* bar, uint32_t parity,
                                              volatile int* abort_flag, int* err, int where) {
    return __all_sync(0xffffffffu, poll_bar(bar, parity, abort_flag, err, where)) != 0;
}

// As wait_bar for copies or MMAs already issued, while a kernel gives up: it
// ignores the abort flags and only the clock ends it.
__device__ __forceinline__ bool drain_bar(uint64_t* bar, uint32_t parity) {
    const uint32_t b = smem_u32(bar);
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0; it < kMaxSpins; ++it) {
        if (mbar_try_wait(b, parity)) return true;
        if ((it & 63) == 63 && global_timer_ns() - t0 > kWaitTimeoutNs) return false;
    }
    return false;
}

}  // namespace tc

// A strided bf16 token view [B][H][N][D] as 4-D boxes of 64 columns x box_rows
// rows of one (b, h), 128-byte swizzled; rows past N read as zeros.  An axis
// whose stride is 0 (length 1, or broadcast) is an axis of length 1: its
// coordinate is 0.
inline bool make_tokens_map(CUtensorMap* m, const svgear_tokens& t, int B, int H, int N, int D,
                            uint32_t box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int64_t st[3] = {t.stride_n, t.stride_h, t.stride_b};
    const int len[3] = {N, H, B};
    cuuint64_t dims[4] = {(cuuint64_t)D, 1, 1, 1};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = st[i] ? (cuuint64_t)len[i] : 1;
        strides[i] = (cuuint64_t)(st[i] ? st[i] : D) * 2;
    }
    cuuint32_t box[4] = {64, box_rows, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.data, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace crosstc {

constexpr int BM = 128;   // query rows per tile
constexpr int BN = 128;   // keys per tile

// One token tensor: boxes of 2^i rows (i = 0..7; a whole tile is [7]) and
// whether its head and batch axes move (a broadcast axis stays at 0).
struct RowMaps {
    CUtensorMap box[8];
    int hmul, bmul;
};
struct TileMap {
    CUtensorMap box;
    int hmul, bmul;
};

// pieces: the smaller boxes too, for batches with key counts of their own.
inline bool make_row_maps(RowMaps* m, const svgear_tokens& t, int B, int H, int N, int D, bool pieces) {
    m->hmul = t.stride_h != 0;
    m->bmul = t.stride_b != 0;
    for (int i = pieces ? 0 : 7; i < 8; ++i)
        if (!make_tokens_map(&m->box[i], t, B, H, N, D, 1u << i)) return false;
    return true;
}
inline bool make_tile_map(TileMap* m, const svgear_tokens& t, int B, int H, int N, int D,
                          int rows = BM) {
    m->hmul = t.stride_h != 0;
    m->bmul = t.stride_b != 0;
    return make_tokens_map(&m->box, t, B, H, N, D, rows);
}

// Copies a 128-row tile from row n0 of head (b, h) into shared memory (D / 64
// regions of 128 rows x 128 bytes); rows past the tensor read as zeros.
template <int D>
__device__ __forceinline__ void load_tile(const TileMap& m, uint32_t dst, int b, int h, int n0,
                                          uint32_t bar) {
    tc::mbar_arrive_expect_tx(bar, BM * D * 2);
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
        tc::tma_load_4d(dst + g * 16384, &m.box, g * 64, n0, h * m.hmul, b * m.bmul, bar);
}

// Brings such a tile into L2.
template <int D>
__device__ __forceinline__ void prefetch_tile(const TileMap& m, int b, int h, int n0) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
        tc::tma_prefetch_4d(&m.box, g * 64, n0, h * m.hmul, b * m.bmul);
}

// As load_tile, with rows past `keys` (the batch's key count) reading as
// zeros: they may hold anything, and 0 * NaN would spoil a product.  Where
// the tile ends inside the tensor but past the keys, its valid rows are
// covered by at most two boxes of 2^k rows (one at the start, one ending at
// the end; where they overlap both write the same bytes) and the rest by
// boxes that start past the tensor.
template <int D>
__device__ __forceinline__ void load_key_tile(const RowMaps& m, uint32_t dst, int b, int h, int n0,
                                              int keys, int N, uint32_t bar) {
    const int hc = h * m.hmul, bc = b * m.bmul;
    const int n = keys - n0;
    if (n >= BN || keys == N) {
        tc::mbar_arrive_expect_tx(bar, BN * D * 2);
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            tc::tma_load_4d(dst + g * 16384, &m.box[7], g * 64, n0, hc, bc, bar);
        return;
    }
    const int k0 = 31 - __clz(n), k1 = 31 - __clz(BN - n);
    const uint32_t rows = (uint32_t)((1 << k0) * (n == (1 << k0) ? 1 : 2) +
                                     (1 << k1) * (BN - n == (1 << k1) ? 1 : 2));
    tc::mbar_arrive_expect_tx(bar, rows * D * 2);
#pragma unroll 1
    for (int g = 0; g < D / 64; ++g) {
        const uint32_t t = dst + g * 16384;
        tc::tma_load_4d(t, &m.box[k0], g * 64, n0, hc, bc, bar);
        if (n != (1 << k0))
            tc::tma_load_4d(t + (n - (1 << k0)) * 128, &m.box[k0], g * 64, n0 + n - (1 << k0), hc, bc, bar);
        tc::tma_load_4d(t + n * 128, &m.box[k1], g * 64, N, hc, bc, bar);
        if (BN - n != (1 << k1))
            tc::tma_load_4d(t + (BN - (1 << k1)) * 128, &m.box[k1], g * 64, N, hc, bc, bar);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Output rows leave through a 128-row tile buffer in shared memory (the layout of
// load_tile) and TMA stores, so that whole lines reach L2: a lane that stores its
// own row touches 32 lines per instruction, and transposing in registers first
// measured twice the time.
// 32 bf16 columns [col, col + 32) of this thread's row, packed in pairs.
__device__ __forceinline__ void stage_row32(uint32_t tile, int row, int col, const uint32_t (&pk)[16]) {
    const uint32_t line = tile + (col >> 6) * 16384 + row * 128;
    const int c0 = (col & 63) >> 3;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (((c0 + q) ^ (row & 7)) << 4)),
                     "r"(pk[4 * q]), "r"(pk[4 * q + 1]), "r"(pk[4 * q + 2]), "r"(pk[4 * q + 3])
                     : "memory");
}
// The warp's 32 staged rows [r0, r0 + 32) of the tile to rows n0.. of head
// (b, h); rows past the tensor are left out (`map` has boxes of 32 rows).
template <int D>
__device__ __forceinline__ void store_staged(const TileMap& map, uint32_t tile, int r0, int b, int h, int n0,
                                             bool any_row, int lane) {
    tc::fence_async_smem();
    __syncwarp();
    if (lane == 0 && any_row) {
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            tc::tma_store_4d(&map.box, tile + g * 16384 + r0 * 128, g * 64, n0, h * map.hmul, b * map.bmul);
        tc::bulk_commit();
    }
}

// Zeros in rows [n0, n0 + 32) of head (b, h) that the tensor has, a warp's lanes
// along the rows.
template <int D>
__device__ __forceinline__ void zero_rows32(const svgear_tokens& t, int b, int h, int n0, int N, int lane) {
    constexpr int L = D / 8, R = 32 / L;   // lanes per row, rows at a time
#pragma unroll 4
    for (int i = 0; i < 32; i += R) {
        const int row = n0 + i + lane / L;
        if (row < N)
            *reinterpret_cast<uint4*>(row_ptr<__nv_bfloat16>(t, b, h, row) + lane % L * 8) = make_uint4(0, 0, 0, 0);
    }
}

// S (128 x 128) = A B^T over D, both K-major tiles in shared memory.
template <int D>
__device__ __forceinline__ void mma_dot(uint32_t d_tmem, uint32_t sA, uint32_t sB) {
    constexpr uint32_t kIdesc = tc::idesc_bf16(BM, BN, false);
    if constexpr (D == 128) {
        tc::mma_bf16_k128(d_tmem, tc::sw128_desc(sA, 16, 1024), tc::sw128_desc(sB, 16, 1024), kIdesc, 0u);
    } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
            tc::mma_bf16(d_tmem, tc::sw128_desc(sA + ks * 32, 16, 1024),
                         tc::sw128_desc(sB + ks * 32, 16, 1024), kIdesc, ks > 0);
    }
}
// O (128 x D) (+)= P X over 64 rows of X: P (128 x 64 bf16) in 32 columns of
// tensor memory, X rows of a tile in shared memory, read MN-major.
template <int D>
__device__ __forceinline__ void mma_rows_k64(uint32_t d_tmem, uint32_t a_tmem, uint32_t sX,
                                             uint32_t accumulate) {
    tc::mma_bf16_ts_k64(d_tmem, a_tmem, tc::sw128_desc(sX, 16384, 1024), tc::idesc_bf16(BM, D, true),
                        accumulate);
}
// The same over 128 rows, P in two runs of 32 columns, 64 columns apart (each
// warpgroup's half over the first columns of its scores).
template <int D>
__device__ __forceinline__ void mma_rows_2x64(uint32_t d_tmem, uint32_t a_tmem, uint32_t sX,
                                              uint32_t accumulate) {
    tc::mma_bf16_ts_2k64(d_tmem, a_tmem, tc::sw128_desc(sX, 16384, 1024), tc::idesc_bf16(BM, D, true),
                         accumulate);
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
// (o0, o1) = (x0, x1) * m + a on packed fp32 pairs
__device__ __forceinline__ void fma2(uint32_t x0, uint32_t x1, uint64_t m, uint64_t a, uint32_t& o0,
                                     uint32_t& o1) {
    asm("{\n\t.reg .b64 x, r;\n\tmov.b64 x, {%2, %3};\n\t"
        "fma.rn.f32x2 r, x, %4, %5;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=r"(o0), "=r"(o1) : "r"(x0), "r"(x1), "l"(m), "l"(a));
}
// s += (p0, p1) on a packed fp32 pair
__device__ __forceinline__ void add2(uint64_t& s, float p0, float p1) {
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tadd.rn.f32x2 %0, %0, x;\n\t}"
        : "+l"(s) : "f"(p0), "f"(p1));
}

// One thread's MMAs are complete once `bar` flips; if that wait expires TMEM
// stays allocated and the device's lost word stops every later tensor-core
// kernel before it allocates.
__device__ __forceinline__ void drain_mma(uint64_t* bar, int* keep_tmem, int* err, int* lost, int where) {
    tc::commit(tc::smem_u32(bar));
    if (!tc::drain_bar(bar, 0)) {
        *keep_tmem = 1;
        tc::mark_tmem_lost(lost);
        if (atomicCAS(err, 0, SVGEAR_ERR_TIMEOUT) == 0) {
            err[1] = where;
            err[2] = blockIdx.x;
        }
    }
}

// Rewrites columns >= valid of this warp's N score columns at taddr to -inf: in
// TMEM, so that the main path carries no selects.
template <int N>
__device__ __forceinline__ void mask_columns(uint32_t taddr, int valid) {
#pragma unroll 1
    for (int c4 = max(valid, 0) / 32; c4 < N / 32; ++c4) {
        uint32_t t[32];
        tc::tmem_ld32(taddr + c4 * 32, t);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (c4 * 32 + e >= valid) t[e] = __float_as_uint(-INFINITY);
        tc::tmem_st32(taddr + c4 * 32, t);
    }
    tc::tmem_st_wait();
}

// Dynamic shared memory of a kernel whose tiles fill it: the 128-byte swizzle
// needs 1024-byte aligned tiles, and the dynamic part starts after the static
// one, which is padded to a multiple of that.  Done once per function and
// context (`done`: the id of the last one; the two calls took 2 us of each
// launch).
inline int set_aligned_smem(const void* fn, uint32_t bytes, std::atomic<unsigned long long>& done) {
    unsigned long long ctx = 0;
    const bool have = SymbolAddressCache::current_id(&ctx);
    if (have && done.load(std::memory_order_relaxed) == ctx) return SVGEAR_OK;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess) return SVGEAR_ERR_CUDA;
    if (fa.sharedSizeBytes % 1024 != 0) return SVGEAR_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return SVGEAR_ERR_CUDA;
    if (have) done.store(ctx, std::memory_order_relaxed);
    return SVGEAR_OK;
}

// A slot ring's position: slot index and the parity of its current use.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
};

}  // namespace crosstc
}  // namespace svgear
