// cross_bwd_sm100.cu -- gradients of the dense cross attention for bf16 tokens
// on tcgen05 / TMEM (sm_100a), from the forward pass's lse and delta = do.o:
//   p_ij = e^{s_ij - lse_i}, ds_ij = p_ij (do_i.v_j - delta_i),
//   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i,
//   dv_j = sum_i p_ij do_i.
// p and ds enter their second product rounded to bf16 (an error of the size of
// the outputs' own rounding); everything else, all sums among it, is fp32.  The
// accumulators cut additions off (one for 16 rows), so equal terms come out low by
// 3.3e-9 a term: 2.5e-4 for dK over 75,600 rows, a sixteenth of the output's rounding,
// 2.1e-3 over 604,800 (a CTA adds no more rows than its share of the call).
//
// Two kernels, each recomputing the scores from Q and K: one keeps a key tile
// and walks the queries (dK, dV), the other keeps a query tile and walks the
// keys (dQ).  One kernel for all three would need five products per tile pair
// instead of seven, but dQ sums over key tiles that other CTAs hold: by atomics
// its result would change from run to run, and TMEM has no room for it (S, dP,
// dV and dK fill the 512 columns).
//
// Roles and barriers are those of the forward kernel: two warpgroups turn score
// tiles into weights, each 64 of a tile's 128 columns, one row per thread; one
// thread per chain of products issues its MMAs; one thread copies tiles by TMA.
// Every wait is bounded (tc_wait.cuh).
#include <math.h>

#include "cross_tc.cuh"
#include "launchers.h"

namespace svgear {
namespace crosstc {
namespace {

using bf16 = __nv_bfloat16;
using tc::poll_bar;
using tc::warp_poll_bar;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int HN = 64;   // columns of a tile per warpgroup
constexpr uint32_t kTmemCols = 512;

// (a, b) - (c, c) on packed fp32 pairs
__device__ __forceinline__ uint64_t sub2(uint32_t a, uint32_t b, uint64_t neg) {
    uint64_t r;
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tadd.rn.f32x2 %0, x, %3;\n\t}"
        : "=l"(r) : "r"(a), "r"(b), "l"(neg));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float lo(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }

// ---------------------------------------------------------------------------
// dK, dV: a persistent CTA per SM takes an equal share of the iterations (key
// tile, query head, query tile); see KvUnit.  K and V of the unit stay in
// shared memory; Q and dO tiles stream through a ring each, with lse and delta of
// their rows in a third.  Rows (TMEM lanes) are keys, columns queries:
//   S^T = K Q^T -> P^T (over S^T) -> dV += P^T dO
//   dP^T = V dO^T -> dS^T (over dP^T) -> dK += dS^T Q
// One thread issues dV(i) and S(i + 1), another dK(i) and dP(i + 1) once S(i + 1)
// is issued, so that S(i + 1) comes first and the weights of i + 1 are computed
// beside dK(i) and dP(i + 1).  (Without that order the four products ran
// interleaved and the weights had the tensor pipe idle, 4,000 cycles an
// iteration; with one thread for all, its barrier tests and commits left the
// pipe idle, 3,300; now 2,980.)
// TMEM: S | dP | dV | dK.
// Bound: the chain S -> P -> dS -> dK between products that take 2,048 cycles of an
// iteration; in long runs also the power limit.  75,600 x 512 keys, 40 heads, d = 128:
// 1.31-1.40 ms in runs of some 20 ms (1.2 PFLOP/s for its four products); the whole
// pass, dQ and delta with it, 2.82 ms there and 3.33 at the power limit's clock (seven
// products at 830 TFLOP/s, 0.61 of a library product's sustained rate).
// A copy takes some 2,000 cycles to arrive.  Q(i) is held from S(i) to dK(i), so
// its ring has three slots where dO's has two: with two of both, S(i + 1) waited
// for its Q in every iteration (4,300 cycles each against 2,048 of MMA work).
// ---------------------------------------------------------------------------
constexpr int kKvThreads = 12 * 32;   // 0-7 weights, 8 TMA, 9 and 10 MMA, 11 lse and delta

template <int D>
constexpr int kv_q_slots() { return D == 128 ? 3 : 4; }
template <int D>
constexpr int kv_g_slots() { return D == 128 ? 2 : 4; }
template <int D>
constexpr uint32_t kv_smem() { return (2 + kv_q_slots<D>() + kv_g_slots<D>()) * (D / 64) * 16384; }

struct KvMaps {
    TileMap q, g, k, v;
};

struct KvShared {
    uint64_t kv_full;
    uint64_t q_full[4], q_empty[4], g_full[4], g_empty[4];
    uint64_t l_full[2], l_empty[2];
    uint64_t s_full, p_full, dp_full, ds_full;
    // S of the next iteration (if any) is on its way.  In turn: nothing holds the
    // arriving thread back until i has been seen, and on one barrier the completion
    // of i + 1 would make i's look open again; i + 2 follows dP(i + 1), which
    // follows the wait for i.
    uint64_t s_issued[2];
    uint64_t acc_full, acc_free;
    uint64_t drain[2];
    alignas(16) float neg_lse2[2][BM];   // -lse log2 e of a query tile's rows
    alignas(16) float neg_delta[2][BM];
    uint32_t tmem_base;
    int abort_flag;
    int keep_tmem;
};

// A CTA's share as pieces of units.
struct Pieces {
    int64_t it, end, per;
    KvCursor cur;
    KvUnit k;
    int64_t first, last;   // iterations of the unit in this piece
    __device__ __forceinline__ Pieces(const CrossArgs& a, int64_t units) {
        per = (int64_t)a.G * ((a.Nq + BM - 1) / BM);
        const int64_t total = units * per;
        it = kv_range(total, blockIdx.x, gridDim.x);
        end = kv_range(total, blockIdx.x + 1, gridDim.x);
        kv_cursor_start<BN>(a, cur);
    }
    __device__ __forceinline__ bool next(const CrossArgs& a) {
        if (it >= end) return false;
        const int64_t u = it / per;
        first = it - u * per;
        last = min(per, first + (end - it));
        k = kv_unit<BN>(a, cur, u);
        it += last - first;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kKvThreads, 1)
cross_dkv_sm100_kernel(const __grid_constant__ KvMaps maps, CrossArgs a, float* __restrict__ part,
                       int* __restrict__ err, int* __restrict__ lost) {
    constexpr uint32_t kTile = (D / 64) * 16384;
    constexpr int NQ = kv_q_slots<D>(), NG = kv_g_slots<D>();
    if (tc::refuse_start(lost, err)) return;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ KvShared sh;
    const uint32_t base = tc::smem_u32(smem_raw);   // 1024-byte aligned: see launch_dkv()
    const uint32_t sK = base, sV = sK + kTile, sQ = sV + kTile, sG = sQ + NQ * kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t units = kv_total_units<BN>(a);
    if (tid == 0) {
        tc::mbar_init(tc::smem_u32(&sh.kv_full), 2);
        for (int s = 0; s < NQ; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.q_full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.q_empty[s]), 1);   // dK, which follows S
        }
        for (int s = 0; s < NG; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.g_full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.g_empty[s]), 2);   // dV and dP
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.l_full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.l_empty[s]), 8);
            tc::mbar_init(tc::smem_u32(&sh.s_issued[s]), 1);
        }
        tc::mbar_init(tc::smem_u32(&sh.s_full), 1);
        tc::mbar_init(tc::smem_u32(&sh.p_full), 8);
        tc::mbar_init(tc::smem_u32(&sh.dp_full), 1);
        tc::mbar_init(tc::smem_u32(&sh.ds_full), 8);
        tc::mbar_init(tc::smem_u32(&sh.acc_full), 2);
        tc::mbar_init(tc::smem_u32(&sh.acc_free), 8);
        tc::mbar_init(tc::smem_u32(&sh.drain[0]), 1);
        tc::mbar_init(tc::smem_u32(&sh.drain[1]), 1);
        sh.abort_flag = 0;
        sh.keep_tmem = 0;
        tc::mbar_init_fence();
    }
    if (warp == 9) {
        tc::tmem_alloc(tc::smem_u32(&sh.tmem_base), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    volatile int* abort_flag = &sh.abort_flag;
    const int qtiles = (a.Nq + BM - 1) / BM;
    const float scale_log2 = a.scale * kLog2e;
    Pieces p(a, units);

    if (warp == 8 && lane == 0) {
        // ------------------------------------------------------------ producer
        Ring qr, gr;
        uint32_t qfills = 0, gfills = 0, n = 0;
        bool ok = true;
        while (ok && p.next(a)) {
            // the last unit's products have read K and V
            if (n > 0 && !(ok = poll_bar(&sh.acc_full, (n - 1) & 1, abort_flag, err, (1 << 16)))) break;
            load_tile<D>(maps.k, sK, p.k.b, p.k.h, p.k.kt * BN, tc::smem_u32(&sh.kv_full));
            load_tile<D>(maps.v, sV, p.k.b, p.k.h, p.k.kt * BN, tc::smem_u32(&sh.kv_full));
            ++n;
            int g = (int)(p.first / qtiles), qt = (int)(p.first - (int64_t)g * qtiles);
            for (int64_t x = p.first; x < p.last; ++x) {
                if (qfills >= NQ && !(ok = poll_bar(&sh.q_empty[qr.slot], qr.phase ^ 1, abort_flag, err, (2 << 16))))
                    break;
                load_tile<D>(maps.q, sQ + qr.slot * kTile, p.k.b, p.k.h * a.G + g, qt * BM,
                             tc::smem_u32(&sh.q_full[qr.slot]));
                ++qfills;
                qr.next(NQ);
                if (gfills >= NG && !(ok = poll_bar(&sh.g_empty[gr.slot], gr.phase ^ 1, abort_flag, err, (2 << 16) + 1)))
                    break;
                load_tile<D>(maps.g, sG + gr.slot * kTile, p.k.b, p.k.h * a.G + g, qt * BM,
                             tc::smem_u32(&sh.g_full[gr.slot]));
                ++gfills;
                gr.next(NG);
                if (++qt == qtiles) {
                    qt = 0;
                    ++g;
                }
            }
        }
        // gave up: let the copies in flight land before the CTA ends
        if (!ok) {
            if (n > 0) tc::drain_bar(&sh.kv_full, (n - 1) & 1);
            for (uint32_t f = qfills > NQ ? qfills - NQ : 0; f < qfills; ++f)
                tc::drain_bar(&sh.q_full[f % NQ], (f / NQ) & 1);
            for (uint32_t f = gfills > NG ? gfills - NG : 0; f < gfills; ++f)
                tc::drain_bar(&sh.g_full[f % NG], (f / NG) & 1);
        }
    } else if (warp == 11) {
        // -------------------------------------------------------- lse and delta
        uint32_t i = 0;
        bool ok = true;
        while (ok && p.next(a)) {
            int g = (int)(p.first / qtiles), qt = (int)(p.first - (int64_t)g * qtiles);
            for (int64_t x = p.first; x < p.last; ++x, ++i) {
                const size_t r0 = ((size_t)p.k.b * a.Hq + p.k.h * a.G + g) * a.Nq + (size_t)qt * BM;
                float l[4], d[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {   // rows past the end: p = e^{-inf} = 0
                    const bool in = qt * BM + 32 * c + lane < a.Nq;
                    l[c] = in ? __ldg(a.lse + r0 + 32 * c + lane) * -kLog2e : -INFINITY;
                    d[c] = in ? -__ldg(a.delta + r0 + 32 * c + lane) : 0.f;
                }
                if (i >= 2 && !(ok = warp_poll_bar(&sh.l_empty[i & 1], ((i >> 1) - 1) & 1, abort_flag, err, (3 << 16))))
                    break;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sh.neg_lse2[i & 1][32 * c + lane] = l[c];
                    sh.neg_delta[i & 1][32 * c + lane] = d[c];
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.l_full[i & 1]));
                if (++qt == qtiles) {
                    qt = 0;
                    ++g;
                }
            }
        }
    } else if (warp == 9 && lane == 0) {
        // ------------------------------------------------------ MMA: S and dV
        Ring qr, gr;
        uint32_t n = 0, i = 0;
        bool ok = true;
        auto issue_s = [&]() {
            mma_dot<D>(tmem, sK, sQ + qr.slot * kTile);
            tc::commit(tc::smem_u32(&sh.s_full));
            qr.next(NQ);
        };
        while (ok && p.next(a)) {
            ok = poll_bar(&sh.kv_full, n & 1, abort_flag, err, (4 << 16)) &&
                 poll_bar(&sh.q_full[qr.slot], qr.phase, abort_flag, err, (5 << 16));
            if (!ok) break;
            tc::fence_after_sync();
            issue_s();
            // the first sum overwrites dV: the last must be read out
            if (n > 0 && !(ok = poll_bar(&sh.acc_free, (n - 1) & 1, abort_flag, err, (6 << 16)))) break;
            for (int64_t x = p.first; x < p.last; ++x, ++i) {
                const bool more = x + 1 < p.last;
                if (!(ok = poll_bar(&sh.g_full[gr.slot], gr.phase, abort_flag, err, (5 << 16) + 1)) ||
                    (more && !(ok = poll_bar(&sh.q_full[qr.slot], qr.phase, abort_flag, err, (5 << 16)))) ||
                    !(ok = poll_bar(&sh.p_full, i & 1, abort_flag, err, (7 << 16))))
                    break;
                tc::fence_after_sync();
                mma_rows_2x64<D>(tmem + 2 * BN, tmem, sG + gr.slot * kTile, x > p.first ? 1u : 0u);
                if (more) issue_s();
                tc::mbar_arrive(tc::smem_u32(&sh.s_issued[i & 1]));
                tc::commit(tc::smem_u32(&sh.g_empty[gr.slot]));
                gr.next(NG);
            }
            if (!ok) break;
            tc::commit(tc::smem_u32(&sh.acc_full));
            ++n;
        }
        drain_mma(&sh.drain[0], &sh.keep_tmem, err, lost, 9 << 16);
    } else if (warp == 10 && lane == 0) {
        // ----------------------------------------------------- MMA: dP and dK
        Ring qr, gr;
        uint32_t n = 0, i = 0;
        bool ok = true;
        auto issue_dp = [&]() {
            mma_dot<D>(tmem + BN, sV, sG + gr.slot * kTile);
            tc::commit(tc::smem_u32(&sh.dp_full));
            tc::commit(tc::smem_u32(&sh.g_empty[gr.slot]));
            gr.next(NG);
        };
        while (ok && p.next(a)) {
            ok = poll_bar(&sh.kv_full, n & 1, abort_flag, err, (4 << 16) + 1) &&
                 poll_bar(&sh.g_full[gr.slot], gr.phase, abort_flag, err, (5 << 16) + 2);
            if (!ok) break;
            tc::fence_after_sync();
            issue_dp();
            if (n > 0 && !(ok = poll_bar(&sh.acc_free, (n - 1) & 1, abort_flag, err, (6 << 16) + 1))) break;
            for (int64_t x = p.first; x < p.last; ++x, ++i) {
                const bool more = x + 1 < p.last;
                if ((more && !(ok = poll_bar(&sh.g_full[gr.slot], gr.phase, abort_flag, err, (5 << 16) + 2))) ||
                    !(ok = poll_bar(&sh.ds_full, i & 1, abort_flag, err, (8 << 16))) ||
                    !(ok = poll_bar(&sh.s_issued[i & 1], (i >> 1) & 1, abort_flag, err, (8 << 16) + 1)))
                    break;
                tc::fence_after_sync();
                // (Q(i) is in shared memory since S(i))
                mma_rows_2x64<D>(tmem + 2 * BN + D, tmem + BN, sQ + qr.slot * kTile, x > p.first ? 1u : 0u);
                if (more) issue_dp();
                tc::commit(tc::smem_u32(&sh.q_empty[qr.slot]));
                qr.next(NQ);
            }
            if (!ok) break;
            tc::commit(tc::smem_u32(&sh.acc_full));
            ++n;
        }
        drain_mma(&sh.drain[1], &sh.keep_tmem, err, lost, (9 << 16) + 1);
    } else if (warp < 8) {
        // -------------------------------------------------------------- weights
        const int h = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_base + h * HN, tP = lane_base + BN + h * HN;
        const uint64_t xs2 = pack2(scale_log2, scale_log2);
        uint32_t n = 0, i = 0;
        bool ok = true;
        while (ok && p.next(a)) {
            for (int64_t x = p.first; x < p.last; ++x, ++i) {
                if (!(ok = warp_poll_bar(&sh.l_full[i & 1], (i >> 1) & 1, abort_flag, err, (10 << 16)) &&
                           warp_poll_bar(&sh.s_full, i & 1, abort_flag, err, (11 << 16))))
                    break;
                tc::fence_after_sync();
                const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(&sh.neg_lse2[i & 1][h * HN]);
                const ulonglong2* nd = reinterpret_cast<const ulonglong2*>(&sh.neg_delta[i & 1][h * HN]);
                uint32_t v[HN];
                tc::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                tc::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                tc::tmem_ld_wait();
                // P^T = 2^(s scale log2 e - lse log2 e)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 l4 = nl[q * 8 + e / 4];
                        uint32_t* y = &v[q * 32 + e];
                        fma2(y[0], y[1], xs2, l4.x, y[0], y[1]);
                        fma2(y[2], y[3], xs2, l4.y, y[2], y[3]);
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] = __float_as_uint(tc::ex2(__uint_as_float(y[z])));
                        pk[e / 2] = bf16_pair(__uint_as_float(y[0]), __uint_as_float(y[1]));
                        pk[e / 2 + 1] = bf16_pair(__uint_as_float(y[2]), __uint_as_float(y[3]));
                    }
                    tc::tmem_st16(tS + q * 16, pk);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.p_full));
                if (!(ok = warp_poll_bar(&sh.dp_full, i & 1, abort_flag, err, (12 << 16)))) break;
                tc::fence_after_sync();
                // dS^T = P^T (dP^T - delta)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t d[32], pk[16];
                    tc::tmem_ld32(tP + q * 32, d);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 d4 = nd[q * 8 + e / 4];
                        const uint32_t* y = &v[q * 32 + e];
                        const uint64_t s0 = mul2(sub2(d[e], d[e + 1], d4.x),
                                                 (uint64_t)y[0] | ((uint64_t)y[1] << 32));
                        const uint64_t s1 = mul2(sub2(d[e + 2], d[e + 3], d4.y),
                                                 (uint64_t)y[2] | ((uint64_t)y[3] << 32));
                        pk[e / 2] = bf16_pair(lo(s0), hi(s0));
                        pk[e / 2 + 1] = bf16_pair(lo(s1), hi(s1));
                    }
                    tc::tmem_st16(tP + q * 16, pk);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(tc::smem_u32(&sh.ds_full));
                    tc::mbar_arrive(tc::smem_u32(&sh.l_empty[i & 1]));
                }
            }
            if (!ok) break;
            // the unit's sums (or this CTA's part of them): warpgroup 0 writes
            // dV, warpgroup 1 dK
            if (!(ok = warp_poll_bar(&sh.acc_full, n & 1, abort_flag, err, (13 << 16)))) break;
            tc::fence_after_sync();
            ++n;
            const bool whole = p.first == 0 && p.last == p.per;
            const float f = h == 0 ? 1.f : a.scale;
            const int row = p.k.kt * BN + r;
            float* dst_part = part + ((((size_t)blockIdx.x * 2 + (p.first == 0 ? 1 : 0)) * 2 + (1 - h)) * BN + r) * D;
            bf16* dst = row_ptr<bf16>(h == 0 ? a.dV : a.dK, p.k.b, p.k.h, row);
            const uint32_t tA = lane_base + 2 * BN + h * D;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tc::tmem_ld16(tA + c * 16, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                if (!whole) {
                    uint4* o4 = reinterpret_cast<uint4*>(dst_part + c * 16);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o4[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                } else if (row < p.k.keys) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pk[e] = bf16_pair(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                    uint4* o4 = reinterpret_cast<uint4*>(dst + c * 16);
                    o4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    o4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.acc_free));
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 9 && !sh.keep_tmem) tc::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// dQ: an item is 128 query rows of one head; a persistent CTA per SM takes
// items in turn.  Q and dO of the item stay in shared memory, K and V tiles
// stream through two rings.  Rows (TMEM lanes) are queries, columns keys:
//   S = Q K^T, dP = dO V^T (two buffers), dS = p (dP - delta) over dP,
//   dQ += dS K.
// S(g + 1) is issued as soon as the weights have read S(g) into registers, dP(g + 2)
// when dQ(g) has read dS(g), so that neither follows the weights of its own tile:
// over the tiles of all items, the arithmetic of g runs beside the products of
// g - 1 and g + 1.  Each product has its own issuing thread: a barrier test costs
// its thread 100 to 300 cycles, a commit 65, and one thread for all three took
// 3,400 cycles per tile for 1,536 of MMA work.  (With S in two buffers and dS over S, S(g + 2) came behind
// dP(g + 1) and dQ(g) and the weights waited for it: some 3,000.)  Now 2,815 at
// 75,600 x 512 keys, where an item ends every four tiles (1.16 ms in runs of some 20 ms,
// 40 heads, d = 128).
// Bound: the weights, which copy two 128 x 128 tiles from TMEM and one back between the
// barriers of three products.
// TMEM: S | dP[0] | dP[1] | dQ.
// The epilogue warps also fetch each item's key count and its rows' lse and delta
// an item ahead, so that the weights' warps find them in shared memory.  (With
// delta = do.o computed there too, from O and dO, they were the slowest warps:
// 1,540 us for 75,600 x 512 keys against 1,160 and a delta pass of 255.)
// ---------------------------------------------------------------------------
constexpr int kQThreads = 16 * 32;   // 0-7 weights, 8 TMA, 9-11 MMA, 12-15 epilogue

// K(g) is held from S(g) to dQ(g): its ring needs a third slot for the copy of
// K(g + 2) to arrive in time.
template <int D>
constexpr int q_k_slots() { return D == 128 ? 3 : 4; }
template <int D>
constexpr int q_v_slots() { return D == 128 ? 2 : 4; }
template <int D>
constexpr uint32_t q_smem() { return (2 + q_k_slots<D>() + q_v_slots<D>()) * (D / 64) * 16384; }

struct QMaps {
    RowMaps k, v;
    TileMap q, g;
};

struct QShared {
    uint64_t q_full, q_empty, g_full, g_empty;
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full, s_read;
    uint64_t dp_full[2], ds_full[2], dq_done[2];
    uint64_t acc_full, acc_free;
    uint64_t row_full[2], row_free[2];   // the item's rows below, in turn
    uint64_t drain[3];
    float neg_lse2[2][BM], neg_delta[2][BM];
    int keys[2];
    uint32_t tmem_base;
    int abort_flag;
    int keep_tmem;
};

// The items of one CTA: item = (b * Hq + h) * qtiles + tile, advanced by the
// grid digit by digit.
struct QItem {
    int item, qt, h, b, dq, dh, db, qtiles, items;
    int hk, keys, T;
    __device__ __forceinline__ void derive(const CrossArgs& a) {
        keys = cross_keys(a, b);
        T = (keys + BN - 1) / BN;
        hk = a.G == 1 ? h : h / a.G;
    }
    __device__ __forceinline__ bool start(const CrossArgs& a) {
        qtiles = (a.Nq + BM - 1) / BM;
        items = a.B * a.Hq * qtiles;
        item = blockIdx.x;
        int x = item;
        qt = x % qtiles; x /= qtiles;
        h = x % a.Hq;
        b = x / a.Hq;
        x = gridDim.x;
        dq = x % qtiles; x /= qtiles;
        dh = x % a.Hq;
        db = x / a.Hq;
        if (item < items) derive(a);
        return item < items;
    }
    __device__ __forceinline__ bool next(const CrossArgs& a) {
        item += gridDim.x;
        qt += dq; h += dh; b += db;
        if (qt >= qtiles) { qt -= qtiles; ++h; }
        if (h >= a.Hq) { h -= a.Hq; ++b; }
        if (item < items) derive(a);
        return item < items;
    }
};

template <int D>
__global__ void __launch_bounds__(kQThreads, 1)
cross_dq_sm100_kernel(const __grid_constant__ QMaps maps, CrossArgs a, int* __restrict__ err,
                      int* __restrict__ lost) {
    constexpr uint32_t kTile = (D / 64) * 16384;
    constexpr int NK = q_k_slots<D>(), NV = q_v_slots<D>();
    if (tc::refuse_start(lost, err)) return;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ QShared sh;
    const uint32_t base = tc::smem_u32(smem_raw);   // 1024-byte aligned: see launch_dq()
    const uint32_t sQ = base, sG = sQ + kTile, sK = sG + kTile, sV = sK + NK * kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        uint64_t* one[] = {&sh.q_full, &sh.q_empty, &sh.g_full, &sh.g_empty, &sh.s_full,
                           &sh.dp_full[0], &sh.dp_full[1], &sh.dq_done[0], &sh.dq_done[1],
                           &sh.acc_full, &sh.drain[0], &sh.drain[1], &sh.drain[2]};
        for (uint64_t* x : one) tc::mbar_init(tc::smem_u32(x), 1);
        tc::mbar_init(tc::smem_u32(&sh.s_read), 8);
        tc::mbar_init(tc::smem_u32(&sh.ds_full[0]), 8);
        tc::mbar_init(tc::smem_u32(&sh.ds_full[1]), 8);
        tc::mbar_init(tc::smem_u32(&sh.acc_free), 4);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.row_full[i]), 4);
            tc::mbar_init(tc::smem_u32(&sh.row_free[i]), 8);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.k_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.k_empty[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.v_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.v_empty[i]), 1);
        }
        sh.abort_flag = 0;
        sh.keep_tmem = 0;
        tc::mbar_init_fence();
    }
    if (warp == 9) {
        tc::tmem_alloc(tc::smem_u32(&sh.tmem_base), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    volatile int* abort_flag = &sh.abort_flag;
    QItem w;

    if (warp == 8 && lane == 0) {
        // ------------------------------------------------------------ producer
        Ring kr, vr;
        uint32_t kfills = 0, vfills = 0, n = 0;
        bool ok = true, q_loaded = false, g_loaded = false;
        for (bool more = w.start(a); ok && more; more = w.next(a)) {
            if (w.T == 0) continue;
            q_loaded = g_loaded = false;
            if (n > 0 && !(ok = poll_bar(&sh.q_empty, (n - 1) & 1, abort_flag, err, (1 << 16)))) break;
            load_tile<D>(maps.q, sQ, w.b, w.h, w.qt * BM, tc::smem_u32(&sh.q_full));
            q_loaded = true;
            auto load_k = [&](int j) {
                if (kfills >= NK && !(ok = poll_bar(&sh.k_empty[kr.slot], kr.phase ^ 1, abort_flag, err, (2 << 16))))
                    return;
                load_key_tile<D>(maps.k, sK + kr.slot * kTile, w.b, w.hk, j * BN, w.keys, a.Nk,
                                 tc::smem_u32(&sh.k_full[kr.slot]));
                ++kfills;
                kr.next(NK);
            };
            auto load_v = [&](int j) {
                if (vfills >= NV && !(ok = poll_bar(&sh.v_empty[vr.slot], vr.phase ^ 1, abort_flag, err, (3 << 16))))
                    return;
                load_key_tile<D>(maps.v, sV + vr.slot * kTile, w.b, w.hk, j * BN, w.keys, a.Nk,
                                 tc::smem_u32(&sh.v_full[vr.slot]));
                ++vfills;
                vr.next(NV);
            };
            load_k(0);
            if (!ok || (n > 0 && !(ok = poll_bar(&sh.g_empty, (n - 1) & 1, abort_flag, err, (1 << 16) + 1)))) break;
            load_tile<D>(maps.g, sG, w.b, w.h, w.qt * BM, tc::smem_u32(&sh.g_full));
            g_loaded = true;
            // the next item's rows on their way from HBM to L2
            QItem x = w;
            if (x.next(a) && x.T > 0) {
                prefetch_tile<D>(maps.q, x.b, x.h, x.qt * BM);
                prefetch_tile<D>(maps.g, x.b, x.h, x.qt * BM);
            }
            load_v(0);
            for (int j = 1; ok && j < w.T; ++j) {   // V's slots come free before K's
                load_v(j);
                if (ok) load_k(j);
            }
            if (!ok) break;
            ++n;
        }
        // gave up: let the copies in flight land before the CTA ends
        if (!ok) {
            if (q_loaded) tc::drain_bar(&sh.q_full, n & 1);
            if (g_loaded) tc::drain_bar(&sh.g_full, n & 1);
            for (uint32_t f = kfills > NK ? kfills - NK : 0; f < kfills; ++f)
                tc::drain_bar(&sh.k_full[f % NK], (f / NK) & 1);
            for (uint32_t f = vfills > NV ? vfills - NV : 0; f < vfills; ++f)
                tc::drain_bar(&sh.v_full[f % NV], (f / NV) & 1);
        }
    } else if (warp >= 9 && warp < 12 && lane == 0) {
        // ----------------------------------------- MMA issue: S, dP or dQ
        const int role = warp - 9;
        Ring ring;
        uint32_t n = 0, g = 0;
        bool ok = true;
        for (bool more = w.start(a); ok && more; more = w.next(a)) {
            if (w.T == 0) continue;
            // the item's Q, its dO, or dQ of the last item read out
            ok = role == 0   ? poll_bar(&sh.q_full, n & 1, abort_flag, err, (4 << 16))
                 : role == 1 ? poll_bar(&sh.g_full, n & 1, abort_flag, err, (4 << 16) + 1)
                             : n == 0 || poll_bar(&sh.acc_free, (n - 1) & 1, abort_flag, err, (4 << 16) + 2);
            if (role == 0) {
                for (int j = 0; ok && j < w.T; ++j, ++g) {
                    // S(g) overwrites S(g - 1), which must be in registers
                    if (!(ok = poll_bar(&sh.k_full[ring.slot], ring.phase, abort_flag, err, (5 << 16)) &&
                               (g == 0 || poll_bar(&sh.s_read, (g - 1) & 1, abort_flag, err, (6 << 16)))))
                        break;
                    tc::fence_after_sync();
                    mma_dot<D>(tmem, sQ, sK + ring.slot * kTile);
                    tc::commit(tc::smem_u32(&sh.s_full));
                    ring.next(NK);
                }
                if (ok) tc::commit(tc::smem_u32(&sh.q_empty));
            } else if (role == 1) {
                for (int j = 0; ok && j < w.T; ++j, ++g) {
                    // dP(g) overwrites dS(g - 2), which dQ must have read
                    const uint32_t b = g & 1;
                    if (!(ok = poll_bar(&sh.v_full[ring.slot], ring.phase, abort_flag, err, (5 << 16) + 1) &&
                               (g < 2 || poll_bar(&sh.dq_done[b], ((g >> 1) & 1) ^ 1, abort_flag, err, (6 << 16) + 1))))
                        break;
                    tc::fence_after_sync();
                    mma_dot<D>(tmem + BN + b * BN, sG, sV + ring.slot * kTile);
                    tc::commit(tc::smem_u32(&sh.dp_full[b]));
                    tc::commit(tc::smem_u32(&sh.v_empty[ring.slot]));
                    ring.next(NV);
                }
                if (ok) tc::commit(tc::smem_u32(&sh.g_empty));
            } else {
                for (int j = 0; ok && j < w.T; ++j, ++g) {
                    const uint32_t b = g & 1;
                    if (!(ok = poll_bar(&sh.ds_full[b], (g >> 1) & 1, abort_flag, err, (7 << 16)))) break;
                    tc::fence_after_sync();
                    // (K(g) is in shared memory since S(g))
                    mma_rows_2x64<D>(tmem + 3 * BN, tmem + BN + b * BN, sK + ring.slot * kTile, j > 0 ? 1u : 0u);
                    tc::commit(tc::smem_u32(&sh.k_empty[ring.slot]));
                    tc::commit(tc::smem_u32(&sh.dq_done[b]));
                    ring.next(NK);
                }
                if (ok) tc::commit(tc::smem_u32(&sh.acc_full));
            }
            ++n;
        }
        drain_mma(&sh.drain[role], &sh.keep_tmem, err, lost, (9 << 16) + role);
    } else if (warp < 8) {
        // -------------------------------------------------------------- weights
        const int h = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_base + h * HN;
        const float scale_log2 = a.scale * kLog2e;
        const uint64_t xs2 = pack2(scale_log2, scale_log2);
        uint32_t g = 0, m = 0;
        bool ok = true;
        const int items = a.B * a.Hq * ((a.Nq + BM - 1) / BM);
        for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++m) {
            if (!(ok = warp_poll_bar(&sh.row_full[m & 1], (m >> 1) & 1, abort_flag, err, (14 << 16)))) break;
            const float neg_lse = sh.neg_lse2[m & 1][r], neg_delta = sh.neg_delta[m & 1][r];
            const int keys = sh.keys[m & 1];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.row_free[m & 1]));
            const uint64_t nl2 = pack2(neg_lse, neg_lse), nd2 = pack2(neg_delta, neg_delta);
            for (int j = 0; j * BN < keys; ++j, ++g) {
                const uint32_t b = g & 1, tP = tS + BN + b * BN;
                if (!(ok = warp_poll_bar(&sh.s_full, g & 1, abort_flag, err, (11 << 16)))) break;
                tc::fence_after_sync();
                const int valid = keys - j * BN - h * HN;
                if (valid < HN) mask_columns<HN>(tS, valid);   // past the keys: p = 0
                uint32_t v[HN];
                tc::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                tc::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                tc::tmem_ld_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.s_read));
#pragma unroll
                for (int e = 0; e < HN; e += 2) {
                    fma2(v[e], v[e + 1], xs2, nl2, v[e], v[e + 1]);
                    v[e] = __float_as_uint(tc::ex2(__uint_as_float(v[e])));
                    v[e + 1] = __float_as_uint(tc::ex2(__uint_as_float(v[e + 1])));
                }
                if (!(ok = warp_poll_bar(&sh.dp_full[b], (g >> 1) & 1, abort_flag, err, (12 << 16)))) break;
                tc::fence_after_sync();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t d[32], pk[16];
                    tc::tmem_ld32(tP + q * 32, d);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint32_t* y = &v[q * 32 + e];
                        const uint64_t s = mul2(sub2(d[e], d[e + 1], nd2), (uint64_t)y[0] | ((uint64_t)y[1] << 32));
                        pk[e / 2] = bf16_pair(lo(s), hi(s));
                    }
                    tc::tmem_st16(tP + q * 16, pk);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.ds_full[b]));
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------- epilogue
        const uint32_t tA = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 3 * BN;
        uint32_t n = 0, m = 0;
        // lse and delta of the warp's 32 rows of item number m, and its keys
        auto prepare = [&](const QItem& x) {
            const int s = m & 1, r0 = (warp & 3) * 32, row0 = x.qt * BM + r0;
            const size_t first = ((size_t)x.b * a.Hq + x.h) * a.Nq + row0;
            const float l = row0 + lane < a.Nq ? __ldg(a.lse + first + lane) : 0.f;
            const float d = row0 + lane < a.Nq ? __ldg(a.delta + first + lane) : 0.f;
            if (m >= 2 && !warp_poll_bar(&sh.row_free[s], ((m >> 1) - 1) & 1, abort_flag, err, (15 << 16)))
                return false;
            sh.neg_lse2[s][r0 + lane] = -l * kLog2e;
            sh.neg_delta[s][r0 + lane] = -d;
            if (lane == 0) sh.keys[s] = x.keys;   // the same from all four warps
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.row_full[s]));
            ++m;
            return true;
        };
        bool more = w.start(a);
        if (more && !prepare(w)) more = false;
        while (more) {
            QItem x = w;
            const bool more_x = x.next(a);
            if (more_x && !prepare(x)) break;
            const int row = w.qt * BM + (warp & 3) * 32 + lane;
            if (w.T == 0) {   // no key
                zero_rows32<D>(a.dQ, w.b, w.h, row - lane, a.Nq, lane);
            } else {
                if (!warp_poll_bar(&sh.acc_full, n & 1, abort_flag, err, (13 << 16))) break;
                tc::fence_after_sync();
                ++n;
                uint32_t pk[D / 2];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32(tA + c * 32, o);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[c * 16 + e] = bf16_pair(__uint_as_float(o[2 * e]) * a.scale,
                                                   __uint_as_float(o[2 * e + 1]) * a.scale);
                }
                tc::fence_before_sync();   // the accumulator has been read
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.acc_free));
                uint4* dst = reinterpret_cast<uint4*>(row_ptr<bf16>(a.dQ, w.b, w.h, row));
                if (row < a.Nq)
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        dst[c] = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            }
            w = x;
            more = more_x;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 9 && !sh.keep_tmem) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
int launch_dkv(const CrossArgs& a, float* part, int* err, int* lost, cudaStream_t st) {
    const void* fn = (const void*)cross_dkv_sm100_kernel<D>;
    KvMaps m;
    if (!make_tile_map(&m.q, a.Q, a.B, a.Hq, a.Nq, D, BM) || !make_tile_map(&m.g, a.dO, a.B, a.Hq, a.Nq, D, BM) ||
        !make_tile_map(&m.k, a.K, a.B, a.Hkv, a.Nk, D, BM) || !make_tile_map(&m.v, a.V, a.B, a.Hkv, a.Nk, D, BM))
        return SVGEAR_ERR_CUDA;
    static std::atomic<unsigned long long> smem_set{0};
    if (int s = set_aligned_smem(fn, kv_smem<D>(), smem_set)) return s;
    cross_dkv_sm100_kernel<D><<<kSms, kKvThreads, kv_smem<D>(), st>>>(m, a, part, err, lost);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

template <int D>
int launch_dq(const CrossArgs& a, int* err, int* lost, cudaStream_t st) {
    const void* fn = (const void*)cross_dq_sm100_kernel<D>;
    QMaps m;
    if (!make_tile_map(&m.q, a.Q, a.B, a.Hq, a.Nq, D, BM) || !make_tile_map(&m.g, a.dO, a.B, a.Hq, a.Nq, D, BM) ||
        !make_row_maps(&m.k, a.K, a.B, a.Hkv, a.Nk, D, a.k_len != nullptr) ||
        !make_row_maps(&m.v, a.V, a.B, a.Hkv, a.Nk, D, a.k_len != nullptr))
        return SVGEAR_ERR_CUDA;
    static std::atomic<unsigned long long> smem_set{0};
    if (int s = set_aligned_smem(fn, q_smem<D>(), smem_set)) return s;
    const long long items = (long long)a.B * a.Hq * ceil_div(a.Nq, BM);
    cross_dq_sm100_kernel<D><<<(int)(items < kSms ? items : kSms), kQThreads, q_smem<D>(), st>>>(m, a, err, lost);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

}  // namespace
}  // namespace crosstc

int launch_cross_backward_sm100(const CrossArgs& a, float* part, int* err, cudaStream_t st) {
    if (tmem_lost_latched()) return SVGEAR_ERR_TMEM_LOST;
    int* lost = nullptr;
    int s = tmem_lost_word(&lost);
    if (s) return s;
    s = a.D == 128 ? crosstc::launch_dq<128>(a, err, lost, st) : crosstc::launch_dq<64>(a, err, lost, st);
    if (s) return s;
    s = a.D == 128 ? crosstc::launch_dkv<128>(a, part, err, lost, st) : crosstc::launch_dkv<64>(a, part, err, lost, st);
    if (s) return s;
    return launch_cross_dkv_join(a, SVGEAR_BF16, crosstc::BM, kSms, part, st);
}

}  // namespace svgear
