// cross_sm100.cu -- dense cross attention forward for bf16 tokens on tcgen05 /
// TMEM (sm_100a).
//
// o_i = sum_j e^{s_ij - m} v_j / l in one pass over the keys with the running
// maximum m and sum l.  The weights enter the product with V rounded to bf16
// (an error of the size of the output's own rounding); l and all statistics
// stay fp32.
//
// One persistent CTA per SM; an item is 128 query rows of one head (and one
// split of its keys).  16 warps:
//   0-3, 4-7  softmax warpgroups, one row per thread (TMEM lane = row):
//             warpgroup h takes keys [64h, 64h + 64) of every 128-key tile
//             with its own running maximum, sum and accumulator O_h;
//   8, 11     TMA producers of Q and K tiles and of V tiles (a ring each);
//   9, 10     issue S = Q K^T and O_h += P_h V;
//   12-15     epilogue: merges the two accumulators like partial attentions and
//             writes the rows, while the softmax is in the next item; they leave
//             through the item's Q slot, which no product reads any more.
// TMEM: S | P[0] | P[1] | O_0 | O_1 (128 + 64 + 64 + d + d columns).  Over the
// CTA's tiles g = 0, 1, ... of all its items, S(g + 1) is issued as soon as the
// softmax has S(g) in registers and P(g) goes to a buffer of its own, so that
// neither product is on the path from one tile's softmax to the next one's.
//
// Two accumulators of d columns, one per warpgroup, need no exchange between the
// warpgroups within an item; 256 query rows per item sharing each key tile (half the
// K and V copies) leave no TMEM for P beside S and took 875 us where this took 797
// (40 heads, 75,600 x 512 keys, d = 128, both in runs of some 20 ms).
//
// Bound: a tile costs some 2,100 cycles against 1,024 of MMA work (0.38-0.50 of the
// tensor pipe): the two warpgroups' instructions for 128 x 128 weights and their copies
// between TMEM and registers (about 350 cycles each beside running MMAs).  A quarter of
// the exponentials as polynomials on the FMA pipe made it slower (836 us): the
// length of each warp's chain counts, not the exponential unit.  820 us in the first 20 ms
// of work (970 TFLOP/s); longer work reaches the power limit, the clock falls towards 1 GHz
// and a call takes 965-975 us (820 TFLOP/s, 0.60 of a library product's sustained rate).
// Few rows over many keys (77 x 118,800, 24 heads) read K and V at 6.2 TB/s at first
// (235 us) and at 5.1-5.6 sustained (263-284 us), where a copy has 6.55.
//
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

constexpr int kThreads = 16 * 32;
constexpr int kLoadWarp = 8, kQkWarp = 9, kPvWarp = 10, kVWarp = 11, kEpilogueWarp = 12;
constexpr int HN = BN / 2;                  // keys of a warpgroup per tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kP = BN, kO = 2 * BN;    // TMEM columns of P[0] and O_0
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kMinSplitTiles = 4;           // fewest key tiles of a split: with 2, one query
                                            // over 512 keys took 14.5 us (two launches)
                                            // against 14.2 and 9 us more on the host; with
                                            // 8, over 1,024 keys 18.4 against 16.5

// A copy takes some 2,000 cycles to arrive and S(g + 2) follows S(g + 1) by one
// tile's softmax (1,500): three K slots.  V(g + 2) has two tiles' time.
template <int D>
constexpr int k_slots() { return D == 128 ? 3 : 4; }
template <int D>
constexpr int v_slots() { return D == 128 ? 2 : 4; }
template <int D>
constexpr uint32_t smem_bytes() { return (2 + k_slots<D>() + v_slots<D>()) * (D / 64) * 16384; }

struct Maps {
    RowMaps k, v;
    TileMap q, o;   // o: boxes of 32 rows
};

struct Shared {
    uint64_t q_full[2], q_free[2];    // Q slot s loaded / its item's output has left it
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full, s_read;
    uint64_t p_full[2], p_free[2];    // P[b] written / read by both PV
    uint64_t o_full, o_free;          // O_0 and O_1 final / read out
    uint64_t ml_full;                 // both warpgroups' (m, l) of the item
    uint64_t drain[2];
    float2 ml[2][BM];                 // [h][row]
    uint32_t tmem_base;
    int abort_flag;
    int keep_tmem;
};

struct Plan {
    int qtiles;       // 128-row tiles per head
    int splits;       // key splits
    int tiles;        // key tiles per split
    int items;
};

// The items of one CTA in turn: item = ((b * Hq + h) * splits + split) * qtiles +
// tile, advanced by the grid digit by digit (divisions once per CTA: they would
// sit on every role's path between items).
struct Work {
    int item, qt, split, h, b;        // digits
    int dq, ds, dh, db;               // the grid's digits
    int hk, keys;
    int t0, T;                        // first key tile and number of tiles
    __device__ __forceinline__ void derive(const CrossArgs& a, const Plan& p) {
        keys = cross_keys(a, b);
        t0 = split * p.tiles;
        T = max(0, min((keys + BN - 1) / BN - t0, p.tiles));
        hk = a.G == 1 ? h : h / a.G;
    }
    __device__ __forceinline__ bool start(const CrossArgs& a, const Plan& p) {
        item = blockIdx.x;
        int x = item;
        qt = x % p.qtiles; x /= p.qtiles;
        split = x % p.splits; x /= p.splits;
        h = x % a.Hq;
        b = x / a.Hq;
        x = gridDim.x;
        dq = x % p.qtiles; x /= p.qtiles;
        ds = x % p.splits; x /= p.splits;
        dh = x % a.Hq;
        db = x / a.Hq;
        if (item < p.items) derive(a, p);
        return item < p.items;
    }
    __device__ __forceinline__ bool next(const CrossArgs& a, const Plan& p) {
        item += gridDim.x;
        qt += dq; split += ds; h += dh; b += db;
        if (qt >= p.qtiles) { qt -= p.qtiles; ++split; }
        if (split >= p.splits) { split -= p.splits; ++h; }
        if (h >= a.Hq) { h -= a.Hq; ++b; }
        if (item < p.items) derive(a, p);
        return item < p.items;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_fwd_sm100_kernel(const __grid_constant__ Maps maps, CrossArgs a, Plan plan, float scale_log2,
                       float* __restrict__ o_part, float* __restrict__ lse_part,
                       int* __restrict__ err, int* __restrict__ lost) {
    constexpr uint32_t kTile = (D / 64) * 16384;
    constexpr int NK = k_slots<D>(), NV = v_slots<D>();
    if (tc::refuse_start(lost, err)) return;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t base = tc::smem_u32(smem_raw);   // 1024-byte aligned: see launch()
    const uint32_t sQ = base, sK = sQ + 2 * kTile, sV = sK + NK * kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.q_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.q_free[i]), 4);
            tc::mbar_init(tc::smem_u32(&sh.p_full[i]), 8);
            tc::mbar_init(tc::smem_u32(&sh.p_free[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.drain[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.k_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.k_empty[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.v_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.v_empty[i]), 1);
        }
        tc::mbar_init(tc::smem_u32(&sh.s_full), 1);
        tc::mbar_init(tc::smem_u32(&sh.s_read), 8);
        tc::mbar_init(tc::smem_u32(&sh.o_full), 1);
        tc::mbar_init(tc::smem_u32(&sh.o_free), 4);
        tc::mbar_init(tc::smem_u32(&sh.ml_full), 8);
        sh.abort_flag = 0;
        sh.keep_tmem = 0;
        tc::mbar_init_fence();
    }
    if (warp == kQkWarp) {
        tc::tmem_alloc(tc::smem_u32(&sh.tmem_base), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    volatile int* abort_flag = &sh.abort_flag;
    Work w;

    if ((warp == kLoadWarp || warp == kVWarp) && lane == 0) {
        // ----------------------------------------------------------- producers
        // (of Q and K, and of V: one for both would hold up K behind a V slot)
        const bool is_k = warp == kLoadWarp;
        const int NS = is_k ? NK : NV;
        uint64_t* full = is_k ? sh.k_full : sh.v_full;
        uint64_t* empty = is_k ? sh.k_empty : sh.v_empty;
        const RowMaps& map = is_k ? maps.k : maps.v;
        const uint32_t slots = is_k ? sK : sV;
        Ring ring;
        uint32_t fills = 0, n = 0;
        bool ok = true;
        for (bool more = w.start(a, plan); ok && more; more = w.next(a, plan)) {
            if (w.T == 0) continue;
            if (is_k) {
                const int s = n & 1;
                if (n >= 2 && !(ok = poll_bar(&sh.q_free[s], ((n >> 1) - 1) & 1, abort_flag, err, (1 << 16)))) break;
                load_tile<D>(maps.q, sQ + s * kTile, w.b, w.h, w.qt * BM, tc::smem_u32(&sh.q_full[s]));
                ++n;
                // a coming item's rows on their way from HBM to L2
                Work x = w;
                if (x.next(a, plan) && x.next(a, plan) && x.T > 0) prefetch_tile<D>(maps.q, x.b, x.h, x.qt * BM);
            }
            for (int j = 0; j < w.T; ++j) {
                if (fills >= (uint32_t)NS && !(ok = poll_bar(&empty[ring.slot], ring.phase ^ 1, abort_flag, err, (2 << 16))))
                    break;
                load_key_tile<D>(map, slots + ring.slot * kTile, w.b, w.hk, (w.t0 + j) * BN, w.keys, a.Nk,
                                 tc::smem_u32(&full[ring.slot]));
                ++fills;
                ring.next(NS);
            }
        }
        // gave up: let the copies in flight land before the CTA ends
        if (!ok) {
            for (uint32_t q = n > 2 ? n - 2 : 0; q < n; ++q) tc::drain_bar(&sh.q_full[q & 1], (q >> 1) & 1);
            for (uint32_t f = fills > (uint32_t)NS ? fills - NS : 0; f < fills; ++f)
                tc::drain_bar(&full[f % NS], (f / NS) & 1);
        }
    } else if ((warp == kQkWarp || warp == kPvWarp) && lane == 0) {
        // ----------------------------------------------------------- MMA issue
        const bool qk = warp == kQkWarp;
        Ring ring;
        uint32_t n = 0, g = 0;
        bool ok = true;
        for (bool more = w.start(a, plan); ok && more; more = w.next(a, plan)) {
            if (w.T == 0) continue;
            if (qk) {
                ok = poll_bar(&sh.q_full[n & 1], (n >> 1) & 1, abort_flag, err, (4 << 16));
                for (int j = 0; ok && j < w.T; ++j, ++g) {
                    // S(g) overwrites S(g - 1), which must be in registers
                    if (!(ok = poll_bar(&sh.k_full[ring.slot], ring.phase, abort_flag, err, (5 << 16)) &&
                               (g == 0 || poll_bar(&sh.s_read, (g - 1) & 1, abort_flag, err, (6 << 16)))))
                        break;
                    tc::fence_after_sync();
                    mma_dot<D>(tmem, sQ + (n & 1) * kTile, sK + ring.slot * kTile);
                    tc::commit(tc::smem_u32(&sh.s_full));
                    tc::commit(tc::smem_u32(&sh.k_empty[ring.slot]));
                    ring.next(NK);
                }
            } else {
                // the first PV overwrites O: the last item's must be read out
                ok = n == 0 || poll_bar(&sh.o_free, (n - 1) & 1, abort_flag, err, (4 << 16) + 1);
                for (int j = 0; ok && j < w.T; ++j, ++g) {
                    const uint32_t b = g & 1;
                    if (!(ok = poll_bar(&sh.v_full[ring.slot], ring.phase, abort_flag, err, (7 << 16)) &&
                               poll_bar(&sh.p_full[b], (g >> 1) & 1, abort_flag, err, (8 << 16))))
                        break;
                    tc::fence_after_sync();
                    const uint32_t tile = sV + ring.slot * kTile, tP = tmem + kP + b * HN, acc = j > 0 ? 1u : 0u;
                    mma_rows_k64<D>(tmem + kO, tP, tile, acc);
                    mma_rows_k64<D>(tmem + kO + D, tP + 32, tile + HN * 128, acc);
                    tc::commit(tc::smem_u32(&sh.p_free[b]));
                    tc::commit(tc::smem_u32(&sh.v_empty[ring.slot]));
                    ring.next(NV);
                }
                if (ok) tc::commit(tc::smem_u32(&sh.o_full));
            }
            ++n;
        }
        drain_mma(&sh.drain[qk ? 0 : 1], &sh.keep_tmem, err, lost, (9 << 16) + (qk ? 0 : 1));
    } else if (warp < 8) {
        // -------------------------------------------------------------- softmax
        const int h = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_base + h * HN, tO = lane_base + kO + h * D;
        uint32_t n = 0, g = 0;
        bool ok = true;
        for (bool more = w.start(a, plan); ok && more; more = w.next(a, plan)) {
            if (w.T == 0) continue;
            float m_use = -INFINITY, l = 0.f;
            for (int j = 0; j < w.T; ++j, ++g) {
                const uint32_t b = g & 1, tP = lane_base + kP + b * HN + h * 32;
                if (!(ok = warp_poll_bar(&sh.s_full, g & 1, abort_flag, err, (10 << 16)))) break;
                tc::fence_after_sync();
                const int valid = w.keys - (w.t0 + j) * BN - h * HN;   // of this half
                if (valid < HN) mask_columns<HN>(tS, valid);
                uint32_t v[HN];
                tc::tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                tc::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                tc::tmem_ld_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.s_read));
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int e = 0; e < HN; e += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(v[e + 4]), __uint_as_float(v[e + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(v[e + 6]), __uint_as_float(v[e + 7]));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scale_log2;   // scale > 0
                const float m_new = fmaxf(m_use, mx);
                // O is rescaled only when a row's maximum grows by more than
                // 2^8 (the weights then stay below 2^8, far from the ends of
                // bf16 and fp32); TMEM accesses are warp-collective, so the
                // warp rescales together.
                const bool need = j > 0 && m_new > m_use + kRescaleThreshold;
                const bool any = __any_sync(0xffffffffu, need);
                float alpha = 1.f;
                if (j == 0) {
                    m_use = m_new;
                } else if (need) {
                    alpha = tc::ex2(m_use - m_new);
                    l *= alpha;
                    m_use = m_new;
                }
                const float neg_m = m_use == -INFINITY ? 0.f : -m_use;   // no finite score so far
                uint64_t s01 = 0ull;
                const uint64_t xs2 = pack2(scale_log2, scale_log2), nm2 = pack2(neg_m, neg_m);
#pragma unroll
                for (int q = 0; q < HN / 32; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        uint32_t a0, a1;
                        fma2(v[q * 32 + e], v[q * 32 + e + 1], xs2, nm2, a0, a1);
                        const float p0 = tc::ex2(__uint_as_float(a0));
                        const float p1 = tc::ex2(__uint_as_float(a1));
                        add2(s01, p0, p1);
                        pk[e >> 1] = bf16_pair(p0, p1);
                    }
                    // P(g - 2) must have been read out of the buffer
                    if (q == 0 && g >= 2) {
                        ok = warp_poll_bar(&sh.p_free[b], ((g >> 1) - 1) & 1, abort_flag, err, (11 << 16));
                        tc::fence_after_sync();   // its MMA's reads before the stores below
                    }
                    tc::tmem_st16(tP + q * 16, pk);
                }
                if (!ok) break;
                l += __uint_as_float((uint32_t)s01) + __uint_as_float((uint32_t)(s01 >> 32));
                if (any) {
                    // PV(g - 1), the last addition to O_h, must be complete
                    if (!(ok = warp_poll_bar(&sh.p_free[b ^ 1], ((g - 1) >> 1) & 1, abort_flag, err, (12 << 16)))) break;
                    tc::fence_after_sync();
                    uint32_t o[16];
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        tc::tmem_ld16(tO + c * 16, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::tmem_st16(tO + c * 16, o);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.p_full[b]));
            }
            if (!ok) break;
            // (the epilogue must have read the last item's pair)
            if (n > 0 && !(ok = warp_poll_bar(&sh.o_free, (n - 1) & 1, abort_flag, err, (14 << 16)))) break;
            sh.ml[h][r] = make_float2(m_use, l);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.ml_full));
            ++n;
        }
    } else if (warp >= kEpilogueWarp) {
        // ------------------------------------------------------------- epilogue
        // o = (a_0 O_0 + a_1 O_1) / (a_0 l_0 + a_1 l_1), a_h = 2^(m_h - m)
        const int r = tid & 127;
        const uint32_t tO = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kO;
        const bool parts = plan.splits > 1;
        uint32_t n = 0;
        for (bool more = w.start(a, plan); more; more = w.next(a, plan)) {
            const int row = w.qt * BM + r;
            const bool write = row < a.Nq;
            const size_t rr = ((size_t)w.b * a.Hq + w.h) * a.Nq + row;
            const size_t part = (size_t)w.split * a.B * a.Hq * a.Nq + rr;
            if (w.T == 0) {   // no key
                if (!parts) zero_rows32<D>(a.O, w.b, w.h, row - lane, a.Nq, lane);
                if (write) (parts ? lse_part[part] : a.lse[rr]) = -INFINITY;
                continue;
            }
            if (!warp_poll_bar(&sh.ml_full, n & 1, abort_flag, err, (13 << 16))) break;
            const float2 x0 = sh.ml[0][r], x1 = sh.ml[1][r];
            const float m = fmaxf(x0.x, x1.x);
            const float mu = m == -INFINITY ? 0.f : m;   // no finite score
            float c0 = tc::ex2(x0.x - mu), c1 = tc::ex2(x1.x - mu);
            const float sum = fmaf(c0, x0.y, c1 * x1.y);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            c0 *= inv;
            c1 *= inv;
            if (write) {
                const float lse = sum == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(sum));
                (parts ? lse_part[part] : a.lse[rr]) = lse;
            }
            if (!warp_poll_bar(&sh.o_full, n & 1, abort_flag, err, (15 << 16))) break;
            tc::fence_after_sync();
            // 32 columns of both accumulators at a time (beside running MMAs a
            // TMEM load takes some 350 cycles whatever its size) in a rolled
            // loop (this code runs once per item, fetched anew each time)
            const uint32_t stage = sQ + (n & 1) * kTile;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o0[32], o1[32];
                tc::tmem_ld32(tO + c * 32, o0);
                tc::tmem_ld32(tO + D + c * 32, o1);
                tc::tmem_ld_wait();
                if (c == D / 32 - 1) {   // the accumulators and the pair have been read
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.o_free));
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    uint32_t y0, y1;
                    fma2(o1[e], o1[e + 1], pack2(c1, c1), 0ull, y0, y1);
                    fma2(o0[e], o0[e + 1], pack2(c0, c0), (uint64_t)y0 | ((uint64_t)y1 << 32), o0[e], o0[e + 1]);
                }
                if (parts) {
                    if (write) {
                        uint4* o4 = reinterpret_cast<uint4*>(o_part + part * D + c * 32);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            o4[q] = make_uint4(o0[4 * q], o0[4 * q + 1], o0[4 * q + 2], o0[4 * q + 3]);
                    }
                } else {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[e] = bf16_pair(__uint_as_float(o0[2 * e]), __uint_as_float(o0[2 * e + 1]));
                    stage_row32(stage, r, c * 32, pk);
                }
            }
            if (!parts) store_staged<D>(maps.o, stage, r - lane, w.b, w.h, row - lane, row - lane < a.Nq, lane);
            if (lane == 0) {   // (nothing staged: at once)
                tc::bulk_wait_read();
                tc::mbar_arrive(tc::smem_u32(&sh.q_free[n & 1]));
            }
            __syncwarp();
            ++n;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kQkWarp && !sh.keep_tmem) tc::tmem_dealloc(tmem, kTmemCols);
}

Plan make_plan(int B, int Hq, int Nq, int Nk) {
    Plan p;
    p.qtiles = ceil_div(Nq, BM);
    const int key_tiles = ceil_div(Nk, BN);
    const CrossSplit s = cross_split((long long)B * Hq * p.qtiles, key_tiles, kSms, kMinSplitTiles);
    p.splits = s.splits;
    p.tiles = s.tiles;
    p.items = B * Hq * p.qtiles * p.splits;
    return p;
}

template <int D>
int launch(const CrossArgs& a, const Plan& plan, float* o_part, float* lse_part, int* err, int* lost,
           cudaStream_t st) {
    const void* fn = (const void*)cross_fwd_sm100_kernel<D>;
    Maps maps;
    const bool pieces = a.k_len != nullptr;
    if (!make_tile_map(&maps.q, a.Q, a.B, a.Hq, a.Nq, D) ||
        !make_tile_map(&maps.o, a.O, a.B, a.Hq, a.Nq, D, 32) ||
        !make_row_maps(&maps.k, a.K, a.B, a.Hkv, a.Nk, D, pieces) ||
        !make_row_maps(&maps.v, a.V, a.B, a.Hkv, a.Nk, D, pieces))
        return SVGEAR_ERR_CUDA;
    static std::atomic<unsigned long long> smem_set{0};
    if (int s = set_aligned_smem(fn, smem_bytes<D>(), smem_set)) return s;
    cross_fwd_sm100_kernel<D><<<plan.items < kSms ? plan.items : kSms, kThreads, smem_bytes<D>(), st>>>(
        maps, a, plan, a.scale * 1.4426950408889634f, o_part, lse_part, err, lost);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

}  // namespace
}  // namespace crosstc

int cross_sm100_parts(int B, int Hq, int Nq, int Nk) {
    return crosstc::make_plan(B, Hq, Nq, Nk).splits;
}

int launch_cross_sm100(const CrossArgs& a, float* o_part, float* lse_part, int* err, cudaStream_t st) {
    if (tmem_lost_latched()) return SVGEAR_ERR_TMEM_LOST;
    int* lost = nullptr;
    if (int s = tmem_lost_word(&lost)) return s;
    const crosstc::Plan p = crosstc::make_plan(a.B, a.Hq, a.Nq, a.Nk);
    return a.D == 128 ? crosstc::launch<128>(a, p, o_part, lse_part, err, lost, st)
                      : crosstc::launch<64>(a, p, o_part, lse_part, err, lost, st);
}

}  // namespace svgear
