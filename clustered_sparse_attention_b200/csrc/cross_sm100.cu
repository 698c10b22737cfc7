// cross_sm100.cu -- dense cross attention forward for bf16 tokens on tcgen05 /
// TMEM (sm_100a).
//
// o_i = sum_j e^{s_ij - m} v_j / l in one pass over the keys with the running
// maximum m and sum l; the weights enter the product with V as bf16 (their
// rounding, 2^-9 of each on average, is of the size of the output's own), l
// and all statistics stay fp32.
//
// One persistent CTA per SM.  An item is 256 query rows of one head: two
// 128-row tiles ("halves") that share every K and V tile, so each shared
// memory byte feeds two MMAs.  12 warps:
//   0-3, 4-7  softmax of half 0 / 1, one row per thread (TMEM lane = row);
//   8         TMA producer: Q tiles, and K and V tiles through one slot ring;
//   9, 10     one thread each issues the MMAs of half 0 / 1, so a half waits
//             only for its own softmax: while one half exponentiates, the
//             other's PV and next QK use the tensor cores;
//   11        idle.
// TMEM: S0 | S1 | O0 | O1; P (bf16) overwrites the first 64 columns of its S.
// The Q tiles of the next item are copied as soon as the last QK has read
// them, and its K tiles follow through the ring, so items overlap except for
// a half's own epilogue.
//
// With few rows (Nq <= 128) over many keys one half would leave the other
// idle: both then take the same rows ("solo"), half h the tiles h, h + 2, ...
// of the item, and their partial results are joined like those of the key
// splits (cross_join_kernel).
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

constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;             // and 10 for half 1
constexpr int kThreads = 12 * 32;
// Register split as launched (168 x 384): 232 for the softmax warpgroups, 40
// for the others.
constexpr uint32_t kSoftmaxRegs = 232;
constexpr uint32_t kIssueRegs = 40;
constexpr int kMinLaunchRegs = 168;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kIssueRegs <= kMinLaunchRegs * kThreads,
              "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
constexpr int kTurnChunk = 2;               // 32-column chunk after which the turn passes
constexpr float kRescaleThreshold = 8.0f;   // log2 units

template <int D>
constexpr int ring_slots() { return D == 128 ? 4 : 8; }

struct Maps {
    RowMaps k, v;
    TileMap q, o;   // o: boxes of 32 rows
};

struct Shared {
    uint64_t q_full[2], q_empty[2];   // the half's Q tile
    uint64_t full[8], empty[8];       // K/V slots
    uint64_t s_full[2], p_full[2];    // S written / P written
    uint64_t o_full[2], o_free[2];    // O final / read out
    uint64_t turn[2];                 // half h may exponentiate its next paired tile
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort_flag;
    int keep_tmem;
};

struct Plan {
    int qpairs;       // 256-row pairs per head
    int splits;       // key splits
    int tiles;        // key tiles per split
    int solo;         // both halves on the same 128 rows
    int items;
};

// The items of one CTA in turn: item = ((b * Hq + h) * splits + split) * qpairs +
// pair, advanced by the grid digit by digit (divisions once per CTA: they
// would sit on every role's path between items).
struct Work {
    int item, qp, split, h, b;        // digits
    int dq, ds, dh, db;               // the grid's digits
    int hk, q0, keys;
    int t0, T;                        // first key tile and number of tiles
    __device__ __forceinline__ void derive(const CrossArgs& a, const Plan& p) {
        q0 = qp * 2 * BM;
        keys = cross_keys(a, b);
        t0 = split * p.tiles;
        T = max(0, min((keys + BN - 1) / BN - t0, p.tiles));
        hk = a.G == 1 ? h : h / a.G;
    }
    __device__ __forceinline__ void start(const CrossArgs& a, const Plan& p) {
        item = blockIdx.x;
        int x = item;
        qp = x % p.qpairs; x /= p.qpairs;
        split = x % p.splits; x /= p.splits;
        h = x % a.Hq;
        b = x / a.Hq;
        x = gridDim.x;
        dq = x % p.qpairs; x /= p.qpairs;
        ds = x % p.splits; x /= p.splits;
        dh = x % a.Hq;
        db = x / a.Hq;
        if (item < p.items) derive(a, p);
    }
    __device__ __forceinline__ void next(const CrossArgs& a, const Plan& p) {
        item += gridDim.x;
        qp += dq; split += ds; h += dh; b += db;
        if (qp >= p.qpairs) { qp -= p.qpairs; ++split; }
        if (split >= p.splits) { split -= p.splits; ++h; }
        if (h >= a.Hq) { h -= a.Hq; ++b; }
        if (item < p.items) derive(a, p);
    }
};

// Tiles that half h takes of an item (0: the half sits it out).
__device__ __forceinline__ int half_tiles(const CrossArgs& a, const Plan& p, const Work& w, int h) {
    if (p.solo) return (w.T + 1 - h) / 2;
    return w.q0 + h * BM < a.Nq ? w.T : 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_fwd_sm100_kernel(const __grid_constant__ Maps maps, CrossArgs a, Plan plan, float scale_log2,
                       float* __restrict__ o_part, float* __restrict__ lse_part,
                       int* __restrict__ err, int* __restrict__ lost) {
    constexpr uint32_t kTile = (D / 64) * 16384;
    constexpr int NS = ring_slots<D>();
    if (tc::refuse_start(lost, err)) return;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sQ = base, sRing = base + 2 * kTile, sStage = sRing + NS * kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int h = 0; h < 2; ++h) {
            tc::mbar_init(tc::smem_u32(&sh.q_full[h]), 1);
            tc::mbar_init(tc::smem_u32(&sh.q_empty[h]), 1);
            tc::mbar_init(tc::smem_u32(&sh.s_full[h]), 1);
            tc::mbar_init(tc::smem_u32(&sh.p_full[h]), 4);
            tc::mbar_init(tc::smem_u32(&sh.o_full[h]), 1);
            tc::mbar_init(tc::smem_u32(&sh.o_free[h]), 4);
            tc::mbar_init(tc::smem_u32(&sh.turn[h]), 4);
            tc::mbar_init(tc::smem_u32(&sh.drain[h]), 1);
        }
        for (int s = 0; s < NS; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.empty[s]), 2);
        }
        sh.abort_flag = 0;
        sh.keep_tmem = 0;
        tc::mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tc::smem_u32(&sh.tmem_base), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    volatile int* abort_flag = &sh.abort_flag;

    if (warp >= 8) {
        tc::regs_dec<kIssueRegs>();
        if (warp == kProducerWarp && lane == 0) {
            // -------------------------------------------------------- producer
            Ring ring;
            uint32_t fills = 0;          // slots filled so far
            uint32_t used[2] = {0, 0};   // Q tiles loaded per half
            bool ok = true;
            Work w;
            for (w.start(a, plan); ok && w.item < plan.items; w.next(a, plan)) {
                for (int h = 0; ok && h < 2; ++h) {
                    if (half_tiles(a, plan, w, h) == 0) continue;
                    if (used[h] > 0 &&
                        !poll_bar(&sh.q_empty[h], (used[h] - 1) & 1, abort_flag, err, (1 << 16) + h)) {
                        ok = false;
                        break;
                    }
                    load_tile<D>(maps.q, sQ + h * kTile, w.b, w.h, w.q0 + (plan.solo ? 0 : h * BM),
                                 tc::smem_u32(&sh.q_full[h]));
                    ++used[h];
                }
                // the next item's query rows on their way from HBM to L2 meanwhile
                if (ok && w.item + (int)gridDim.x < plan.items) {
                    Work x = w;
                    x.next(a, plan);
                    for (int h = 0; h < 2; ++h)
                        if (half_tiles(a, plan, x, h) > 0 && !(plan.solo && h))
                            prefetch_tile<D>(maps.q, x.b, x.h, x.q0 + h * BM);
                }
                for (int j = 0; ok && j < 2 * w.T; ++j) {
                    if (fills >= NS &&
                        !poll_bar(&sh.empty[ring.slot], ring.phase ^ 1, abort_flag, err, (2 << 16) + j)) {
                        ok = false;
                        break;
                    }
                    load_key_tile<D>((j & 1) ? maps.v : maps.k, sRing + ring.slot * kTile, w.b, w.hk,
                                     (w.t0 + (j >> 1)) * BN, w.keys, a.Nk, tc::smem_u32(&sh.full[ring.slot]));
                    ++fills;
                    ring.next(NS);
                }
            }
            // gave up: let the copies in flight land before the CTA ends
            if (!ok) {
                for (int h = 0; h < 2; ++h)
                    if (used[h] > 0) tc::drain_bar(&sh.q_full[h], (used[h] - 1) & 1);
                for (uint32_t f = fills > NS ? fills - NS : 0; f < fills; ++f)
                    tc::drain_bar(&sh.full[f % NS], (f / NS) & 1);
            }
        } else if ((warp == kMmaWarp || warp == kMmaWarp + 1) && lane == 0) {
            // ------------------------------------------------------- MMA issue
            const int h = warp - kMmaWarp;
            const uint32_t tS = tmem + h * BN, tO = tmem + 2 * BN + h * D;
            Ring ring;
            uint32_t n = 0, tiles = 0;   // items and tiles of this half so far
            bool ok = true;
            auto skip_slot = [&]() {
                ok = poll_bar(&sh.full[ring.slot], ring.phase, abort_flag, err, (3 << 16) + h);
                if (ok) tc::mbar_arrive(tc::smem_u32(&sh.empty[ring.slot]));
                ring.next(NS);
            };
            Work w;
            for (w.start(a, plan); ok && w.item < plan.items; w.next(a, plan)) {
                const int mine = half_tiles(a, plan, w, h);
                int j = 0;   // tile of the ring position
                // passes the tiles of the other half
                auto skip_to = [&](int t) {
                    for (; ok && j < t; ++j) {
                        skip_slot();
                        if (ok) skip_slot();
                    }
                };
                if (mine == 0) {
                    skip_to(w.T);
                    continue;
                }
                const int step = plan.solo ? 2 : 1;
                const bool solo = plan.solo != 0;
                skip_to(solo ? h : 0);
                ok = ok && poll_bar(&sh.q_full[h], n & 1, abort_flag, err, (4 << 16) + h) &&
                     poll_bar(&sh.full[ring.slot], ring.phase, abort_flag, err, (5 << 16));
                if (!ok) break;
                tc::fence_after_sync();
                mma_dot<D>(tS, sQ + h * kTile, sRing + ring.slot * kTile);
                tc::commit(tc::smem_u32(&sh.s_full[h]));
                tc::commit(tc::smem_u32(&sh.empty[ring.slot]));
                if (mine == 1) tc::commit(tc::smem_u32(&sh.q_empty[h]));
                ring.next(NS);
                for (int i = 0; i < mine; ++i) {
                    // everything the next two products need but P is waited
                    // for ahead of it, so that PV and the next QK follow P
                    // without a pause.  (The ring holds what this waits for:
                    // V, the other half's K and V when solo, the next K.)
                    const int vslot = ring.slot;
                    if (!(ok = poll_bar(&sh.full[vslot], ring.phase, abort_flag, err, (8 << 16) + i))) break;
                    ring.next(NS);
                    ++j;
                    const bool more = i + 1 < mine;
                    if (more) {
                        skip_to(j + step - 1);
                        if (!ok || !(ok = poll_bar(&sh.full[ring.slot], ring.phase, abort_flag, err, (5 << 16) + i)))
                            break;
                    }
                    // the first PV overwrites O: the last item's must be read out
                    if (i == 0 && n > 0 &&
                        !(ok = poll_bar(&sh.o_free[h], (n - 1) & 1, abort_flag, err, (7 << 16) + h)))
                        break;
                    if (!(ok = poll_bar(&sh.p_full[h], tiles & 1, abort_flag, err, (6 << 16) + i))) break;
                    ++tiles;
                    tc::fence_after_sync();
                    mma_rows<D>(tO, tS, sRing + vslot * kTile, i > 0 ? 1u : 0u);
                    if (more) {
                        mma_dot<D>(tS, sQ + h * kTile, sRing + ring.slot * kTile);
                        tc::commit(tc::smem_u32(&sh.s_full[h]));
                        tc::commit(tc::smem_u32(&sh.empty[vslot]));
                        tc::commit(tc::smem_u32(&sh.empty[ring.slot]));
                        if (i + 2 == mine) tc::commit(tc::smem_u32(&sh.q_empty[h]));
                        ring.next(NS);
                    } else {
                        tc::commit(tc::smem_u32(&sh.o_full[h]));
                        tc::commit(tc::smem_u32(&sh.empty[vslot]));
                    }
                }
                if (!ok) break;
                skip_to(w.T);
                ++n;
            }
            // every MMA of this thread is complete once its drain flips; if
            // that wait expires TMEM stays allocated and the device's lost
            // word stops every later tensor-core kernel before it allocates
            tc::commit(tc::smem_u32(&sh.drain[h]));
            if (!tc::drain_bar(&sh.drain[h], 0)) {
                sh.keep_tmem = 1;
                tc::mark_tmem_lost(lost);
                if (atomicCAS(err, 0, SVGEAR_ERR_TIMEOUT) == 0) {
                    err[1] = (9 << 16) + h;
                    err[2] = blockIdx.x;
                }
            }
        }
        __syncwarp();
    } else {
        tc::regs_inc<kSoftmaxRegs>();
        // -------------------------------------------------------------- softmax
        const int h = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = lane_base + h * BN, tO = lane_base + 2 * BN + h * D;
        uint32_t n = 0, tiles = 0, turns = 0;
        bool ok = true;
        uint32_t v[BN];
        Work w;
        for (w.start(a, plan); ok && w.item < plan.items; w.next(a, plan)) {
            const int mine = half_tiles(a, plan, w, h);
            const int paired = min(mine, half_tiles(a, plan, w, 1 - h));
            const int row = w.q0 + (plan.solo ? 0 : h * BM) + r;
            float m_use = -INFINITY, l = 0.f;
            for (int i = 0; i < mine; ++i) {
                if (!(ok = warp_poll_bar(&sh.s_full[h], tiles & 1, abort_flag, err, (10 << 16) + i))) break;
                ++tiles;
                tc::fence_after_sync();
                const int j = w.t0 + (plan.solo ? 2 * i + h : i);
                const int valid = w.keys - j * BN;
                if (valid < BN) {
                    // the batch's last tile: -inf past the keys, rewritten in
                    // TMEM so that the main path carries no selects
#pragma unroll 1
                    for (int c4 = valid / 32; c4 < BN / 32; ++c4) {
                        uint32_t t[32];
                        tc::tmem_ld32(tS + c4 * 32, t);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c4 * 32 + e >= valid) t[e] = __float_as_uint(-INFINITY);
                        tc::tmem_st32(tS + c4 * 32, t);
                    }
                    tc::tmem_st_wait();
                }
                tc::tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                tc::tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                tc::tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&v[64]));
                tc::tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&v[96]));
                tc::tmem_ld_wait();
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int e = 0; e < BN; e += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(v[e + 4]), __uint_as_float(v[e + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(v[e + 6]), __uint_as_float(v[e + 7]));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scale_log2;   // scale > 0
                const float m_new = fmaxf(m_use, mx);
                // O is rescaled only when a row's maximum grows by more than
                // 2^8 (the weights then stay below 2^8, far from bf16's and
                // fp32's ranges); TMEM accesses are warp-collective, so the
                // warp rescales together.  s_full came with the commit after
                // the previous PV, so O is complete here.
                const bool need = i > 0 && m_new > m_use + kRescaleThreshold;
                const bool any = __any_sync(0xffffffffu, need);
                float alpha = 1.f;
                if (i == 0) {
                    m_use = m_new;
                } else if (need) {
                    alpha = tc::ex2(m_use - m_new);
                    l *= alpha;
                    m_use = m_new;
                }
                const float neg_m = m_use == -INFINITY ? 0.f : -m_use;   // every score -inf so far
                // the halves take turns on the exp unit
                if (i < paired) {
                    if ((h == 1 || turns > 0) &&
                        !(ok = warp_poll_bar(&sh.turn[h], (turns - 1 + h) & 1, abort_flag, err, (12 << 16) + i)))
                        break;
                    ++turns;
                }
                uint64_t s01 = 0ull;
                const uint64_t xs2 = pack2(scale_log2, scale_log2), nm2 = pack2(neg_m, neg_m);
#pragma unroll
                for (int q = 0; q < BN / 32; ++q) {
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
                    tc::tmem_st16(tS + q * 16, pk);
                    if (q == kTurnChunk && i < paired && lane == 0)
                        tc::mbar_arrive(tc::smem_u32(&sh.turn[1 - h]));
                }
                l += __uint_as_float((uint32_t)s01) + __uint_as_float((uint32_t)(s01 >> 32));
                if (any) {
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
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.p_full[h]));
            }
            if (!ok) break;
            if (mine > 0) {
                if (!(ok = warp_poll_bar(&sh.o_full[h], n & 1, abort_flag, err, (11 << 16)))) break;
                tc::fence_after_sync();
                ++n;
            }
            // epilogue; an item without tiles leaves zeros and lse = -inf
            const bool write = row < a.Nq;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse = l == 0.f ? -INFINITY : fmaf(m_use, 0.6931471805599453f, logf(l));
            const size_t rr = ((size_t)w.b * a.Hq + w.h) * a.Nq + row;
            const bool parts = plan.splits > 1 || plan.solo;
            const size_t part = (size_t)(plan.solo ? 2 * w.split + h : w.split) * a.B * a.Hq * a.Nq + rr;
            if (write) {
                if (parts) lse_part[part] = lse;
                else a.lse[rr] = lse;
            }
            auto free_o = [&]() {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.o_free[h]));
            };
            if (mine == 0) {
                if (write && !parts) {
                    uint4* o4 = reinterpret_cast<uint4*>(row_ptr<bf16>(a.O, w.b, w.h, row));
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c) o4[c] = make_uint4(0, 0, 0, 0);
                }
            } else if (parts) {
                uint32_t o[32];
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    tc::tmem_ld32(tO + c4 * 32, o);
                    tc::tmem_ld_wait();
                    if (write) {
                        float4* o4 = reinterpret_cast<float4*>(o_part + part * D + c4 * 32);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            o4[q] = make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                                                __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
                    }
                }
                free_o();
            } else {
                const int n0 = row - lane;
                uint32_t o[D];
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    tc::tmem_ld32(tO + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[c * 32]));
                tc::tmem_ld_wait();
                free_o();
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        pk[e] = bf16_pair(__uint_as_float(o[c * 64 + 2 * e]) * inv, __uint_as_float(o[c * 64 + 2 * e + 1]) * inv);
                    store_rows<0>(maps.o, sStage + warp * 4096, pk, c * 64, w.b, w.h, n0, n0 < a.Nq, lane);
                }
            }
        }
        if (lane == 0) tc::bulk_wait_read<0>();   // shared memory outlives its stores
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp && !sh.keep_tmem) tc::tmem_dealloc(tmem, kTmemCols);
}

Plan make_plan(int B, int Hq, int Nq, int Nk) {
    Plan p;
    p.qpairs = ceil_div(Nq, 2 * BM);
    const int key_tiles = ceil_div(Nk, BN);
    const CrossSplit s = cross_split((long long)B * Hq * p.qpairs, key_tiles, kSms, 2);
    p.splits = s.splits;
    p.tiles = s.tiles;
    p.solo = Nq <= BM && p.tiles >= 2;
    p.items = B * Hq * p.qpairs * p.splits;
    return p;
}

template <int D>
int launch(const CrossArgs& a, const Plan& plan, float* o_part, float* lse_part, int* err, int* lost,
           cudaStream_t st) {
    const void* fn = (const void*)cross_fwd_sm100_kernel<D>;
    static int launch_regs = 0;
    if (launch_regs == 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess) return SVGEAR_ERR_CUDA;
        launch_regs = fa.numRegs;
    }
    if (launch_regs < kMinLaunchRegs) return SVGEAR_ERR_UNSUPPORTED;
    Maps maps;
    if (!make_tile_map(&maps.q, a.Q, a.B, a.Hq, a.Nq, D) || !make_tile_map(&maps.o, a.O, a.B, a.Hq, a.Nq, D, 32) ||
        !make_row_maps(&maps.k, a.K, a.B, a.Hkv, a.Nk, D, a.k_len != nullptr) ||
        !make_row_maps(&maps.v, a.V, a.B, a.Hkv, a.Nk, D, a.k_len != nullptr))
        return SVGEAR_ERR_CUDA;
    const size_t smem = (size_t)(2 + ring_slots<D>()) * (D / 64) * 16384 + 8 * 4096 + 1024;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return SVGEAR_ERR_CUDA;
    cross_fwd_sm100_kernel<D><<<plan.items < kSms ? plan.items : kSms, kThreads, smem, st>>>(
        maps, a, plan, a.scale * 1.4426950408889634f, o_part, lse_part, err, lost);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

}  // namespace
}  // namespace crosstc

int cross_sm100_parts(int B, int Hq, int Nq, int Nk) {
    const crosstc::Plan p = crosstc::make_plan(B, Hq, Nq, Nk);
    return p.solo ? 2 * p.splits : p.splits;
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
