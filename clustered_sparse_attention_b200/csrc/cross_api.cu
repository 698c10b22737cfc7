// cross_api.cu -- the C ABI of the dense cross attention and the 8-bit
// activation checkpoints: argument validation, workspace layout and launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "carve.h"
#include "common.cuh"
#include "cross.h"
#include "launchers.h"

using namespace svgear;

namespace svgear {

// As many splits as fit the slots beside one another.  Item counts that do not divide
// the slots leave some empty: 77 queries read K and V at 5.6 TB/s with 24 heads (six
// splits), 5.0 with 40 (three) and 4.3 with 80 (none).
CrossSplit cross_split(long long items, int key_tiles, int slots, int min_tiles) {
    CrossSplit sp{1, key_tiles};
    const long long want = std::min<long long>(items > 0 ? slots / items : 1, key_tiles / min_tiles);
    if (want > 1) {
        sp.tiles = ceil_div(key_tiles, want);
        sp.splits = ceil_div(key_tiles, sp.tiles);
    }
    return sp;
}

}  // namespace svgear

namespace {

constexpr int kSimtMinTiles = 2;   // fewest 64-key tiles of a split

// Queries or keys of a head: rounding up to a tile must not pass 32 bits (rows that
// overlap, stride_n < d, make such lengths fit a GPU).
constexpr int kMaxLength = INT32_MAX - 1023;

int check_cross_dims(const svgear_cross_dims& d) {
    if (d.B < 0 || d.Hq < 0 || d.Hkv < 0 || d.Nq < 1 || d.Nk < 1) return SVGEAR_ERR_INVALID_ARG;
    if (d.dtype != SVGEAR_F32 && d.dtype != SVGEAR_BF16) return SVGEAR_ERR_UNSUPPORTED;
    if (d.d != 64 && d.d != 128) return SVGEAR_ERR_UNSUPPORTED;
    if ((d.Hq == 0) != (d.Hkv == 0) || (d.Hkv > 0 && d.Hq % d.Hkv != 0)) return SVGEAR_ERR_INVALID_ARG;
    if ((long long)d.B * d.Hq > 65535) return SVGEAR_ERR_UNSUPPORTED;   // grid y limit
    if ((long long)d.B * d.Hq * d.Nq >= (1ll << 31) || (long long)d.B * d.Hkv * d.Nk >= (1ll << 31))
        return SVGEAR_ERR_UNSUPPORTED;   // 32-bit row numbers
    if (d.Nq > kMaxLength || d.Nk > kMaxLength) return SVGEAR_ERR_UNSUPPORTED;
    return SVGEAR_OK;
}

// A token view of B x H x N rows of d elements: 16-byte aligned rows; an
// output's rows must not overlap.  Strides of axes of length 1 are never
// used and come back as 0.
int check_view(svgear_tokens& t, int B, int H, int N, int d, int dtype, bool output) {
    const int64_t es = dtype == SVGEAR_F32 ? 4 : 2;
    if (B == 0 || H == 0) return SVGEAR_OK;   // no row
    if (!t.data || ((uintptr_t)t.data & 15u)) return SVGEAR_ERR_INVALID_ARG;
    int64_t* st[3] = {&t.stride_b, &t.stride_h, &t.stride_n};
    const int len[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) {
        if (len[i] <= 1) {
            *st[i] = 0;
            continue;
        }
        if (*st[i] < 0 || *st[i] >= (1ll << 38) || (*st[i] * es) % 16 != 0) return SVGEAR_ERR_INVALID_ARG;
    }
    if (N > 1 && t.stride_n == 0) return SVGEAR_ERR_INVALID_ARG;
    if (output) {
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int a, int b) { return *st[a] < *st[b]; });
        int64_t extent = d;
        for (int i : order) {
            if (len[i] <= 1) continue;
            if (*st[i] < extent) return SVGEAR_ERR_INVALID_ARG;
            extent += *st[i] * (len[i] - 1);
        }
    }
    return SVGEAR_OK;
}

CrossArgs make_args(const svgear_cross_dims& d, const int32_t* k_len, float scale) {
    CrossArgs a;
    memset(&a, 0, sizeof(a));
    a.k_len = k_len;
    a.B = d.B;
    a.Hq = d.Hq;
    a.Hkv = d.Hkv;
    a.G = d.Hkv ? d.Hq / d.Hkv : 1;
    a.Nq = d.Nq;
    a.Nk = d.Nk;
    a.D = d.d;
    a.scale = scale;
    return a;
}

// Addresses that the kernels' loads and stores would fault on.
bool aligned(const void* p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
bool bad_buffers(const float* lse, const int32_t* k_len, const void* ws) {
    return !aligned(lse, sizeof(float)) || !aligned(k_len, sizeof(int32_t)) || !ws || !aligned(ws, 16);
}

bool bad_scale(float scale) { return !(scale > 0.f) || !isfinite(scale * 1.4426950408889634f); }

size_t rows_of(const svgear_cross_dims& d) { return (size_t)d.B * d.Hq * d.Nq; }

struct FwdWs {
    int* status;
    float* o_part;     // [parts][B][Hq][Nq][d], with more than one part
    float* lse_part;   // [parts][B][Hq][Nq]
    int parts;
    CrossSplit sp;     // fp32
};
FwdWs carve_fwd(Carve& cv, const svgear_cross_dims& d) {
    FwdWs w;
    if (d.dtype == SVGEAR_BF16) {
        w.parts = cross_sm100_parts(d.B, d.Hq, d.Nq, d.Nk);
    } else {
        const long long items = (long long)d.B * d.Hq * ceil_div(d.Nq, kCrossSimtM);
        w.sp = cross_split(items, ceil_div(d.Nk, kCrossSimtN), kSms, kSimtMinTiles);
        w.parts = w.sp.splits;
    }
    w.status = cv.take<int>(4);
    const size_t parts = w.parts > 1 ? w.parts * rows_of(d) : 0;
    w.o_part = cv.take<float>(parts * d.d);
    w.lse_part = cv.take<float>(parts);
    return w;
}

struct BwdWs {
    int* status;
    float* delta;   // [B][Hq][Nq]
    char* qx;       // q unpacked from its checkpoint [B][Hq][Nq][d]
    float* part;    // [kSms][2][dK, dV][keys per tile][d] partial sums
    float* dq_part; // NULL without
};
BwdWs carve_bwd(Carve& cv, const svgear_cross_dims& d, bool held) {
    BwdWs w;
    w.status = cv.take<int>(4);
    w.delta = cv.take<float>(rows_of(d));
    w.qx = cv.take<char>(held ? rows_of(d) * d.d * (d.dtype == SVGEAR_F32 ? 4 : 2) : 0);
    w.part = cv.take<float>((size_t)kSms * 2 * 2 * (d.dtype == SVGEAR_BF16 ? kCrossTcN : kCrossSimtN) * d.d);
    const size_t dq = cross_dq_part_floats(d);
    w.dq_part = cv.take<float>(dq);
    if (dq == 0) w.dq_part = nullptr;
    return w;
}

int backward(svgear_tokens dO, svgear_tokens Q, const HeldTokens* qh, svgear_tokens K, svgear_tokens V,
             svgear_tokens O, const HeldTokens* oh, const float* lse, svgear_cross_dims dims,
             const int32_t* k_len, float scale, svgear_tokens dQ, svgear_tokens dK, svgear_tokens dV,
             void* ws, size_t ws_bytes, void* stream) {
    int s = check_cross_dims(dims);
    if (s) return s;
    const int B = dims.B, Hq = dims.Hq, Hkv = dims.Hkv, Nq = dims.Nq, Nk = dims.Nk;
    if ((!qh && ((s = check_view(Q, B, Hq, Nq, dims.d, dims.dtype, false)) ||
                 (s = check_view(O, B, Hq, Nq, dims.d, dims.dtype, false)))) ||
        (s = check_view(dO, B, Hq, Nq, dims.d, dims.dtype, false)) ||
        (s = check_view(K, B, Hkv, Nk, dims.d, dims.dtype, false)) ||
        (s = check_view(V, B, Hkv, Nk, dims.d, dims.dtype, false)) ||
        (s = check_view(dQ, B, Hq, Nq, dims.d, dims.dtype, true)) ||
        (s = check_view(dK, B, Hkv, Nk, dims.d, dims.dtype, true)) ||
        (s = check_view(dV, B, Hkv, Nk, dims.d, dims.dtype, true)))
        return s;
    const bool none = B == 0 || Hq == 0;
    if ((!lse && !none) || bad_buffers(lse, k_len, ws) || bad_scale(scale)) return SVGEAR_ERR_INVALID_ARG;
    if (ws_bytes < svgear_cross_workspace_bytes(
                       qh ? SVGEAR_CROSS_BACKWARD_CKPT : SVGEAR_CROSS_BACKWARD, dims))
        return SVGEAR_ERR_WORKSPACE;
    if (none) return SVGEAR_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Carve cv(ws);
    BwdWs w = carve_bwd(cv, dims, qh != nullptr);
    CrossArgs a = make_args(dims, k_len, scale);
    if (qh) {
        Q.data = w.qx;
        Q.stride_n = dims.d;
        Q.stride_h = (int64_t)Nq * dims.d;
        Q.stride_b = Q.stride_h * Hq;
    }
    a.Q = Q; a.K = K; a.V = V; a.O = O; a.dO = dO; a.dQ = dQ; a.dK = dK; a.dV = dV;
    a.lse = const_cast<float*>(lse);
    a.delta = w.delta;
    a.dq_part = w.dq_part;
    a.status = w.status;   // cleared by the delta kernel
    if ((s = launch_cross_delta(a, dims.dtype, qh, oh, w.qx, st))) return s;
    return dims.dtype == SVGEAR_BF16 ? launch_cross_backward_sm100(a, w.part, w.status, st)
                                     : launch_cross_backward_simt(a, kSms, w.part, st);
}

int check_token_dims(const svgear_dims& d) {
    if (d.B < 0 || d.H < 0 || d.N < 1) return SVGEAR_ERR_INVALID_ARG;
    if (d.dtype != SVGEAR_F32 && d.dtype != SVGEAR_BF16) return SVGEAR_ERR_UNSUPPORTED;
    if (d.d != 64 && d.d != 128) return SVGEAR_ERR_UNSUPPORTED;
    if ((long long)d.B * d.H > 65535) return SVGEAR_ERR_UNSUPPORTED;
    if ((long long)d.B * d.H * d.N >= (1ll << 31)) return SVGEAR_ERR_UNSUPPORTED;
    return SVGEAR_OK;
}

}  // namespace

extern "C" {

size_t svgear_cross_workspace_bytes(int32_t op, svgear_cross_dims dims) {
    if (check_cross_dims(dims)) return 0;
    Carve cv(nullptr);
    if (op == SVGEAR_CROSS_FORWARD)
        carve_fwd(cv, dims);
    else if (op == SVGEAR_CROSS_BACKWARD || op == SVGEAR_CROSS_BACKWARD_CKPT)
        carve_bwd(cv, dims, op == SVGEAR_CROSS_BACKWARD_CKPT);
    else
        return 0;
    return cv.off + kAlign;
}

int svgear_cross_attend(svgear_tokens Q, svgear_tokens K, svgear_tokens V, svgear_cross_dims dims,
                        const int32_t* k_len, float scale, svgear_tokens O, float* lse, void* ws,
                        size_t ws_bytes, void* stream) {
    int s = check_cross_dims(dims);
    if (s) return s;
    if ((s = check_view(Q, dims.B, dims.Hq, dims.Nq, dims.d, dims.dtype, false)) ||
        (s = check_view(K, dims.B, dims.Hkv, dims.Nk, dims.d, dims.dtype, false)) ||
        (s = check_view(V, dims.B, dims.Hkv, dims.Nk, dims.d, dims.dtype, false)) ||
        (s = check_view(O, dims.B, dims.Hq, dims.Nq, dims.d, dims.dtype, true)))
        return s;
    const bool none = dims.B == 0 || dims.Hq == 0;
    if ((!lse && !none) || bad_buffers(lse, k_len, ws) || bad_scale(scale)) return SVGEAR_ERR_INVALID_ARG;
    if (ws_bytes < svgear_cross_workspace_bytes(SVGEAR_CROSS_FORWARD, dims)) return SVGEAR_ERR_WORKSPACE;
    if (none) return SVGEAR_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Carve cv(ws);
    FwdWs w = carve_fwd(cv, dims);
    CrossArgs a = make_args(dims, k_len, scale);
    a.Q = Q; a.K = K; a.V = V; a.O = O;
    a.lse = lse;
    if (dims.dtype == SVGEAR_BF16) {
        if (cudaMemsetAsync(w.status, 0, 4 * sizeof(int), st) != cudaSuccess) return SVGEAR_ERR_CUDA;
        s = launch_cross_sm100(a, w.o_part, w.lse_part, w.status, st);
    } else {
        a.status = w.status;
        s = launch_cross_simt(a, w.sp, w.o_part, w.lse_part, st);
    }
    if (s) return s;
    return w.parts > 1 ? launch_cross_join(a, dims.dtype, w.parts, w.o_part, w.lse_part, st)
                       : SVGEAR_OK;
}

int svgear_cross_attend_backward(svgear_tokens dO, svgear_tokens Q, svgear_tokens K, svgear_tokens V,
                                 svgear_tokens O, const float* lse, svgear_cross_dims dims,
                                 const int32_t* k_len, float scale, svgear_tokens dQ,
                                 svgear_tokens dK, svgear_tokens dV, void* ws, size_t ws_bytes,
                                 void* stream) {
    return backward(dO, Q, nullptr, K, V, O, nullptr, lse, dims, k_len, scale, dQ, dK, dV, ws,
                    ws_bytes, stream);
}

int svgear_cross_attend_backward_ckpt(svgear_tokens dO, const int8_t* q_codes, const uint8_t* q_exps,
                                      svgear_tokens K, svgear_tokens V, const int8_t* o_codes,
                                      const uint8_t* o_exps, const float* lse,
                                      svgear_cross_dims dims, const int32_t* k_len, float scale,
                                      svgear_tokens dQ, svgear_tokens dK, svgear_tokens dV, void* ws,
                                      size_t ws_bytes, void* stream) {
    if (dims.B != 0 && dims.Hq != 0 &&
        (!q_codes || !q_exps || !o_codes || !o_exps || ((uintptr_t)q_codes & 15u) ||
         ((uintptr_t)o_codes & 15u)))
        return SVGEAR_ERR_INVALID_ARG;
    const HeldTokens q{q_codes, q_exps}, o{o_codes, o_exps};
    const svgear_tokens none{nullptr, 0, 0, 0};
    return backward(dO, none, &q, K, V, none, &o, lse, dims, k_len, scale, dQ, dK, dV, ws, ws_bytes,
                    stream);
}

int svgear_checkpoint_save(svgear_tokens X, svgear_dims dims, int8_t* codes, uint8_t* exps,
                           void* stream) {
    int s = check_token_dims(dims);
    if (s) return s;
    if ((s = check_view(X, dims.B, dims.H, dims.N, dims.d, dims.dtype, false))) return s;
    if (dims.B == 0 || dims.H == 0) return SVGEAR_OK;
    if (!codes || !exps || ((uintptr_t)codes & 15u)) return SVGEAR_ERR_INVALID_ARG;
    return launch_checkpoint_save(X, dims, codes, exps, static_cast<cudaStream_t>(stream));
}

int svgear_checkpoint_load(const int8_t* codes, const uint8_t* exps, svgear_dims dims, svgear_tokens X,
                           void* stream) {
    int s = check_token_dims(dims);
    if (s) return s;
    if ((s = check_view(X, dims.B, dims.H, dims.N, dims.d, dims.dtype, true))) return s;
    if (dims.B == 0 || dims.H == 0) return SVGEAR_OK;
    if (!codes || !exps || ((uintptr_t)codes & 15u)) return SVGEAR_ERR_INVALID_ARG;
    return launch_checkpoint_load(codes, exps, dims, X, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
