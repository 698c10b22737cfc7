// checkpoint.cu -- activation checkpoints in 8 bits: groups of 32 elements
// share a power of two 2^e, the smallest with e >= -127 for which every
// |round(x / 2^e)| is at most 127, and each element is that rounded quotient
// (half to even).  e stops at 121, where codes saturate at 127, so that a finite
// value loads as a finite one.  The scaling by a power of two is exact, so the only
// rounding is the one to the integer: |error| <= 2^(e-1), which for e > -127 is at most
// 1/127 of the group's largest magnitude (2^e and 1/127 where codes saturate).  At
// e = -127 it is the absolute 2^-128 alone: a group below that loads as zeros.
//
// Memory-bound: four units of 16 elements a thread (one 16-byte store of codes
// each, one exponent byte per two threads).  75,600 x 40 x 128 bf16 saved and loaded in
// 375 us in the first 20 ms of work and 417 sustained, 0.96 and 0.86 of the measured
// copy rate (one unit a thread took 431 where this took 392).
#include "common.cuh"
#include "cross.h"
#include "launchers.h"

namespace svgear {
namespace {

constexpr int kPer = 16;    // elements per thread and unit; two threads share a group
constexpr int kUnits = 4;   // units per thread, 256 apart, all loaded up front

// the row of tokens that holds element `row * d` of the dense order
template <typename T>
__device__ __forceinline__ T* token_row(const svgear_tokens& t, uint32_t row, uint32_t H, uint32_t N) {
    const uint32_t bh = row / N, n = row - bh * N, b = bh / H, h = bh - b * H;
    return row_ptr<T>(t, (int)b, (int)h, n);
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
checkpoint_save_kernel(svgear_tokens X, uint32_t rows, uint32_t H, uint32_t N,
                       int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
    constexpr int TR = D / kPer;   // threads per row: a power of two, so the
                                   // two threads of a group are in one warp
    const uint64_t i0 = (uint64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
    const int c = (int)(i0 % TR) * kPer;
    uint4 raw[kUnits][sizeof(T) * kPer / 16];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {   // every load before the first use
        const uint64_t row = (i0 + 256 * u) / TR;
        const T* src = token_row<const T>(X, row < rows ? (uint32_t)row : rows - 1, H, N) + c;
#pragma unroll
        for (int k = 0; k < (int)(sizeof(T) * kPer / 16); ++k)
            raw[u][k] = Elem<T>::load_raw(src + k * Elem<T>::kPerChunk);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint64_t i = i0 + 256 * u, row = i / TR;
        float x[kPer];
#pragma unroll
        for (int k = 0; k < (int)(sizeof(T) * kPer / 16); ++k) Elem<T>::unpack(raw[u][k], x + k * Elem<T>::kPerChunk);
        // magnitudes compare as integers, with infinities and NaN above the rest
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const bool finite = top < 0x7F800000u;
        // biased exponent of the step: 64 <= top / step < 128, and one more where
        // that rounds to 128 (mantissa of top >= 127.5 / 64 - 1)
        const uint32_t eb = top >> 23;
        uint32_t e8 = eb > 6 ? eb - 6 : 0u;
        if (eb >= 6 && (top & 0x7FFFFFu) >= 0x7F0000u) ++e8;
        e8 = min(e8, 248u);   // 64 steps of the next one would load as infinity
        const float inv = __uint_as_float((254u - e8) << 23);   // 1 / step, exact
        uint32_t w[kPer / 4];
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            w[q] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[q] |= ((uint32_t)max(min(__float2int_rn(x[4 * q + e] * inv), 127), -127) & 0xFFu) << (8 * e);
            if (!finite) w[q] = 0;
        }
        if (row < rows) {
            const uint64_t o = row * D + c;
            *reinterpret_cast<uint4*>(codes + o) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((i & 1) == 0) exps[o / 32] = (uint8_t)(finite ? e8 : 255u);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
checkpoint_load_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                       svgear_tokens X, uint32_t rows, uint32_t H, uint32_t N) {
    constexpr int TR = D / kPer;
    const uint64_t i0 = (uint64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
    const int c = (int)(i0 % TR) * kPer;
    uint4 raw[kUnits];
    uint32_t e8[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint64_t row = (i0 + 256 * u) / TR, o = (row < rows ? row : rows - 1) * D + c;
        raw[u] = __ldg(reinterpret_cast<const uint4*>(codes + o));
        e8[u] = __ldg(exps + o / 32);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint64_t row = (i0 + 256 * u) / TR;
        if (row >= rows) return;
        const float step = held_step(e8[u]);
        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        float x[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = (float)(int8_t)(w[e / 4] >> (8 * (e % 4))) * step;
        T* dst = token_row<T>(X, (uint32_t)row, H, N) + c;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < kPer; e += 4)
                *reinterpret_cast<float4*>(dst + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < kPer; e += 8) {
                uint32_t p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[e + 2 * k], x[e + 2 * k + 1]);
                    p[k] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(dst + e) = make_uint4(p[0], p[1], p[2], p[3]);
            }
        }
    }
}

template <typename T, int D>
int save(const svgear_tokens& X, const svgear_dims& d, int8_t* codes, uint8_t* exps, cudaStream_t st) {
    const uint32_t rows = (uint32_t)((long long)d.B * d.H * d.N);
    checkpoint_save_kernel<T, D><<<ceil_div((long long)rows * (D / kPer), 256 * kUnits), 256, 0, st>>>(
        X, rows, d.H, d.N, codes, exps);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}
template <typename T, int D>
int load(const int8_t* codes, const uint8_t* exps, const svgear_dims& d, const svgear_tokens& X,
         cudaStream_t st) {
    const uint32_t rows = (uint32_t)((long long)d.B * d.H * d.N);
    checkpoint_load_kernel<T, D><<<ceil_div((long long)rows * (D / kPer), 256 * kUnits), 256, 0, st>>>(
        codes, exps, X, rows, d.H, d.N);
    count_launches(1);
    SVGEAR_LAUNCH_CHECK();
    return SVGEAR_OK;
}

}  // namespace

int launch_checkpoint_save(svgear_tokens X, svgear_dims d, int8_t* codes, uint8_t* exps,
                           cudaStream_t st) {
    if (d.dtype == SVGEAR_F32)
        return d.d == 128 ? save<float, 128>(X, d, codes, exps, st) : save<float, 64>(X, d, codes, exps, st);
    return d.d == 128 ? save<__nv_bfloat16, 128>(X, d, codes, exps, st)
                      : save<__nv_bfloat16, 64>(X, d, codes, exps, st);
}
int launch_checkpoint_load(const int8_t* codes, const uint8_t* exps, svgear_dims d, svgear_tokens X,
                           cudaStream_t st) {
    if (d.dtype == SVGEAR_F32)
        return d.d == 128 ? load<float, 128>(codes, exps, d, X, st) : load<float, 64>(codes, exps, d, X, st);
    return d.d == 128 ? load<__nv_bfloat16, 128>(codes, exps, d, X, st)
                      : load<__nv_bfloat16, 64>(codes, exps, d, X, st);
}

}  // namespace svgear
