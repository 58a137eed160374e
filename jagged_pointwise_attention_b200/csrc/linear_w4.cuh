// linear_w4.cuh -- projections of a few rows with 4-bit weights:
//   y[m, n] = epilogue(sum_k x[m, k] (code[n, k] - 8) scale[n, k / G] + bias[n])
// and the quantization that lays the weights out. Two codes share a byte (the
// even k in the low four bits); one bf16 scale per group of G weights of a row.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ln_gate.cuh"

namespace hstu {

struct LinearW4Args {
    const __nv_bfloat16* x;
    int64_t ldx;
    int M, K, N, G;
    const uint8_t* w;           // [N, K / 2], row stride ldw bytes
    int64_t ldw;
    const __nv_bfloat16* s;     // [N, K / G], row stride lds
    int64_t lds;
    const float* bias;          // [N] or null
    const __nv_bfloat16* r;     // residual
    int64_t ldr;
    __nv_bfloat16* y;
    int64_t ldy;
};

// epilogue: 0 none, 1 SiLU, 2 residual
template <int EPI>
__device__ __forceinline__ void w4_store(const LinearW4Args& a, int m, int n, float v) {
    if (a.bias) v += a.bias[n];
    if (EPI == 1) v = v / (1.f + __expf(-v));
    if (EPI == 2) v += __bfloat162float(a.r[m * a.ldr + n]);
    a.y[m * a.ldy + n] = __float2bfloat16(v);
}

// One warp per weight row and eight rows of x.
template <int EPI>
__global__ void __launch_bounds__(128) linear_w4_kernel(const LinearW4Args a) {
    const int n = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int m0 = blockIdx.y * 8, mr = min(8, a.M - m0);
    if (n >= a.N) return;
    float acc[8] = {};
    for (int k = lane * 8; k < a.K; k += 256) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(a.w + n * a.ldw + k / 2);
        const float s = __bfloat162float(a.s[n * a.lds + k / a.G]);
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = (static_cast<int>((c >> (4 * e)) & 15u) - 8) * s;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            if (m < mr) {
                float f[8];
                unpack8(*reinterpret_cast<const uint4*>(a.x + (m0 + m) * a.ldx + k), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m] = fmaf(w[e], f[e], acc[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 8; ++m) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        if (lane == 0 && m < mr) w4_store<EPI>(a, m0 + m, n, acc[m]);
    }
}

// ------------------------------------------------------------------ quantization

struct QuantW4Args {
    const __nv_bfloat16* w;     // [N, K], row stride ldw
    int64_t ldw;
    int64_t N;
    int K;
    uint8_t* codes;             // [N, K / 2], row stride ldc
    int64_t ldc;
    __nv_bfloat16* s;           // [N, K / G], row stride lds
    int64_t lds;
};

// scale = bf16(amax / 7), code = clamp(rint(w / scale), -8, 7) + 8. The codes
// are taken with the rounded scale, the one that the product uses. A group of
// zeros (or one whose scale rounds to zero) gets scale 1 and codes 8; a group
// with a weight that is not finite gets scale NaN, so the product shows it.
// E consecutive weights a lane, G / E lanes a group.
template <int G>
__global__ void __launch_bounds__(256) quant_w4_kernel(const QuantW4Args a) {
    constexpr int E = G == 128 ? 4 : 2, L = G / E;
    const int groups = a.K / G;
    const int64_t total = a.N * groups;
    const int lane = threadIdx.x & 31;
    // the warp's first group; a warp covers 32 / L groups
    for (int64_t w0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (32 / L);
         w0 < total; w0 += static_cast<int64_t>(gridDim.x) * 8 * (32 / L)) {
        const int64_t gi = w0 + lane / L;
        const bool live = gi < total;
        const int64_t n = live ? gi / groups : 0;
        const int g = live ? static_cast<int>(gi % groups) : 0;
        const int k = g * G + (lane % L) * E;
        uint32_t bits[E];
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            bits[e] = live ? static_cast<uint32_t>(__bfloat16_as_ushort(a.w[n * a.ldw + k + e])) << 16
                           : 0u;
            top = max(top, bits[e] & 0x7fffffffu);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool finite = top < 0x7f800000u;
        const float amax = __uint_as_float(top);
        __nv_bfloat16 s = __float2bfloat16(amax / 7.f);
        const bool zero = __bfloat162float(s) == 0.f;
        const float sf = zero ? 1.f : __bfloat162float(s);
        uint32_t word = 0u;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            int c = 8;
            if (finite && !zero) {
                const float q = rintf(__uint_as_float(bits[e]) / sf);
                c = static_cast<int>(fminf(fmaxf(q, -8.f), 7.f)) + 8;
            }
            word |= static_cast<uint32_t>(c) << (4 * e);
        }
        if (live) {
            uint8_t* dst = a.codes + n * a.ldc + k / 2;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) dst[e] = static_cast<uint8_t>(word >> (8 * e));
            if (lane % L == 0)
                a.s[n * a.lds + g] = finite ? __float2bfloat16(sf)
                                            : __ushort_as_bfloat16(static_cast<unsigned short>(0x7fff));
        }
    }
}

}  // namespace hstu
