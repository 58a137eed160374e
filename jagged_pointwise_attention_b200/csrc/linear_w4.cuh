// linear_w4.cuh -- projections of a few rows with 4-bit weights:
//   y[m, n] = epilogue(sum_k x[m, k] (code[n, k] - 8) scale[n, k / G] + bias[n])
// and the quantization that lays the weights out. Two codes share a byte (the
// even k in the low four bits); one bf16 scale per group of G weights of a row.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

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
    int epi;                    // 0 none, 1 SiLU, 2 residual
};

__device__ __forceinline__ void w4_store(const LinearW4Args& a, int64_t m, int n, float v) {
    if (a.bias) v += a.bias[n];
    if (a.epi == 1) v = v / (1.f + __expf(-v));
    if (a.epi == 2) v += __bfloat162float(a.r[m * a.ldr + n]);
    a.y[m * a.ldy + n] = __float2bfloat16(v);
}

// Bound by the codes' bytes. A block takes 16 MT rows of W; its warps split K
// into contiguous runs of 128-code blocks, so even one row tile spreads over
// all its bytes, and add their sums in shared memory at the end. Each warp
// streams its codes through a ring of its own (16-byte cp.async, kW4Stages
// blocks deep, no barrier of the block), which also frees the mapping of codes
// to lanes: one 4-byte word is eight consecutive codes, the four lanes of a
// fragment row hold 32 consecutive ones, so every m16n8k16 product stays inside
// one scale group whatever its size.
//
// Codes become bf16 without a conversion, a published way to unpack 4-bit weights
// whose constants follow from the format: 128 has the bits 0x4300 and a last place
// of 1, so 0x4300 | c is 128 + c, and minus 136 is exact. c - 8 and x are exact
// bf16, so a group's products and their sum are plain fp32; the scale multiplies
// the group's sum. The order of k inside a fragment is free as long as W and x
// share it: nibbles i and i + 4 of a word are one register, and x is paired to
// match.
//
// 16384 x 8192 weights, eight rows: 26.6 us (groups of 32: 38), 2.6 TB/s of codes,
// scales and x. No unit is full there: integer pipe 46%, issue slots 50%, tensor
// pipe 19%. 512 blocks of four warps, four an SM, are 0.86 of a wave: three
// blocks on 80 of the SMs, so three or four warps a scheduler, each of which waits
// for its own loads and its own sums in turn. Four row tiles a warp (29 us), two
// or eight warps a block (31 us), six stages (36 us) and x not loaded ahead (33
// us) were slower. 16 rows 41 us, 32 59, 64 92 to 96: 255 registers leave eight
// warps an SM, which wait for x and for their own results (issue slots 30%, tensor
// pipe 36%). One row tile of W for 64 rows was 128 us, two blocks of 32 rows 110.
constexpr int kW4Stages = 4;
constexpr int kW4Pitch = 80;        // bytes of a row in the ring: 64 and 16 against bank conflicts

template <int MT>
constexpr int w4_stage_bytes() { return 16 * MT * kW4Pitch; }

// (b & mask) | magic as one operation; the compiler took two.
__device__ __forceinline__ uint32_t w4_pair(uint32_t c, int p) {
    uint32_t b, v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(c >> (4 * p)), "r"(0x000f000fu), "r"(0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(b), "r"(0x43084308u));
    return v;
}

// MT: 16-row tiles of W a block; NT: 8-row tiles of x a block. G: group size.
template <int MT, int NT, int G>
__global__ void __launch_bounds__(256) linear_w4_kernel(const LinearW4Args a) {
    extern __shared__ __align__(16) uint8_t w4_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16 * MT, m0 = blockIdx.y * 8 * NT;
    const int nkb = a.K / 128;
    const int kb0 = nkb * warp / warps, kb1 = nkb * (warp + 1) / warps;
    uint8_t* ring = w4_smem + warp * kW4Stages * w4_stage_bytes<MT>();
    // copies of a block: lane's 16-byte piece of rows lane / 4, + 8, ...
    const uint8_t* src[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)     // rows past N repeat the last one
        src[i] = a.w + static_cast<int64_t>(min(n0 + 8 * i + g, a.N - 1)) * a.ldw + 16 * t;
    auto fetch = [&](int kb) {
        if (kb < kb1) {
            uint8_t* dst = ring + (kb - kb0) % kW4Stages * w4_stage_bytes<MT>();
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                cp_async16(dst + (8 * i + g) * kW4Pitch + 16 * t, src[i] + static_cast<int64_t>(kb) * 64);
        }
        cp_async_commit();
    };
    for (int s = 0; s < kW4Stages - 1; ++s) fetch(kb0 + s);

    const __nv_bfloat16* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)         // rows past M repeat the last one
        xr[n] = a.x + static_cast<int64_t>(min(m0 + 8 * n + g, a.M - 1)) * a.ldx + 8 * t;
    const __nv_bfloat16* sr[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
        sr[i] = a.s + static_cast<int64_t>(min(n0 + 8 * i + g, a.N - 1)) * a.lds;

    // the scales are loaded a block ahead; x too while that costs few registers,
    // else 32 codes ahead (24 rows, 8192 x 2048: 19.5 -> 17.4 us; two row tiles and
    // 32 rows lose an eighth by it)
    constexpr int GB = 128 / G;          // groups of a block
    constexpr bool kAhead = NT <= 2;
    constexpr bool kStep = (MT == 1 && NT == 4) || (MT == 2 && NT == 8);
    constexpr int kUnroll = kStep ? 1 : 4;      // (one row tile, 32 rows: 13 and 20 us at 4096 x 4096)
    uint4 xn[kAhead ? NT : 1][4];
    __nv_bfloat16 sn[2 * MT][GB];
    auto ahead = [&](int kb) {
        if (kb >= kb1) return;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
#pragma unroll
            for (int q = 0; q < GB; ++q) sn[i][q] = __ldg(sr[i] + kb * GB + q);
        if (kAhead) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xn[n][j] = ldg_nc_v4(xr[n] + kb * 128 + j * 32);
        }
    };
    ahead(kb0);
    uint4 xj[kStep ? NT : 1];
    if (kStep && kb0 < kb1) {
#pragma unroll
        for (int n = 0; n < NT; ++n) xj[kStep ? n : 0] = ldg_nc_v4(xr[n] + kb0 * 128);
    }
    float acc[MT][NT][4] = {};
#pragma unroll kUnroll
    for (int kb = kb0; kb < kb1; ++kb) {
        float sc[2 * MT][GB];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
#pragma unroll
            for (int q = 0; q < GB; ++q) sc[i][q] = __bfloat162float(sn[i][q]);
        uint4 xc[kAhead ? NT : 1][4];
        if (kAhead) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) xc[n][j] = xn[n][j];
        }
        ahead(kb + 1);
        fetch(kb + kW4Stages - 1);
        cp_async_wait<kW4Stages - 1>();
        __syncwarp();
        const uint8_t* st = ring + (kb - kb0) % kW4Stages * w4_stage_bytes<MT>();
        float sum[MT][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {    // 32 codes: two steps of 16
            if (j * 32 % G == 0) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[m][n][e] = 0.f;
            }
            uint32_t xb[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = kAhead ? xc[kAhead ? n : 0][j]
                                : kStep ? xj[kStep ? n : 0] : ldg_nc_v4(xr[n] + kb * 128 + j * 32);
                if (kStep && (j < 3 || kb + 1 < kb1))
                    xj[kStep ? n : 0] = ldg_nc_v4(xr[n] + kb * 128 + (j + 1) * 32);
                xb[n][0] = __byte_perm(v.x, v.z, 0x5410);
                xb[n][1] = __byte_perm(v.x, v.z, 0x7632);
                xb[n][2] = __byte_perm(v.y, v.w, 0x5410);
                xb[n][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t c0 = *reinterpret_cast<const uint32_t*>(
                    st + (16 * m + g) * kW4Pitch + 16 * j + 4 * t);
                const uint32_t c1 = *reinterpret_cast<const uint32_t*>(
                    st + (16 * m + 8 + g) * kW4Pitch + 16 * j + 4 * t);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t wf[4] = {w4_pair(c0, 2 * h), w4_pair(c1, 2 * h),
                                            w4_pair(c0, 2 * h + 1), w4_pair(c1, 2 * h + 1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16(sum[m][n], wf, xb[n][2 * h], xb[n][2 * h + 1]);
                }
            }
            if ((j + 1) * 32 % G == 0) {
                constexpr int per = G / 32;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[m][n][e] = fmaf(sc[2 * m + (e >> 1)][j / per], sum[m][n][e],
                                                acc[m][n][e]);
            }
        }
        __syncwarp();                    // the stage is read
    }
    cp_async_wait<0>();
    __syncthreads();                     // the rings are free: they hold the warps' sums now
    constexpr int R = 16 * MT, C = 8 * NT;
    float* red = reinterpret_cast<float*>(w4_smem);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(warp * C + 8 * n + 2 * t + (e & 1)) * R + 16 * m + g + 8 * (e >> 1)] = acc[m][n][e];
    __syncthreads();
    for (int i = threadIdx.x; i < R * C; i += blockDim.x) {
        const int r = i % R, c = i / R;
        if (n0 + r >= a.N || m0 + c >= a.M) continue;
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += red[(w * C + c) * R + r];
        w4_store(a, m0 + c, n0 + r, v);
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
// E consecutive weights a lane, G / E lanes a group. Loads of two bytes and stores
// of one: 16384 x 8192 weights take 236 us in groups of 128 (64: 346, 32: 366),
// the bytes alone 51; weights are laid out once.
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
