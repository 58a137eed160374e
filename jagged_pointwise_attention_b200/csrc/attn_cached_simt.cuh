// attn_cached_simt.cuh -- attention of new tokens over a paged cache on CUDA
// cores, fp32 arithmetic (attn_cached.cuh has the formula and the work line).
//
// A block of 128 threads takes key tiles of 64 keys for tiles of R queries: 8,
// or 16 where there are more new tokens (each tile reads its keys again).
// A tile's keys, values and timestamps are copied to shared memory at once
// (cp.async; rows padded by four floats, so the 16-byte reads of eight lanes
// fall into different banks), its pages looked up a tile ahead. There is one
// buffer, so a tile's copies are waited for before its arithmetic and overlap only
// with other blocks' (64 sequences of 200 to 1100 tokens, five in a row, 2 heads
// of 32: 29 us, the bytes alone 3.4). With many queries the arithmetic on CUDA
// cores and the keys read again for every 16 of them count (32 sequences of 256 to
// 2048, 64 drafted tokens: 211 to 262 us, the bytes alone 12.7). Scores: thread t
// has key t % 64 and half of the queries. Values: thread t has column t % DMAX of
// the output and every (128 / DMAX)-th key.
#pragma once

#include "attn_cached.cuh"

namespace hstu {

constexpr int kSimtKeys = 64;
constexpr int kSimtThreads = 128;
constexpr int kSimtBlocks = 4 * 148;

template <int DMAX, int R>
struct CachedSimtSmem {
    alignas(16) float q[R][DMAX];
    alignas(16) float k[kSimtKeys][DMAX + 4];       // columns behind dqk stay zero
    alignas(16) float v[kSimtKeys][DMAX + 4];
    alignas(16) float p[kSimtKeys][R + 4];
    int64_t tk[kSimtKeys];
    int64_t tq[R];
    int64_t scratch[kSimtThreads / 32 + 8];
    int page[kSimtKeys];            // the key's page (its number in the cache), -1 none
    int pk[kSimtKeys];
    uint32_t vis[2][kSimtKeys];     // bit i of half h: query h R / 2 + i sees the key
    float tb[64];
    TreeSmem tree;
};

// VEC: rows are 16-byte aligned, dqk and dv multiples of four
template <int DMAX, int R, bool VEC>
__global__ void __launch_bounds__(kSimtThreads) attn_cached_simt_kernel(const CachedArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using S = CachedSimtSmem<DMAX, R>;
    S& sm = *reinterpret_cast<S*>(smem_raw);
    using L = Line<kSimtKeys, R>;
    constexpr int kGroups = kSimtThreads / DMAX;        // key groups of the value pass
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    LineAt at;
    const int64_t total = L::template locate<kSimtThreads>(a, blockIdx.x, gridDim.x, sm.scratch, at,
                                                           blockIdx.x == 0);
    const int64_t begin = L::cut(total, blockIdx.x, gridDim.x);
    int64_t left = L::cut(total, blockIdx.x + 1, gridDim.x) - begin;
    if (tid == 0) write_head<kSimtKeys, R>(a, at, total, begin);
    if (left <= 0) return;
    for (int i = tid; i < kSimtKeys * (DMAX + 4); i += kSimtThreads) (&sm.k[0][0])[i] = 0.f;
    const float* qp = static_cast<const float*>(a.q);
    const float* kp = static_cast<const float*>(a.k);
    const float* vp = static_cast<const float*>(a.v);
    const int page_mask = (1 << a.shift) - 1;
    const bool use_pos = a.pos != nullptr, use_time = a.tsc != nullptr;
    int tree_of = -1, head_of = -1;
    bool first_item = true;
    while (left > 0) {
        const int nt = L::tiles(at.s, at.qt);
        const int take = static_cast<int>(min(left, static_cast<int64_t>(nt - at.j)));
        const int q0 = at.qt * R;
        const int rows = min(R, at.s.n - q0);
        const int len = at.s.ctx + min(at.s.n, q0 + R);
        if (a.parents != nullptr && tree_of != at.b) {
            build_tree(a, at.s, sm.tree, tid, kSimtThreads, [] { __syncthreads(); });
            tree_of = at.b;
        }
        __syncthreads();
        for (int i = tid; i < R * DMAX; i += kSimtThreads) {
            const int r = i / DMAX, c = i % DMAX;
            float f = 0.f;
            if (r < rows && c < a.dqk)
                f = qp[(at.s.off + q0 + r) * a.q_stride + static_cast<int64_t>(at.h) * a.dqk + c];
            sm.q[r][c] = f;
        }
        if (tid < rows && use_time) sm.tq[tid] = a.ts[at.s.off + q0 + tid];
        if (use_time && head_of != at.h) {
            if (tid < 64) sm.tb[tid] = a.tb[static_cast<int64_t>(at.h) * a.NB + min(tid, a.NB - 1)];
            head_of = at.h;
        }
        float acc[R] = {};
        const int col = tid % DMAX, grp = tid / DMAX;
        const int32_t* table = a.table + static_cast<int64_t>(at.b) * a.table_stride;
        const int64_t hk = static_cast<int64_t>(at.h) * a.dqk, hv = static_cast<int64_t>(at.h) * a.dv;
        auto look = [&](int key) { return tid < kSimtKeys && key < len ? __ldg(table + (key >> a.shift)) : 0; };
        int ahead = look(at.j * kSimtKeys + tid);
        for (int j = at.j; j < at.j + take; ++j) {
            const int k0 = j * kSimtKeys, nk = min(kSimtKeys, len - k0);
            // the tile's keys: page, position
            __syncthreads();
            if (tid < kSimtKeys) {
                int page = -1, pk = 0;
                if (tid < nk) {
                    const int key = k0 + tid;
                    page = ahead;
                    if (page < 0 || page >= a.num_pages) {
                        raise_error(kErrBadInput);
                        page = -1;
                    }
                    pk = key;
                    if (a.parents != nullptr && key >= at.s.ctx)
                        pk = at.s.ctx + sm.tree.depth[key - at.s.ctx];
                    if (use_time && page >= 0)
                        cp_async8(&sm.tk[tid], a.tsc + page * a.tsc_page + (key & page_mask));
                }
                sm.page[tid] = page;
                sm.pk[tid] = pk;
            }
            __syncthreads();
            constexpr int W = VEC ? 4 : 1;          // floats a copy
            const int ck = a.dqk / W, cv = a.dv / W;
            for (int i = tid; i < kSimtKeys * (DMAX / W); i += kSimtThreads) {
                const int r = i / (DMAX / W), c = i % (DMAX / W);
                if (sm.page[r] < 0) continue;
                const int64_t row = (k0 + r) & page_mask;
                if (c < ck) {
                    const float* src = kp + sm.page[r] * a.k_page + row * a.k_tok + hk + W * c;
                    if (VEC) cp_async16(&sm.k[r][W * c], src);
                    else cp_async4(&sm.k[r][c], src);
                }
                if (c < cv) {
                    const float* src = vp + sm.page[r] * a.v_page + row * a.v_tok + hv + W * c;
                    if (VEC) cp_async16(&sm.v[r][W * c], src);
                    else cp_async4(&sm.v[r][c], src);
                }
            }
            ahead = look(k0 + kSimtKeys + tid);
            cp_async_wait_all();
            __syncthreads();
            // scores of key tid % 64 and half of the queries
            {
                constexpr int HALF = R / 2;
                const int r = tid % kSimtKeys, half = tid / kSimtKeys, i0 = half * HALF;
                float s[HALF] = {};
                for (int c = 0; c < a.dqk; c += 4) {
                    const float4 kv = *reinterpret_cast<const float4*>(&sm.k[r][c]);
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        const float4 qv = *reinterpret_cast<const float4*>(&sm.q[i0 + i][c]);
                        s[i] = fmaf(kv.x, qv.x, s[i]);
                        s[i] = fmaf(kv.y, qv.y, s[i]);
                        s[i] = fmaf(kv.z, qv.z, s[i]);
                        s[i] = fmaf(kv.w, qv.w, s[i]);
                    }
                }
                const int m = k0 + r - at.s.ctx;        // new token's index, < 0: cached
                uint32_t vis = 0u;
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    const int qi = q0 + i0 + i;
                    bool see = sm.page[r] >= 0 && i0 + i < rows;
                    if (m >= 0)
                        see = see && (a.parents != nullptr
                                          ? ((sm.tree.seen[qi >> 5][m] >> (qi & 31)) & 1u) != 0u
                                          : m <= qi);
                    float p = 0.f;
                    if (see) {
                        const int pq = at.s.ctx + (a.parents != nullptr ? sm.tree.depth[qi] : qi);
                        float x = s[i];
                        if (use_pos)
                            x += a.pos[static_cast<int64_t>(at.h) * a.P + min(pq - sm.pk[r], a.P - 1)];
                        if (use_time) x += sm.tb[time_bucket64(sm.tq[i0 + i] - sm.tk[r], 63)];
                        p = x / (1.f + expf(-x));
                        vis |= 1u << i;
                    }
                    sm.p[r][i0 + i] = p;
                }
                sm.vis[half][r] = vis;
            }
            __syncthreads();
            if (col < a.dv) {
                const uint32_t every = 0xffffffffu >> (32 - rows);
                for (int r = grp; r < nk; r += kGroups) {
                    const float v = sm.v[r][col];
                    const uint32_t vis = sm.vis[0][r] | (sm.vis[1][r] << (R / 2));
                    if (vis == every) {
#pragma unroll
                        for (int i = 0; i < R; i += 4) {
                            const float4 p = *reinterpret_cast<const float4*>(&sm.p[r][i]);
                            acc[i] = fmaf(p.x, v, acc[i]);
                            acc[i + 1] = fmaf(p.y, v, acc[i + 1]);
                            acc[i + 2] = fmaf(p.z, v, acc[i + 2]);
                            acc[i + 3] = fmaf(p.w, v, acc[i + 3]);
                        }
                    } else {
                        // a key that a query does not see adds nothing, whatever its value
                        // is (not 0 * v, which is NaN for a v that is not finite)
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if ((vis >> i) & 1u) acc[i] = fmaf(sm.p[r][i], v, acc[i]);
                    }
                }
            }
        }
        float(*red)[DMAX] = reinterpret_cast<float(*)[DMAX]>(&sm.v[0][0]);    // V has been read by then
        // sum over the key groups, then the rows (or this block's part of them)
        if (kGroups > 1) {
            for (int g = 1; g < kGroups; ++g) {
                __syncthreads();
                if (grp == g) {
#pragma unroll
                    for (int i = 0; i < R; ++i) red[i][col] = acc[i];
                }
                __syncthreads();
                if (grp == 0) {
#pragma unroll
                    for (int i = 0; i < R; ++i) acc[i] += red[i][col];
                }
            }
        }
        if (grp == 0 && col < a.dv) {
            const bool whole = take == nt;
            float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (first_item ? 0 : 1)) *
                                        a.part_rows * a.dv;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i >= rows) break;
                if (whole)
                    static_cast<float*>(a.out)[(at.s.off + q0 + i) * a.out_stride +
                                               static_cast<int64_t>(at.h) * a.dv + col] =
                        acc[i] * a.inv_n;
                else
                    part[i * a.dv + col] = acc[i];
            }
        }
        left -= take;
        first_item = false;
        if (left > 0) L::next_item(a, at);
    }
}

}  // namespace hstu
