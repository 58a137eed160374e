// attn_cached_mma.cuh -- attention of up to sixteen new tokens over short paged
// sequences, which a block takes whole, and of heads of 32, bf16
// (attn_cached.cuh has the formula and the work line).
//
// Bound by latencies and the cache's bytes, so the layout serves the loads.
// Keys come in groups of 16, which never cross a page. Each warp of a block
// (four for whole sequences, so that blocks share an SM, twelve along the line)
// takes every n-th group of the block's part and feeds itself: its lane
// 0 issues the TMA loads of a group's K and V rows into the warp's own ring,
// groups ahead and across item borders, so no barrier of the block stands
// between two loads. The tokens' timestamps ride on the same barrier as 8-byte
// copies. 128 sequences of 20 to 200 tokens, 2 heads of 64, one new token: 9.6
// us with its launch, of which about 7 are dependent loads: lengths, page
// numbers, keys and values, and above 128 tokens keys and values once more (a
// warp has two groups in flight and up to four to read).
//
// Products run as 16 keys x 8 queries (m16n8k16), transposed against the usual
// order: S^T = K Q^T and O^T = V^T P^T. So the long axis fills the 16 rows, a
// single query wastes seven columns of eight and not fifteen of sixteen, and
// P^T comes out of the first product's layout by one 8 x 8 transpose a tile
// (movmatrix). The tensor pipe idles either way; on tcgen05, with a block an
// SM, the same sequences took 21 us. P is rounded to bf16 as in the tcgen05 kernel.
//
// Heads of 32 take tiles of at most 32 queries, each of which reads the cache
// again: one token over 16 sequences of up to 8192, 16 heads: 85 us (bytes alone
// 28); trees of 64 over 32 of 256 to 4096: 422 us (23).
#pragma once

#include "attn_cached.cuh"

namespace hstu {

constexpr int kMmaKeys = 16;            // keys of a group

template <int D, int NT, bool WHOLE>
struct CachedMmaSmem {
    // Whole items: four warps, so that blocks share an SM. 92 KB a block at heads
    // of 128 (rings 64, sums 17, tree 9), 52 at 64 and 32 at 32: two blocks an SM,
    // four and six; launched for two, and for three at 64 and 32.
    static constexpr int kWarps = WHOLE ? 4 : 12;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kBlocksPerSm = !WHOLE ? 1 : D == 128 ? 2 : 3;
    static constexpr int kNQ = 8 * NT;
    static constexpr int kRowBytes = D >= 64 ? 128 : 64;    // bytes of a box row
    static constexpr int kBoxes = D / 64 > 0 ? D / 64 : 1;
    static constexpr int kBoxBytes = kMmaKeys * kRowBytes;
    static constexpr int kHalfBytes = kBoxes * kBoxBytes;   // K or V of a group
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kStages = D == 128 || WHOLE ? 2 : 4;
    static constexpr int kPitch = D + 4;                    // of a row of the sums, floats
    // copies of the sums: fewer where a copy is large
    static constexpr int kCopies = NT == 1 ? 4 : NT == 2 ? 2 : 1;
    static constexpr int kOffRed = kWarps * kStages * kStageBytes;
    static constexpr int kOffQ = kOffRed;                   // NT > 2: until the sums come
    static constexpr int kQPitch = D * 2 + 16;
    static constexpr int kOffTk = kOffRed + kCopies * kNQ * kPitch * 4;    // [warp][stage][16]
    static constexpr int kOffTq = kOffTk + kWarps * kStages * kMmaKeys * 8;
    static constexpr int kOffTb = kOffTq + kNQ * 8;
    static constexpr int kOffBar = kOffTb + 64 * 4;
    static constexpr int kOffPage = kOffBar + kWarps * kStages * 8;
    static constexpr int kOffScratch = kOffPage + kWarps * kStages * 4;
    static constexpr int kOffTree = (kOffScratch + (kWarps + 8) * 8 + 15) / 16 * 16;
    static constexpr int kOffOdd = kOffTree + static_cast<int>(sizeof(TreeSmem));
    static constexpr int kOffAbort = kOffOdd + 8 * 4;
    static constexpr int kBytes = kOffAbort + 16;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory per block");
};

// What the keys of `odd` (counted from part0) add to columns c, c + 1 of new
// token qi.
template <int D>
__device__ __noinline__ float2 odd_sum(const CachedArgs& a, const uint32_t* odd, const TreeSmem& tree,
                                       int64_t off, int b, int h, int ctx, int part0, int qi, int c) {
    float2 sum = make_float2(0.f, 0.f);
    const bool chain = a.parents == nullptr;
#pragma unroll 1
    for (int o = 0; o < kMaxTree; ++o) {
        if (!((odd[o >> 5] >> (o & 31)) & 1u)) continue;
        const int key = part0 + o, m = key - ctx;
        if (chain ? m > qi : !((tree.seen[qi >> 5][m] >> (qi & 31)) & 1u)) continue;
        const int page = a.table[static_cast<int64_t>(b) * a.table_stride + (key >> a.shift)];
        const int row = key & ((1 << a.shift) - 1);
        const float p = odd_weight<D>(a, h, off + qi, ctx + (chain ? qi : tree.depth[qi]),
                                      page, row, chain ? key : ctx + tree.depth[m]);
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + page * a.v_page +
                                 row * a.v_tok + static_cast<int64_t>(h) * D + c;
        sum.x = fmaf(p, __bfloat162float(v[0]), sum.x);
        sum.y = fmaf(p, __bfloat162float(v[1]), sum.y);
    }
    return sum;
}

// WHOLE: block i takes item i whole (short sequences: no part, no join, no
// search); otherwise an equal part of the line.
template <int D, int NT, bool WHOLE>
__global__ void __launch_bounds__(CachedMmaSmem<D, NT, WHOLE>::kThreads,
                                  CachedMmaSmem<D, NT, WHOLE>::kBlocksPerSm)
attn_cached_mma_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CachedArgs a, int qtiles) {
    using S = CachedMmaSmem<D, NT, WHOLE>;
    using L = Line<kMmaKeys, S::kNQ>;
    constexpr int NQ = S::kNQ, ST = S::kStages, KS = D / 16;
    constexpr int kMmaWarps = S::kWarps, kMmaThreads = S::kThreads;
    constexpr bool kQRegs = NT <= 2;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps seeing shared memory)
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;      // fragment row, column pair
    uint8_t* ring = smem + warp * ST * S::kStageBytes;
    float* red = reinterpret_cast<float*>(smem + S::kOffRed);
    int64_t* tks = reinterpret_cast<int64_t*>(smem + S::kOffTk) + warp * ST * kMmaKeys;
    int64_t* tqs = reinterpret_cast<int64_t*>(smem + S::kOffTq);
    float* tbs = reinterpret_cast<float*>(smem + S::kOffTb);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBar) + warp * ST;
    int* pages = reinterpret_cast<int*>(smem + S::kOffPage) + warp * ST;
    int64_t* scratch = reinterpret_cast<int64_t*>(smem + S::kOffScratch);
    TreeSmem& tree = *reinterpret_cast<TreeSmem*>(smem + S::kOffTree);
    uint32_t* odd = reinterpret_cast<uint32_t*>(smem + S::kOffOdd);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffAbort);
    const bool use_pos = a.pos != nullptr, use_time = a.tsc != nullptr;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(&full[s], 33);   // expect_tx + 32 copy arrivals
        mbar_fence_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    LineAt at;
    int64_t left;               // groups of the block's part that are not done
    if (WHOLE) {
        at.h = blockIdx.x % a.H;
        at.qt = blockIdx.x / a.H % qtiles;
        at.b = blockIdx.x / a.H / qtiles;
        at.j = 0;
        bool ok;
        at.s = cached_seq(a, at.b, ok);
        ok = ok && (at.b > 0 || at.s.off == 0);
        if (!ok && at.h == 0 && at.qt == 0 && tid == 0) raise_error(kErrBadInput);
        left = at.qt * NQ < at.s.n ? L::tiles(at.s, at.qt) : 0;
        __syncthreads();
    } else {
        const int64_t total = L::template locate<kMmaThreads>(a, blockIdx.x, gridDim.x, scratch, at,
                                                              blockIdx.x == 0);
        const int64_t begin = L::cut(total, blockIdx.x, gridDim.x);
        left = L::cut(total, blockIdx.x + 1, gridDim.x) - begin;
        if (tid == 0) write_head<kMmaKeys, NQ>(a, at, total, begin);
    }
    if (left <= 0) return;

    // ---- loads: this warp's next group, a cursor of its own
    LineAt lat = at;
    int64_t lleft = left;                               // from lat's item on
    int lend = static_cast<int>(min(lleft, static_cast<int64_t>(L::tiles(lat.s, lat.qt) - lat.j)));
    int lj = lat.j + warp;                              // next group of the item
    lend += lat.j;
    int lpage = -1, lstage = 0, issued = 0;
    bool more = true;
    auto seek = [&]() {         // to the next group of this warp; starts the load of its page
        while (lj >= lend) {
            lleft -= lend - lat.j;
            if (lleft <= 0) {
                more = false;
                return;
            }
            L::next_item(a, lat);
            lend = static_cast<int>(min(lleft, static_cast<int64_t>(L::tiles(lat.s, lat.qt))));
            lj = warp;
        }
        lpage = __ldg(a.table + static_cast<int64_t>(lat.b) * a.table_stride +
                      ((lj * kMmaKeys) >> a.shift));
    };
    auto issue = [&]() {
        if (!more) return;
        const int row = (lj * kMmaKeys) & ((1 << a.shift) - 1);
        const bool good = lpage >= 0 && lpage < a.num_pages;
        uint8_t* dst = ring + lstage * S::kStageBytes;
        if (lane == 0) {
            if (!good) raise_error(kErrBadInput);
            pages[lstage] = good ? lpage : -1;
            mbar_arrive_expect_tx(&full[lstage], S::kStageBytes);
            const int z = good ? lpage : a.num_pages;   // past the cache: zeros
#pragma unroll
            for (int i = 0; i < S::kBoxes; ++i) {
                tma_load_3d(dst + i * S::kBoxBytes, &tmK, &full[lstage], lat.h * D + 64 * i, row, z);
                tma_load_3d(dst + S::kHalfBytes + i * S::kBoxBytes, &tmV, &full[lstage],
                            lat.h * D + 64 * i, row, z);
            }
        }
        if (use_time && good && lane < kMmaKeys)
            cp_async8(tks + lstage * kMmaKeys + lane, a.tsc + lpage * a.tsc_page + row + lane);
        cp_async_arrive(&full[lstage]);
        lstage = lstage + 1 == ST ? 0 : lstage + 1;
        ++issued;
        lj += kMmaWarps;
        seek();
    };
    seek();
    __syncwarp();

    // ---- the items
    int stage = 0;
    uint32_t phase = 0;
    int tree_of = -1, head_of = -1;
    bool first_item = true, failed = false;
    while (left > 0) {
        const int nt = L::tiles(at.s, at.qt);
        const int take = static_cast<int>(min(left, static_cast<int64_t>(nt - at.j)));
        const int q0 = at.qt * NQ, rows = min(NQ, at.s.n - q0);
        const int len = at.s.ctx + min(at.s.n, q0 + NQ);
        // keys from here on are seen by some queries and not by others
        const int part0 = at.s.ctx + (a.parents != nullptr ? 0 : q0);
        if (a.parents != nullptr && tree_of != at.b) {
            build_tree(a, at.s, tree, tid, kMmaThreads, [] { __syncthreads(); });
            tree_of = at.b;
        }
        const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) +
                                  (at.s.off + q0) * a.q_stride + static_cast<int64_t>(at.h) * D;
        // the item's own loads are on their way before the ring's first ones
        const int64_t tq_mine = use_time && tid < NQ ? __ldg(a.ts + at.s.off + q0 + min(tid, rows - 1)) : 0;
        const bool new_head = use_time && head_of != at.h && tid >= 64 && tid < 128;
        const float tb_mine = new_head ? __ldg(a.tb + static_cast<int64_t>(at.h) * a.NB +
                                               min(tid - 64, a.NB - 1))
                                       : 0.f;
        head_of = at.h;
        // Q^T fragments; queries behind the last are zeros
        uint32_t qf[kQRegs ? NT : 1][KS][2];
        if (!kQRegs) __syncthreads();   // the previous item's sums have been read
        if (kQRegs) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int r = 8 * n + g;
                    const uint32_t* p =
                        reinterpret_cast<const uint32_t*>(qp + r * a.q_stride + ks * 16 + 2 * t);
                    qf[n][ks][0] = r < rows ? __ldg(p) : 0u;
                    qf[n][ks][1] = r < rows ? __ldg(p + 4) : 0u;
                }
        } else {
            for (int i = tid; i < NQ * (D / 8); i += kMmaThreads) {
                const int r = i / (D / 8), c = i % (D / 8);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) v = ldg_nc_v4(qp + r * a.q_stride + 8 * c);
                *reinterpret_cast<uint4*>(smem + S::kOffQ + r * S::kQPitch + 16 * c) = v;
            }
        }
        if (first_item) {
#pragma unroll 1
            for (int s = 0; s < ST; ++s) issue();
        }
        __syncthreads();        // the previous item's tables and sums have been read
        if (use_time && tid < NQ) tqs[tid] = tq_mine;
        if (tid >= 32 && tid < 40) odd[tid - 32] = 0u;      // new keys to be added alone
        if (new_head) tbs[tid - 64] = tb_mine;
        int pq[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = min(q0 + 8 * n + 2 * t + e, at.s.n - 1);
                pq[n][e] = at.s.ctx + (a.parents != nullptr ? tree.depth[r] : r);
            }
        __syncthreads();
        // timestamps of the lane's queries: low words, and the item's extremes,
        // with which a group sees whether its differences fit in 32 bits
        int tql[NT][2];
        int64_t tmin = 0, tmax = 0;
        if (use_time) {
            tmin = tmax = tqs[0];
#pragma unroll 1
            for (int i = 1; i < rows; ++i) {
                tmin = min(tmin, tqs[i]);
                tmax = max(tmax, tqs[i]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) tql[n][e] = static_cast<int>(tqs[8 * n + 2 * t + e]);
        }
        const float* posh = use_pos ? a.pos + static_cast<int64_t>(at.h) * a.P : nullptr;
        float acc[KS][NT][4];
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;

#pragma unroll 1
        for (int j = at.j + warp; j < at.j + take; j += kMmaWarps) {
            const int k0 = j * kMmaKeys;
            const bool tail = k0 + kMmaKeys > at.s.ctx;     // new tokens, or rows behind them
            // position biases of keys k0 + g and k0 + g + 8 (row r of the pair)
            int pk[2] = {k0 + g, k0 + g + 8};
            if (tail && a.parents != nullptr) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int m = pk[r] - at.s.ctx;
                    if (m >= 0) pk[r] = at.s.ctx + tree.depth[min(m, at.s.n - 1)];
                }
            }
            float x[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int rel = min(pq[n][e & 1] - pk[e >> 1], a.P - 1);
                    if (tail) rel = max(rel, 0);    // a new token that is not seen
                    x[n][e] = use_pos ? __ldg(posh + rel) : 0.f;
                }
            if (!failed && !warp_wait(&full[stage], phase, abort_flag)) {
                failed = true;
                if (lane == 0) raise_error(kErrTimeout);
            }
            const bool paged = pages[stage] >= 0;
            const uint32_t kb = smem_u32(ring + stage * S::kStageBytes);
            const uint32_t vb = kb + S::kHalfBytes;
            // S^T = K Q^T
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t kf[4];
                const int r = lane & 15, c = 2 * ks + (lane >> 4);
                const uint32_t ad =
                    D >= 64 ? kb + (c >> 3) * S::kBoxBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)
                            : kb + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
                ldsm4(ad, kf);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t b0, b1;
                    if (kQRegs) {
                        b0 = qf[n][ks][0];
                        b1 = qf[n][ks][1];
                    } else {
                        const uint32_t* p = reinterpret_cast<const uint32_t*>(
                            smem + S::kOffQ + (8 * n + g) * S::kQPitch + ks * 32 + 4 * t);
                        b0 = p[0];
                        b1 = p[4];
                    }
                    mma_bf16(s[n], kf, b0, b1);
                }
            }
            // scores to weights
            if (use_time) {
                const int64_t tk0 = tks[stage * kMmaKeys + g], tk1 = tks[stage * kMmaKeys + g + 8];
                const int64_t lim = int64_t{1} << 31;
                const bool near = tmax - tk0 < lim && tmax - tk1 < lim && tmin - tk0 > -lim &&
                                  tmin - tk1 > -lim;
                if (__all_sync(0xffffffffu, near)) {
                    const int kl[2] = {static_cast<int>(tk0), static_cast<int>(tk1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[n][e] += table_at(tbs, bucket_bytes(tql[n][e & 1] - kl[e >> 1]) - kBucketBias);
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[n][e] += tbs[time_bucket64(
                                tqs[8 * n + 2 * t + (e & 1)] - (e >> 1 ? tk1 : tk0), 63)];
                }
            }
            uint32_t pf[NT][2];
            float p[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f = s[n][e] + x[n][e];
                    bool see = paged;
                    if (tail) {
                        const int m = k0 + g + 8 * (e >> 1) - at.s.ctx;
                        const int qi = q0 + 8 * n + 2 * t + (e & 1);
                        if (m >= at.s.n || qi >= at.s.n) see = false;
                        else if (m >= 0)
                            see = see && (a.parents != nullptr
                                              ? ((tree.seen[qi >> 5][m] >> (qi & 31)) & 1u) != 0u
                                              : m <= qi);
                    }
                    p[n][e] = see ? silu_exp(f) : 0.f;
                }
                pf[n][0] = movm_t(pack_bf16x2(p[n][0], p[n][1]));
                pf[n][1] = movm_t(pack_bf16x2(p[n][2], p[n][3]));
            }
            // O^T += V^T P^T. Rows of V that some query does not see are
            // multiplied by zero, so they have to be finite: rows behind the
            // sequence and rows of new tokens that are not finite are cleared,
            // and the latter are added alone to the queries that see them.
            if (tail) {
                const int nk = min(kMmaKeys, len - k0);
                uint32_t gone = 0xffffu & ~((1u << nk) - 1u);
                const int r = lane & 15;
                if (k0 + r >= at.s.ctx && r < nk) {
                    bool bad = false;
#pragma unroll 1
                    for (int c = lane >> 4; c < D / 8; c += 2) {
                        const int cc = D >= 64 ? ((c & 7) ^ (r & 7)) : (c ^ ((r >> 1) & 3));
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            ring + stage * S::kStageBytes + S::kHalfBytes + (c >> 3) * S::kBoxBytes +
                            r * S::kRowBytes + (cc << 4));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad = bad || (w[i] & 0x7f80u) == 0x7f80u ||
                                  (w[i] & 0x7f800000u) == 0x7f800000u;
                    }
                    // (a key that a chain's whole tile sees counts as it is)
                    if (bad && k0 + r >= part0) {
                        gone |= 1u << r;
                        atomicOr(&odd[(k0 + r - part0) >> 5], 1u << ((k0 + r - part0) & 31));
                    }
                }
                gone = __reduce_or_sync(0xffffffffu, gone);
                if (gone) {
#pragma unroll 1
                    for (int i = lane; i < S::kHalfBytes / 16; i += 32) {
                        const int r = i * 16 / S::kRowBytes % kMmaKeys;
                        if ((gone >> r) & 1u)
                            *reinterpret_cast<uint4*>(ring + stage * S::kStageBytes + S::kHalfBytes +
                                                      i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();   // the next TMA copy comes after these stores
                    __syncwarp();
                }
            }
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                uint32_t vf[4];
                const int mi = lane >> 3, r = (lane & 7) + (mi >> 1) * 8, c = 2 * m + (mi & 1);
                const uint32_t ad =
                    D >= 64 ? vb + (c >> 3) * S::kBoxBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)
                            : vb + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
                ldsm4_t(ad, vf);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(acc[m][n], vf, pf[n][0], pf[n][1]);
            }
            __syncwarp();               // the stage is read: fill it again
            issue();
            stage = stage + 1 == ST ? 0 : stage + 1;
            phase ^= stage == 0;
        }
        if (!kQRegs) __syncthreads();   // Q has been read by every warp
        // sum over the warps: warp w adds to copy w % kCopies, kCopies at a time
#pragma unroll 1
        for (int r = 0; r < kMmaWarps / S::kCopies; ++r) {
            if (r > 0) __syncthreads();
            if (warp / S::kCopies == r) {
                float* dst = red + (warp % S::kCopies) * NQ * S::kPitch + 2 * t * S::kPitch + g;
                // all of a row tile's sums are read before the first is written
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    float old[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            old[n][e] = r == 0 ? 0.f
                                               : dst[(8 * n + (e & 1)) * S::kPitch + 16 * m + 8 * (e >> 1)];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[(8 * n + (e & 1)) * S::kPitch + 16 * m + 8 * (e >> 1)] =
                                old[n][e] + acc[m][n][e];
                }
            }
        }
        __syncthreads();
        const bool whole = WHOLE || take == nt;
        uint32_t any_odd = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) any_odd |= odd[i];
        float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (first_item ? 0 : 1)) * a.part_rows * D;
        for (int i = tid; i < rows * (D / 2); i += kMmaThreads) {
            const int r = i / (D / 2), c = 2 * (i % (D / 2));
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < S::kCopies; ++w) {
                const float2 u = *reinterpret_cast<const float2*>(red + (w * NQ + r) * S::kPitch + c);
                v.x += u.x;
                v.y += u.y;
            }
            if (any_odd) {
                const float2 u = odd_sum<D>(a, odd, tree, at.s.off, at.b, at.h, at.s.ctx, part0, q0 + r, c);
                v.x += u.x;
                v.y += u.y;
            }
            if (whole)
                *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                             (at.s.off + q0 + r) * a.out_stride +
                                             static_cast<int64_t>(at.h) * D + c) =
                    pack_bf16x2(v.x * a.inv_n, v.y * a.inv_n);
            else
                *reinterpret_cast<float2*>(part + r * D + c) = v;
        }
        left -= take;
        first_item = false;
        if (left > 0) L::next_item(a, at);
    }
    // after a wait that gave up: no copy may land behind the block's end
    if (failed) {
        for (int i = max(0, issued - ST); i < issued; ++i)
            mbar_wait(&full[i % ST], (i / ST) & 1, nullptr, kWaitLimitCycles / 16);
    }
}

}  // namespace hstu
