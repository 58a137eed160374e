// attn_cached_tc.cuh -- attention of many new tokens (trees of dozens, rows of
// candidates, pieces of a prompt) over a paged cache, bf16 on tcgen05
// (attn_cached.cuh has the formula and the work line).
//
// Items are tiles of NQ queries of one head; a step is 128 keys:
//   S^T [128 keys x nq]   = K Q^T              TMEM, two buffers
//   P^T = silu(S^T + biases), bf16             shared memory, two buffers
//   O^T [D x nq]         += V^T P^T            TMEM, two buffers (items)
// The long axis fills the 128 rows of the first product and the head the rows
// of the second, so the width of both is the item's own count of queries
// (rounded up to 16), and few queries cost few columns. A thread of the
// pointwise stage owns one key: its position and timestamp are its own, the
// queries' come as broadcasts, and its row of P^T is an operand with the
// queries contiguous. (Heads of 64: rows 64 to 127 of the second product read
// the same V once more and nobody reads them.)
//
// Warp roles, so that nothing but the pointwise stage itself stands between
// two steps, across items too:
//   0-7   pointwise, two groups of four that take turns at the steps
//   8-11  the items' rows: O^T to the output or to the block's part
//   12    K and V by TMA, a page (or 128 tokens of one) a box, a lane a page,
//         and the keys' timestamps; both in the order the products use them,
//         K0 K1 V0 K2 V1 ..., so one ring serves both
//   13    issues the products, owns TMEM
//   14    ahead of the others: an item's Q, its tables (positions, times,
//         who sees whom), and each step's window of position biases
//
// Bound by the cache's bytes up to about 64 queries, above that by the
// pointwise stage: two SFU operations and about fourteen others a pair.
#pragma once

#include "attn_cached.cuh"

namespace hstu {

constexpr int kTcKeys = 128;
constexpr int kTcPointWarps = 8;
constexpr int kTcThreads = (kTcPointWarps + 4 + 3) * 32;

// What an item's queries have in common with every step.
template <int NQ>
struct alignas(16) TcTables {
    int64_t tq[NQ];                     // timestamps
    int tqr[NQ];                        // behind the first, where that fits
    int qo[NQ];                         // 4 x position behind the tile's lowest
    float tb[64];                       // the head's time biases
    int64_t first;                      // tq[0]
    int lo, hi;                         // least and greatest of tqr
    int close;                          // all within 2^30 of the first
    int span;                           // greatest of qo / 4
    uint32_t odd[8];                    // new keys to be added alone (see below)
};

template <int D, int NQ>
struct CachedTcSmem {
    static constexpr int kSlotBytes = kTcKeys * D * 2;
    static constexpr int kSlots = D == 64 ? 6 : NQ == 64 ? 4 : 3;
    static constexpr int kPBytes = NQ / 64 * 16384;
    static constexpr int kQBytes = NQ * D * 2;
    // Steps whose timestamps are kept: they are read until P_i is written, and
    // K_i+4 (rings of up to four) or K_i+5 (of six) comes after that.
    static constexpr int kTcTimes = kSlots <= 4 ? 4 : 8;
    static constexpr int kWin = kTcKeys + kMaxTree;         // positions of a step
    static constexpr int kOffQ = kSlots * kSlotBytes;
    static constexpr int kOffP = kOffQ + kQBytes;
    static constexpr int kOffWin = kOffP + 2 * kPBytes;     // [step % 4][kWin]
    static constexpr int kOffTk = kOffWin + 4 * kWin * 4;   // [step % kTcTimes][128]
    static constexpr int kOffTab = kOffTk + kTcTimes * kTcKeys * 8;
    static constexpr int kOffTree = kOffTab + 2 * static_cast<int>(sizeof(TcTables<NQ>));
    static constexpr int kOffBar = kOffTree + 2 * static_cast<int>(sizeof(TreeSmem));
    static constexpr int kOffScratch = kOffBar + 64 * 8;
    static constexpr int kOffBad = kOffScratch + (kTcThreads / 32 + 9) * 8;   // [step % kTcTimes]
    static constexpr int kOffTmem = kOffBad + kTcTimes * 4;
    static constexpr int kOffAbort = kOffTmem + 8;
    static constexpr int kBytes = kOffAbort + 8;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory per block");
    static_assert(2 * kSlots + 35 <= 64, "barriers");
};

// Adds the keys of T.odd (new tokens whose values are not finite, cleared for
// the product) to the queries that see them, one by one, in the part's column d
// of a warp's lane; then, if `complete`, writes the output's column. Rare, so
// kept out of the kernel's registers.
template <int D, int NQ>
__device__ __noinline__ void add_odd_keys(const CachedArgs& a, const TcTables<NQ>& T,
                                          const TreeSmem& tree, int64_t row0, int ctx, int first_new,
                                          int q0, int rows, int h, int b, int d, float* part,
                                          bool complete) {
    const int lane = threadIdx.x & 31;
    const bool chain = a.parents == nullptr;
    const int64_t hd = static_cast<int64_t>(h) * D;
#pragma unroll 1
    for (int o = 0; o < kMaxTree; ++o) {
        if (!((T.odd[o >> 5] >> (o & 31)) & 1u)) continue;
        const int m = first_new + o, key = ctx + m;
        const int pg = a.table[static_cast<int64_t>(b) * a.table_stride + (key >> a.shift)];
        const int row = key & ((1 << a.shift) - 1);
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + pg * a.k_page + row * a.k_tok + hd;
        const float v = __bfloat162float(
            static_cast<const __nv_bfloat16*>(a.v)[pg * a.v_page + row * a.v_tok + hd + d]);
        const int pk = chain ? key : ctx + tree.depth[m];
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 32) {
            const int c = c0 + lane, qi = q0 + c;       // this lane's query
            const bool see =
                c < rows && (chain ? m <= qi : ((tree.seen[qi >> 5][m] >> (qi & 31)) & 1u) != 0u);
            float p = 0.f;
            if (see) {
                const __nv_bfloat16* q =
                    static_cast<const __nv_bfloat16*>(a.q) + (row0 + c) * a.q_stride + hd;
                float s = 0.f;
#pragma unroll 1
                for (int x = 0; x < D; ++x)
                    s = fmaf(__bfloat162float(q[x]), __bfloat162float(k[x]), s);
                if (a.pos)
                    s += a.pos[static_cast<int64_t>(h) * a.P +
                               min(ctx + first_new + T.qo[c] / 4 - pk, a.P - 1)];
                if (a.tsc) s += T.tb[time_bucket64(T.tq[c] - a.tsc[pg * a.tsc_page + row], 63)];
                p = silu_exp(s);
            }
            const uint32_t sees = __ballot_sync(0xffffffffu, see);
#pragma unroll 1
            for (int e = 0; e < 32 && c0 + e < rows; ++e) {
                const float pe = __shfl_sync(0xffffffffu, p, e);
                if ((sees >> e) & 1u) part[(c0 + e) * D] = fmaf(pe, v, part[(c0 + e) * D]);
            }
        }
    }
    if (!complete) return;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row0 * a.out_stride + hd + d;
#pragma unroll 1
    for (int c = 0; c < rows; ++c) out[c * a.out_stride] = __float2bfloat16(part[c * D] * a.inv_n);
}

template <int D, int NQ>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_cached_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CachedArgs a) {
    using S = CachedTcSmem<D, NQ>;
    using L = Line<kTcKeys, NQ>;
    constexpr int NS = S::kSlots, kTcTimes = S::kTcTimes;
    constexpr int kWarpOut = kTcPointWarps, kWarpKv = kWarpOut + 4, kWarpMma = kWarpKv + 1,
                  kWarpAhead = kWarpMma + 1;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps seeing shared memory)
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t* tks = reinterpret_cast<int64_t*>(smem + S::kOffTk);
    TcTables<NQ>* tabs = reinterpret_cast<TcTables<NQ>*>(smem + S::kOffTab);
    TreeSmem* trees = reinterpret_cast<TreeSmem*>(smem + S::kOffTree);
    uint32_t* bads = reinterpret_cast<uint32_t*>(smem + S::kOffBad);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    uint64_t* empty = full + NS;
    uint64_t* q_full = empty + NS;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;         // [2]
    uint64_t* p_full = s_full + 2;          // [2]
    uint64_t* p_empty = p_full + 2;         // [2]
    uint64_t* o_full = p_empty + 2;         // [2]
    uint64_t* o_empty = o_full + 2;         // [2]
    uint64_t* tab_full = o_empty + 2;       // [2]
    uint64_t* tab_empty = tab_full + 2;     // [2]
    uint64_t* point_done = tab_empty + 2;   // [2]
    uint64_t* win_full = point_done + 2;    // [4]
    uint64_t* win_empty = win_full + 4;     // [4]
    uint64_t* tk_full = win_empty + 4;      // [kTcTimes]
    uint64_t* drain = tk_full + kTcTimes;
    int64_t* scratch = reinterpret_cast<int64_t*>(smem + S::kOffScratch);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffTmem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffAbort);
    const bool use_pos = a.pos != nullptr, use_time = a.tsc != nullptr;
    const bool chain = a.parents == nullptr;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        *abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 128);
            mbar_init(&p_empty[s], 1);
            mbar_init(&o_full[s], 1);
            mbar_init(&o_empty[s], 4);
            mbar_init(&tab_full[s], 1);
            mbar_init(&tab_empty[s], 4);
            mbar_init(&point_done[s], kTcPointWarps);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&win_full[s], 32);
            mbar_init(&win_empty[s], 4);
        }
        for (int s = 0; s < kTcTimes; ++s) mbar_init(&tk_full[s], 33);
        mbar_init(drain, 1);
        mbar_fence_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    LineAt at;
    const int64_t total = L::template locate<kTcThreads>(a, blockIdx.x, gridDim.x, scratch, at,
                                                         blockIdx.x == 0);
    const int64_t begin = L::cut(total, blockIdx.x, gridDim.x);
    const int64_t steps = L::cut(total, blockIdx.x + 1, gridDim.x) - begin;
    if (tid == 0) write_head<kTcKeys, NQ>(a, at, total, begin);
    if (steps <= 0) return;
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: S at 0 and 128, O at 256 and 384

    // A walk over the block's items and steps, one for each use of them.
    struct Walk {
        LineAt at;
        int64_t left;           // steps from the item's first of this block on
        int take, j;            // the item's steps here, and how many are behind
        __device__ __forceinline__ void enter() {
            take = static_cast<int>(min(left, static_cast<int64_t>(L::tiles(at.s, at.qt) - at.j)));
            j = 0;
        }
        __device__ __forceinline__ void next_item(const CachedArgs& a) {
            left -= take;
            if (left <= 0) return;
            L::next_item(a, at);
            enter();
        }
        __device__ __forceinline__ void next(const CachedArgs& a) {
            if (++j == take) next_item(a);
        }
        __device__ __forceinline__ int q0() const { return at.qt * NQ; }
        __device__ __forceinline__ int rows() const { return min(NQ, at.s.n - at.qt * NQ); }
        __device__ __forceinline__ int len() const { return at.s.ctx + min(at.s.n, (at.qt + 1) * NQ); }
    };
    Walk w;
    w.at = at;
    w.left = steps;
    w.enter();

    // Position biases of a step: a window of the head's table by distance, from
    // the distance between the tile's lowest query and `origin` up. A key at
    // position pk finds that of a query x positions behind the lowest at entry
    // origin - pk + x. Where all keys are a tree's new tokens, origin is the
    // context's end: entries below zero, which may be read but lie inside this
    // block's shared memory, belong to pairs that are not seen.
    auto deep = [&](const LineAt& I, int k0) { return !chain && k0 >= I.s.ctx; };
    auto origin = [&](const LineAt& I, int k0) {
        return deep(I, k0) ? I.s.ctx : k0 + kTcKeys - 1;
    };

    if (warp == kWarpKv) {
        // ------------------------------------------------------------ K, V, timestamps
        Walk kw = w, vw = w;
        const int box_shift = min(7, a.shift), box = 1 << box_shift, boxes = kTcKeys >> box_shift;
        const int page_mask = (1 << a.shift) - 1;
        int64_t seq = 0;
        // this lane's page of the step; bad ones (and those behind the item's
        // tokens) are past the cache, where TMA reads zeros
        auto page_of = [&](const Walk& v, bool& bad) {
            const int key = (v.at.j + v.j) * kTcKeys + lane * box;
            int page = a.num_pages;
            bad = false;
            if (lane < boxes && key < v.len()) {
                page = __ldg(a.table + static_cast<int64_t>(v.at.b) * a.table_stride + (key >> a.shift));
                bad = page < 0 || page >= a.num_pages;
                if (bad) page = a.num_pages;
            }
            return page;
        };
        auto load = [&](const Walk& v, const CUtensorMap* tm, int page) {
            const int s = static_cast<int>(seq % NS);
            if (seq >= NS && !warp_wait(&empty[s], (seq / NS - 1) & 1, abort_flag)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], S::kSlotBytes);
            __syncwarp();
            if (lane < boxes) {
                uint8_t* dst = smem + s * S::kSlotBytes + lane * box * 128;
                const int row = ((v.at.j + v.j) * kTcKeys + lane * box) & page_mask;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(dst + c * 16384, tm, &full[s], v.at.h * D + 64 * c, row, page);
            }
            ++seq;
            return true;
        };
        // K_i and the timestamps of its keys
        int64_t ki = 0;
        auto load_k = [&](int page, bool bad) {
            if (!load(kw, &tmK, page)) return false;
            const int p = static_cast<int>(ki % kTcTimes);
            const uint32_t m = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) {
                if (m) raise_error(kErrBadInput);
                bads[p] = m;
                mbar_arrive(&tk_full[p]);
            }
            if (use_time) {
                const int k0 = (kw.at.j + kw.j) * kTcKeys, len = kw.len();
#pragma unroll
                for (int u = 0; u < kTcKeys / 32; ++u) {
                    const int r = lane + 32 * u;
                    const int pg = __shfl_sync(0xffffffffu, page, r >> box_shift);
                    if (k0 + r < len && pg < a.num_pages)
                        cp_async8(tks + p * kTcKeys + r,
                                  a.tsc + pg * a.tsc_page + ((k0 + r) & page_mask));
                }
            }
            cp_async_arrive(&tk_full[p]);
            ++ki;
            kw.next(a);
            return true;
        };
        // pages are looked up a step ahead of their loads
        bool bad;
        int page = page_of(kw, bad);
        int vpage = page;
        bool ok = load_k(page, bad);
        for (int64_t i = 0; ok && i < steps; ++i) {
            const bool more = i + 1 < steps;
            if (more) {
                page = page_of(kw, bad);
                ok = load_k(page, bad);
            }
            if (ok) ok = load(vw, &tmV, vpage);
            vw.next(a);
            vpage = page;
        }
        // every copy has landed before the block ends
        for (int s = 0; s < NS; ++s) {
            const int64_t c = seq > s ? (seq - s + NS - 1) / NS : 0;
            if (c > 0 && !warp_wait(&full[s], (c - 1) & 1, nullptr) && lane == 0)
                raise_error(kErrTimeout);
        }
        cp_async_wait_all();
    } else if (warp == kWarpAhead) {
        // ------------------------------------------------------------ Q, tables, windows
        int it = 0, tree_of = -1, tree_at = 1;
        int64_t i = 0;
        bool ok = true;
        auto load_q = [&]() {
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, S::kQBytes);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_2d(smem + S::kOffQ + c * NQ * 128, &tmQ, q_full, w.at.h * D + 64 * c,
                                static_cast<int>(w.at.s.off) + w.q0());
            }
        };
        load_q();
        while (w.left > 0) {
            const LineAt& I = w.at;
            const int q0 = w.q0(), rows = w.rows();
            TcTables<NQ>& T = tabs[it & 1];
            ok = it < 2 || warp_wait(&tab_empty[it & 1], (it / 2 - 1) & 1, abort_flag);
            if (!ok) break;
            if (!chain && tree_of != I.b) {
                // the place holds the tree before the last, whose items are done
                tree_at ^= 1;
                build_tree(a, I.s, trees[tree_at], lane, 32, [] { __syncwarp(); });
                tree_of = I.b;
            }
            const int64_t* tsq = a.ts + I.s.off + q0;
            const int64_t first = use_time ? __ldg(tsq) : 0;
            const int64_t lim = int64_t{1} << 30;
            bool close = true;
            int lo = 0, hi = 0;
            for (int c = lane; c < NQ; c += 32) {
                const int m = min(c, rows - 1);
                const int64_t t = use_time ? __ldg(tsq + m) : 0;
                const int d = static_cast<int>(t - first);
                close = close && t - first < lim && first - t < lim;
                lo = min(lo, d);
                hi = max(hi, d);
                T.tq[c] = t;
                T.tqr[c] = d;
                T.qo[c] = 4 * (chain ? m : trees[tree_at].depth[q0 + m]);
            }
            if (use_time) {
                const float* tb = a.tb + static_cast<int64_t>(I.h) * a.NB;
                T.tb[lane] = __ldg(tb + min(lane, a.NB - 1));
                T.tb[lane + 32] = __ldg(tb + min(lane + 32, a.NB - 1));
            }
            if (lane < 8) T.odd[lane] = 0u;
            close = __all_sync(0xffffffffu, close);
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            const int span = chain ? rows - 1 : trees[tree_at].deepest;
            if (lane == 0) {
                T.first = first;
                T.lo = lo;
                T.hi = hi;
                T.close = close;
                T.span = span;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_full[it & 1]);
            if (it > 0) {
                ok = warp_wait(q_empty, (it - 1) & 1, abort_flag);
                if (!ok) break;
                load_q();
            }
            ++it;
            const float* posh = use_pos ? a.pos + static_cast<int64_t>(I.h) * a.P : nullptr;
            for (int j = 0; j < w.take; ++j, ++i) {
                const int b = static_cast<int>(i & 3);
                ok = i < 4 || warp_wait(&win_empty[b], (i / 4 - 1) & 1, abort_flag);
                if (!ok) break;
                if (use_pos) {
                    float* win = reinterpret_cast<float*>(smem + S::kOffWin) + b * S::kWin;
                    const int k0 = (I.j + j) * kTcKeys;
                    const int least = I.s.ctx + (chain ? q0 : 0) - origin(I, k0);
                    const int n = (deep(I, k0) ? 1 : kTcKeys) + span;
                    for (int x = lane; x < n; x += 32)
                        cp_async4(win + x, posh + max(0, min(least + x, a.P - 1)));
                }
                cp_async_arrive(&win_full[b]);
            }
            if (!ok) break;
            w.next_item(a);
        }
        // (Q loads: one before the walk, then one an item)
        if (!warp_wait(q_full, (max(it, 1) - 1) & 1, nullptr) && lane == 0) raise_error(kErrTimeout);
        cp_async_wait_all();
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            Walk sw = w, ow = w;
            int sit = 0, oit = 0;           // items
            bool ok = true;
            const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + S::kOffQ));
            const uint64_t dk0 = desc_kmajor_sw128(smem_u32(smem));
            const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(smem), D == 64 ? 0 : 16384);
            const uint64_t dp0 = desc_mnmajor_sw128(smem_u32(smem + S::kOffP), 16384);
            auto columns = [](const Walk& v) { return (v.rows() + 15) / 16 * 16; };
            auto scores = [&](int64_t i) {
                const int64_t seq = i == 0 ? 0 : 2 * i - 1;
                const int s = static_cast<int>(seq % NS);
                if ((sw.j == 0 && !mbar_wait(q_full, sit & 1, abort_flag)) ||
                    !mbar_wait(&full[s], (seq / NS) & 1, abort_flag))
                    return false;
                tc_fence_after();
                const uint32_t idesc = idesc_bf16_f32(128, columns(sw), 0, 0);
                const uint64_t dk = dk0 + static_cast<uint64_t>(s * (S::kSlotBytes >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_ss(tmem + (i & 1) * 128,
                                 dk + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                 dq + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idesc,
                                 kk > 0 ? 1u : 0u);
                umma_commit(&s_full[i & 1]);
                umma_commit(&empty[s]);
                if (sw.j == sw.take - 1) {
                    umma_commit(q_empty);
                    ++sit;
                }
                sw.next(a);
                return true;
            };
            auto values = [&](int64_t i) {
                const int64_t seq = i + 1 < steps ? 2 * i + 2 : 2 * i + 1;
                const int s = static_cast<int>(seq % NS);
                if (!mbar_wait(&full[s], (seq / NS) & 1, abort_flag) ||
                    (ow.j == 0 && oit >= 2 &&
                     !mbar_wait(&o_empty[oit & 1], (oit / 2 - 1) & 1, abort_flag)) ||
                    !mbar_wait(&p_full[i & 1], (i >> 1) & 1, abort_flag))
                    return false;
                tc_fence_after();
                const uint32_t idesc = idesc_bf16_f32(128, columns(ow), 1, 1);
                const uint64_t dv = dv0 + static_cast<uint64_t>(s * (S::kSlotBytes >> 4));
                const uint64_t dp = dp0 + static_cast<uint64_t>((i & 1) * (S::kPBytes >> 4));
                const uint32_t dst = tmem + 256 + (oit & 1) * 128;
#pragma unroll
                for (int kk = 0; kk < kTcKeys / 16; ++kk)
                    umma_bf16_ss(dst, dv + ((kk * 2048) >> 4), dp + ((kk * 2048) >> 4), idesc,
                                 ow.j > 0 || kk > 0 ? 1u : 0u);
                umma_commit(&empty[s]);
                umma_commit(&p_empty[i & 1]);
                if (ow.j == ow.take - 1) {
                    umma_commit(&o_full[oit & 1]);
                    ++oit;
                }
                ow.next(a);
                return true;
            };
            ok = scores(0);
            if (ok && steps > 1) ok = scores(1);
            for (int64_t i = 0; ok && i < steps; ++i) {
                ok = values(i);
                // the group that wrote P_i has read S_i
                if (ok && i + 2 < steps) ok = scores(i + 2);
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0, nullptr)) raise_error(kErrTimeout);
        }
        __syncwarp();
    } else if (warp < kTcPointWarps) {
        // ------------------------------------------------------------ pointwise stage
        const int grp = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;              // the step's key
        const uint32_t s_col = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + grp * 128;
        const uint32_t prow = smem_u32(smem + S::kOffP + grp * S::kPBytes) + r * 128;
        const int box_shift = min(7, a.shift);
        int64_t i = 0;                                  // step of the block
        int it = 0, tree_of = -1, tree_at = 1;
        bool ok = true;
        while (ok && w.left > 0) {
            const LineAt& I = w.at;
            const int q0 = w.q0(), len = w.len(), nc = (w.rows() + 15) / 16 * 16;
            if (!chain && tree_of != I.b) {
                tree_at ^= 1;
                tree_of = I.b;
            }
            const TreeSmem& tree = trees[tree_at];
            TcTables<NQ>& T = tabs[it & 1];
            ok = warp_wait(&tab_full[it & 1], (it >> 1) & 1, abort_flag);
            if (!ok) break;
            const int64_t first = T.first, lim = int64_t{1} << 30;
            const int t_lo = T.lo, t_hi = T.hi, span = T.span;
            const bool close = T.close;
            // keys from here on are seen by some queries and not by others
            const int part0 = I.s.ctx + (chain ? q0 : 0);
            for (int j = (i & 1) == grp ? 0 : 1; j < w.take; j += 2) {
                const int64_t st = i + j;
                const int k0 = (I.j + j) * kTcKeys, key = k0 + r;
                const int m = key - I.s.ctx;            // new token's index, < 0: cached
                const int tp = static_cast<int>(st % kTcTimes), wb = static_cast<int>(st & 3);
                ok = warp_wait(&tk_full[tp], (st / kTcTimes) & 1, abort_flag) &&
                     warp_wait(&win_full[wb], (st >> 2) & 1, abort_flag);
                if (!ok) break;
                const bool paged = key < len && !((bads[tp] >> (r >> box_shift)) & 1u);
                const int64_t tk = use_time && paged ? tks[tp * kTcKeys + r] : first;
                const int pk = m < 0 || chain ? key : I.s.ctx + (m < I.s.n ? tree.depth[m] : 0);
                const float* wr = reinterpret_cast<const float*>(smem + S::kOffWin) + wb * S::kWin +
                                  (origin(I, k0) - pk);
                const bool near = __all_sync(0xffffffffu, close && first - tk < lim && tk - first < lim);
                // Most keys are far from the new tokens: all queries fall into one
                // or two buckets, and one comparison replaces the table.
                const int tkr = static_cast<int>(tk - first);
                const uint32_t b_lo = bucket_bytes(t_lo - tkr), b_hi = bucket_bytes(t_hi - tkr);
                const bool two = near && __all_sync(0xffffffffu, b_hi - b_lo <= 4u);
                float add_lo = 0.f, add_hi = 0.f;
                int turn = 0;                           // first relative time of the upper bucket
                if (two && use_time) {
                    add_lo = table_at(T.tb, b_lo - kBucketBias);
                    add_hi = table_at(T.tb, b_hi - kBucketBias);
                    if (b_hi != b_lo) turn = tkr + (1 << ((b_hi - kBucketBias) >> 2));
                }
                if (use_pos && span == 0) {             // candidates side by side
                    add_lo += wr[0];
                    add_hi += wr[0];
                }
                ok = warp_wait(&s_full[grp], (st >> 1) & 1, abort_flag) &&
                     (st < 2 || warp_wait(&p_empty[grp], ((st >> 1) - 1) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const bool fast = k0 + kTcKeys <= part0;
#pragma unroll 1
                for (int c0 = 0; c0 < nc; c0 += 16) {
                    uint32_t sv[16];
                    tmem_ld16(s_col + c0, sv);
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(sv[e]);
                    // (entries behind the last query's belong to columns nobody reads)
                    if (use_pos && span > 0) {
                        if (chain) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] += wr[c0 + e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 qo = *reinterpret_cast<const int4*>(T.qo + c0 + e);
                                x[e] += table_at(wr, qo.x);
                                x[e + 1] += table_at(wr, qo.y);
                                x[e + 2] += table_at(wr, qo.z);
                                x[e + 3] += table_at(wr, qo.w);
                            }
                        }
                    }
                    if (two) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const int4 tq = *reinterpret_cast<const int4*>(T.tqr + c0 + e);
                            x[e] += tq.x >= turn ? add_hi : add_lo;
                            x[e + 1] += tq.y >= turn ? add_hi : add_lo;
                            x[e + 2] += tq.z >= turn ? add_hi : add_lo;
                            x[e + 3] += tq.w >= turn ? add_hi : add_lo;
                        }
                    } else {
                        if (near) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 tq = *reinterpret_cast<const int4*>(T.tqr + c0 + e);
                                x[e] += table_at(T.tb, bucket_bytes(tq.x - tkr) - kBucketBias);
                                x[e + 1] += table_at(T.tb, bucket_bytes(tq.y - tkr) - kBucketBias);
                                x[e + 2] += table_at(T.tb, bucket_bytes(tq.z - tkr) - kBucketBias);
                                x[e + 3] += table_at(T.tb, bucket_bytes(tq.w - tkr) - kBucketBias);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[e] += T.tb[time_bucket64(T.tq[c0 + e] - tk, 63)];
                        }
                        if (use_pos && span == 0) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] += wr[0];
                        }
                    }
                    uint32_t seen = 0xffffu;
                    if (!fast) {
                        if (m >= I.s.n) seen = 0u;
                        else if (m >= 0) {
                            const int d = m - q0 - c0;      // chain: the first query that sees the key
                            seen = chain ? (d <= 0 ? 0xffffu : d < 16 ? 0xffffu << d : 0u)
                                         : tree.seen[(q0 + c0) >> 5][m] >> (c0 & 16);
                        }
                    }
                    if (!paged) seen = 0u;
                    uint32_t pk2[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        pk2[e] = pack_bf16x2(silu_exp(x[2 * e]), silu_exp(x[2 * e + 1]));
                    if ((seen & 0xffffu) != 0xffffu) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            pk2[e] &= ((seen >> (2 * e)) & 1u) * 0xffffu |
                                      ((seen >> (2 * e + 1)) & 1u) * 0xffff0000u;
                    }
                    // 64 queries a 128-byte row, 16-byte pieces in the 128-byte swizzle
                    const uint32_t base = prow + (c0 >> 6) * 16384;
                    const int c = (c0 & 63) >> 3;
                    st_shared_v4(base + ((c ^ (r & 7)) << 4), pk2[0], pk2[1], pk2[2], pk2[3]);
                    st_shared_v4(base + (((c + 1) ^ (r & 7)) << 4), pk2[4], pk2[5], pk2[6], pk2[7]);
                }
                if (!fast) {
                    // V rows that some query does not see meet zeros in P, so they
                    // have to be finite: rows behind the sequence and rows of new
                    // tokens that are not finite become zeros, and the latter are
                    // added alone to the queries that see them.
                    const int64_t seq = st + 1 < steps ? 2 * st + 2 : 2 * st + 1;
                    const int s = static_cast<int>(seq % NS);
                    ok = warp_wait(&full[s], (seq / NS) & 1, abort_flag);
                    if (!ok) break;
                    uint8_t* vr = smem + s * S::kSlotBytes + r * 128;
                    bool clear = key >= len;
                    if (key >= part0 && key < len) {
                        bool bad = false;
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4*>(
                                vr + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4));
                            const uint32_t f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                bad = bad || (f[e] & 0x7f80u) == 0x7f80u ||
                                      (f[e] & 0x7f800000u) == 0x7f800000u;
                        }
                        if (bad) {
                            const int o = key - part0;      // < 256: a tile's chain or a tree
                            atomicOr(&T.odd[o >> 5], 1u << (o & 31));
                            clear = true;
                        }
                    }
                    if (clear) {
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(vr + (c >> 3) * 16384 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[grp]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&win_empty[wb]);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&point_done[it & 1]);
            i += w.take;
            ++it;
            w.next_item(a);
        }
    } else {
        // ------------------------------------------------------------ the items' rows
        const int quarter = warp & 3;
        const int d = quarter * 32 + lane;              // column of the output, TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        int it = 0, tree_of = -1, tree_at = 1;
        while (w.left > 0) {
            const LineAt& I = w.at;
            const int q0 = w.q0(), rows = w.rows();
            if (!chain && tree_of != I.b) {
                tree_at ^= 1;
                tree_of = I.b;
            }
            const TreeSmem& tree = trees[tree_at];
            const TcTables<NQ>& T = tabs[it & 1];
            if (!warp_wait(&point_done[it & 1], (it >> 1) & 1, abort_flag) ||
                !warp_wait(&o_full[it & 1], (it >> 1) & 1, abort_flag))
                break;
            tc_fence_after();
            uint32_t any_odd = 0u;
#pragma unroll
            for (int o = 0; o < 8; ++o) any_odd |= T.odd[o];
            // (with odd keys the rows go through the block's part, whole or not)
            const bool complete = w.take == L::tiles(I.s, I.qt), whole = complete && !any_odd;
            float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (it == 0 ? 0 : 1)) * NQ * D + d;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (I.s.off + q0) * a.out_stride +
                                 static_cast<int64_t>(I.h) * D + (d & ~1);
#pragma unroll 1
            for (int c0 = 0; c0 < rows && quarter * 32 < D; c0 += 32) {
                uint32_t ov[32];
                tmem_ld32(tmem + 256 + (it & 1) * 128 + lane_base + c0, ov);
                if (whole) {
                    // even lanes write columns d, d + 1 of query e, odd ones of e + 1
                    const bool odd_lane = lane & 1;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float x0 = __uint_as_float(ov[e]) * a.inv_n;
                        const float x1 = __uint_as_float(ov[e + 1]) * a.inv_n;
                        const float other = __shfl_xor_sync(0xffffffffu, odd_lane ? x0 : x1, 1);
                        const int c = c0 + e + (odd_lane ? 1 : 0);
                        if (c < rows)
                            *reinterpret_cast<uint32_t*>(out + c * a.out_stride) =
                                odd_lane ? pack_bf16x2(other, x1) : pack_bf16x2(x0, other);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c0 + e < rows) part[(c0 + e) * D] = __uint_as_float(ov[e]);
                }
            }
            if (any_odd && quarter * 32 < D)
                add_odd_keys<D, NQ>(a, T, tree, I.s.off + q0, I.s.ctx, chain ? q0 : 0, q0, rows, I.h, I.b,
                                    d, part, complete);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&o_empty[it & 1]);
                mbar_arrive(&tab_empty[it & 1]);
            }
            ++it;
            w.next_item(a);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) raise_error(kErrTimeout);
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace hstu
