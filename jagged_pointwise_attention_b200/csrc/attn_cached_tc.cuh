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
//   12    K by TMA, a page (or 128 tokens of one) a box, a lane a page, and
//         the keys' timestamps
//   13    V, likewise
//   14    issues the first products, owns TMEM
//   15    issues the second products (an issuer that waits for one product's
//         operands would hold up the other's)
//   16    the walk along the line: publishes the items in a ring
//   17    an item's Q and its tables (positions, times, who sees whom)
//   18    each step's window of position biases
// A load takes 2.5 to 3 us while HBM is busy, so nothing asks for its data when
// it needs it. All roles run at once, so what they run together has to stay in the
// instruction cache: loops are short, waits are out of line, and only one role
// knows how to walk the line. (82 KB of code, of which about a third runs in the
// steady state; at 122 KB instruction fetches were the bound, and the 64-token
// trees took 86 us when this brought them to 62.)
//
// Bound by the cache's bytes and a launch's start for few queries. From about 64
// on by latency in the pointwise stage: no unit is full (64-token trees, heads of
// 128: SFU 21%, issue slots 40%, tensor pipe 10%; 128 tokens, heads of 64: 32, 47
// and 11%), but the TMEM load, table reads, exp2, reciprocal, pack and store of
// eight queries follow one another, in two warps a scheduler. 32 sequences of 256
// to 4096 tokens with the join, 4 heads of 128 (8 of 64): 8 new tokens 42 us (47),
// 32 44 (53), 64 53 (78), 128 89 (136), against 23 us for the bytes (150 MB)
// alone. One token over 16 sequences of up to 8192: 43 us (180 MB, 4.2 TB/s). A
// launch has found its line after 3 us and issues the first product at 7 to 8; a
// tree's first weights come at 12, since one warp builds an item's tree for its
// tables (ready at 11). The join takes 3 to 5. Sixteen pointwise warps gained a
// tenth at 128 queries and lost 2% at one; the approximate tanh would save one of
// the two SFU operations and miss silu's bf16 step.
//
// P is rounded to bf16, the type that a product with a bf16 V takes: at most 2^-8
// of a weight, like the dense forward. Outputs are then 0.0023 to 0.0024 (relative,
// root mean square) from the 64-bit ones, of which their own rounding is 0.0017.
// Two bf16 terms a weight would keep it, for twice the second product and twice
// P's stores in the stage that is the bound.
#pragma once

#include "attn_cached.cuh"

namespace hstu {

constexpr int kTcKeys = 128;
constexpr int kTcPointWarps = 8;
constexpr int kTcThreads = (kTcPointWarps + 4 + 7) * 32;
constexpr int kTcItems = 8;             // ring of published items
// What an item's end costs a block, in steps (64-token trees 59 us with none, 54
// with one, 53 with two and three; 128 new tokens 99, 93, 89, 88).
constexpr int kTcEnd = 2;

// An item of the block's part of the line.
struct alignas(8) TcItem {
    int64_t row0;                       // first row of q and out
    int32_t b, h, ctx, n, q0;           // q0: first query, among the new tokens
    int32_t tile, take;                 // first key tile, how many are this block's (0: the end)
    int32_t whole;                      // the block has all of them
};

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

// Who sees whom among a sequence's new tokens, for the tile's queries.
template <int NQ>
struct alignas(16) TcTree {
    uint32_t seen[NQ / 32][kMaxTree];   // [query / 32][key]: bit of the query
    uint8_t depth[kMaxTree];
    int deepest;                        // greatest depth
};

// Built by one warp; `parent` is its scratch.
template <int NQ>
__device__ __forceinline__ void build_tile_tree(const int32_t* parents, int n, int q0,
                                                TcTree<NQ>& tree, int16_t* parent) {
    const int lane = threadIdx.x & 31;
    for (int m = lane; m < n; m += 32) {
        const int p = __ldg(parents + m);
        const bool ok = p >= -1 && p < m;
        if (!ok) raise_error(kErrBadInput);
        parent[m] = static_cast<int16_t>(ok ? p : -1);
#pragma unroll
        for (int w = 0; w < NQ / 32; ++w) tree.seen[w][m] = 0u;
    }
    __syncwarp();
    int deepest = 0;
    for (int m = lane; m < n; m += 32) {
        const int q = m - q0;
        const bool mine = q >= 0 && q < NQ;
        int d = -1;
        for (int p = m; p >= 0; p = parent[p]) {    // parents are smaller: ends
            if (mine) atomicOr(&tree.seen[q >> 5][p], 1u << (q & 31));
            ++d;
        }
        tree.depth[m] = static_cast<uint8_t>(d);
        deepest = max(deepest, d);
    }
    deepest = __reduce_max_sync(0xffffffffu, deepest);
    if (lane == 0) tree.deepest = deepest;
    __syncwarp();
}

template <int D, int NQ>
struct CachedTcSmem {
    static constexpr int kSlotBytes = kTcKeys * D * 2;
    // Rings: a K tile is held from its load to its product, a V tile until P is there.
    static constexpr int kK = D == 64 ? 3 : NQ == 64 ? 2 : 1, kV = D == 64 || NQ == 64 ? 3 : 2;
    static constexpr int kPBytes = NQ / 64 * 16384;
    static constexpr int kQBytes = NQ * D * 2;
    // Steps whose timestamps are kept: they are read until P_i is written, and
    // K_i+kK+2 comes after that.
    static constexpr int kTimes = kK + 2 <= 4 ? 4 : 8;
    static constexpr int kWin = kTcKeys + kMaxTree;         // positions of a step
    static constexpr int kOffV = kK * kSlotBytes;
    static constexpr int kOffQ = kOffV + kV * kSlotBytes;
    static constexpr int kOffP = kOffQ + kQBytes;
    static constexpr int kOffWin = kOffP + 2 * kPBytes;     // [step % 4][kWin]
    static constexpr int kOffTk = kOffWin + 4 * kWin * 4;   // [step % kTimes][128]
    static constexpr int kOffTab = kOffTk + kTimes * kTcKeys * 8;
    static constexpr int kOffTree = kOffTab + 2 * static_cast<int>(sizeof(TcTables<NQ>));
    static constexpr int kOffItems = kOffTree + 2 * static_cast<int>(sizeof(TcTree<NQ>)) + 2 * kMaxTree;
    static constexpr int kOffBar = kOffItems + kTcItems * static_cast<int>(sizeof(TcItem));
    static constexpr int kBars = 2 * (kK + kV) + 38 + kTimes + 2 * kTcItems;
    static constexpr int kOffBad = kOffBar + kBars * 8;     // [step % kTimes]
    static constexpr int kOffTmem = kOffBad + kTimes * 4;
    static constexpr int kOffAbort = kOffTmem + 8;
    static constexpr int kAlloc = kOffAbort + 8;
    static_assert(kAlloc <= 227 * 1024, "shared memory per block");
};

// Adds the keys of T.odd (new tokens whose values are not finite, cleared for
// the product) to the queries that see them, one by one, in the part's column d
// of a warp's lane; then, if `complete`, writes the output's column. Rare, so
// kept out of the kernel's registers.
template <int D, int NQ>
__device__ __noinline__ void add_odd_keys(const CachedArgs& a, const TcTables<NQ>& T,
                                          const TcTree<NQ>& tree, int64_t row0, int ctx, int first_new,
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
        const float v = __bfloat162float(
            static_cast<const __nv_bfloat16*>(a.v)[pg * a.v_page + row * a.v_tok + hd + d]);
        const int pk = chain ? key : ctx + tree.depth[m];
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 32) {
            const int c = c0 + lane, qi = q0 + c;       // this lane's query
            const bool see =
                c < rows && (chain ? m <= qi : ((tree.seen[c >> 5][m] >> (c & 31)) & 1u) != 0u);
            float p = 0.f;
            if (see)
                p = odd_weight<D>(a, h, row0 + c, ctx + first_new + T.qo[c] / 4, pg, row, pk);
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

// Index and phase of a ring's place.
template <int N>
struct TcPlace {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            phase ^= 1u;
        }
    }
};

template <int D, int NQ>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_cached_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CachedArgs a) {
    using S = CachedTcSmem<D, NQ>;
    using L = Line<kTcKeys, NQ, kTcEnd>;
    constexpr int NK = S::kK, NV = S::kV, NT = S::kTimes;
    constexpr int kWarpOut = kTcPointWarps, kWarpK = kWarpOut + 4, kWarpV = kWarpK + 1,
                  kWarpS = kWarpV + 1, kWarpO = kWarpS + 1, kWarpWalk = kWarpO + 1,
                  kWarpTab = kWarpWalk + 1, kWarpWin = kWarpTab + 1;
    static_assert((kWarpWin + 1) * 32 == kTcThreads, "warp roles");
    extern __shared__ __align__(1024) uint8_t cached_tc_smem[];
    uint8_t* smem = cached_tc_smem;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t* tks = reinterpret_cast<int64_t*>(smem + S::kOffTk);
    TcTables<NQ>* tabs = reinterpret_cast<TcTables<NQ>*>(smem + S::kOffTab);
    TcTree<NQ>* trees = reinterpret_cast<TcTree<NQ>*>(smem + S::kOffTree);
    TcItem* items = reinterpret_cast<TcItem*>(smem + S::kOffItems);
    uint32_t* bads = reinterpret_cast<uint32_t*>(smem + S::kOffBad);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    uint64_t* k_empty = k_full + NK;
    uint64_t* v_full = k_empty + NK;
    uint64_t* v_empty = v_full + NV;
    uint64_t* q_full = v_empty + NV;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;         // [2]
    uint64_t* s_empty = s_full + 2;         // [2]
    uint64_t* p_full = s_empty + 2;         // [2]
    uint64_t* p_empty = p_full + 2;         // [2]
    uint64_t* o_full = p_empty + 2;         // [2]
    uint64_t* o_empty = o_full + 2;         // [2]
    uint64_t* tab_full = o_empty + 2;       // [2]
    uint64_t* tab_empty = tab_full + 2;     // [2]
    uint64_t* point_done = tab_empty + 2;   // [2]
    uint64_t* drain = point_done + 2;       // [2]
    uint64_t* v_loading = drain + 2;        // [4]: steps whose V is looked at
    uint64_t* v_clean = v_loading + 4;      // [4]
    uint64_t* win_full = v_clean + 4;       // [4]
    uint64_t* win_empty = win_full + 4;     // [4]
    uint64_t* tk_full = win_empty + 4;      // [NT]
    uint64_t* item_full = tk_full + NT;     // [kTcItems]
    uint64_t* item_empty = item_full + kTcItems;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffTmem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffAbort);
    const bool use_pos = a.pos != nullptr, use_time = a.tsc != nullptr;
    const bool chain = a.parents == nullptr;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Barriers: how many arrivals each expects.
    for (int x = tid; x < S::kBars; x += kTcThreads) {     // (the last is item_empty[kTcItems - 1])
        uint64_t* bar = k_full + x;
        int count = 1;
        if (bar >= item_empty || (bar >= s_empty && bar < s_empty + 2) ||
            (bar >= o_empty && bar < o_empty + 2) || (bar >= tab_empty && bar < tab_empty + 2) ||
            (bar >= win_empty && bar < win_empty + 4))
            count = 4;                      // a warp of the pointwise group or of the rows each
        else if (bar >= p_full && bar < p_full + 2) count = 128;
        else if (bar >= v_clean && bar < v_clean + 4) count = 128;
        else if (bar >= point_done && bar < point_done + 2) count = kTcPointWarps;
        else if (bar >= win_full && bar < win_full + 4) count = 32;
        else if (bar >= tk_full && bar < tk_full + NT) count = 33;
        mbar_init(bar, count);
    }
    mbar_fence_init();
    if (tid == 0) {
        *abort_flag = 0;
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    LineAt at;
    const int64_t total = L::template locate<kTcThreads>(
        a, blockIdx.x, gridDim.x, reinterpret_cast<int64_t*>(smem + S::kOffWin), at, blockIdx.x == 0);
    const int64_t begin = L::cut(total, blockIdx.x, gridDim.x);
    int64_t left = L::cut(total, blockIdx.x + 1, gridDim.x) - begin;    // of the block's part
    if (tid == 0) write_head<kTcKeys, NQ, kTcEnd>(a, at, total, begin);
    if (left > INT32_MAX) {                 // days of work
        if (tid == 0) raise_error(kErrBadInput);
        return;
    }
    if (left > 0 && at.j >= L::tiles(at.s, at.qt)) {    // it begins behind an item's tiles
        left -= L::tiles(at.s, at.qt) + kTcEnd - at.j;
        if (left > 0) L::next_item(a, at);
    }
    if (left <= 0) return;
    if (warp == kWarpS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: S at 0 and 128, O at 256 and 384

    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait_far(bar, parity, abort_flag); };
    auto item_rows = [&](const TcItem& I) { return min(NQ, I.n - I.q0); };
    auto item_len = [&](const TcItem& I) { return I.ctx + min(I.n, I.q0 + NQ); };
    // keys from here on are seen by some queries and not by others
    auto item_part0 = [&](const TcItem& I) { return I.ctx + (chain ? I.q0 : 0); };
    // Position biases of a step: a window of the head's table by distance, from
    // the distance between the tile's lowest query and `origin` up. A key at
    // position pk finds that of a query x positions behind the lowest at entry
    // origin - pk + x. Where all keys are a tree's new tokens, origin is the
    // context's end: entries below zero, which may be read but lie inside this
    // block's shared memory, belong to pairs that are not seen.
    auto deep = [&](const TcItem& I, int k0) { return !chain && k0 >= I.ctx; };
    auto origin = [&](const TcItem& I, int k0) { return deep(I, k0) ? I.ctx : k0 + kTcKeys - 1; };
    TcPlace<kTcItems> ip;                   // the role's item

    if (warp == kWarpWalk) {
        // ------------------------------------------------------------ the walk
        for (int n = 0;; ++n) {
            if (n >= kTcItems && !wait(&item_empty[ip.s], ip.phase ^ 1u)) break;
            const int nt = left > 0 ? L::tiles(at.s, at.qt) : 0;
            const int take = static_cast<int>(min(left, static_cast<int64_t>(nt - at.j)));
            if (lane == 0) {
                TcItem& I = items[ip.s];
                I.row0 = at.s.off + at.qt * NQ;
                I.b = at.b;
                I.h = at.h;
                I.ctx = at.s.ctx;
                I.n = at.s.n;
                I.q0 = at.qt * NQ;
                I.tile = at.j;
                I.take = take;
                I.whole = take == nt;
                mbar_arrive(&item_full[ip.s]);
            }
            if (take == 0) break;           // the end: nothing is left
            ip.next();
            left -= take + kTcEnd;
            if (left > 0) L::next_item(a, at);
            else left = at.j = 0;
        }
    } else if (warp == kWarpK || warp == kWarpV) {
        // ------------------------------------------------------------ K (and timestamps), V
        const bool is_k = warp == kWarpK;
        const CUtensorMap* tm = is_k ? &tmK : &tmV;
        uint64_t *fulls = is_k ? k_full : v_full, *empties = is_k ? k_empty : v_empty;
        const int ring = is_k ? NK : NV;
        uint8_t* base = smem + (is_k ? 0 : S::kOffV);
        const int box_shift = min(7, a.shift), boxes = kTcKeys >> box_shift;
        const int page_mask = (1 << a.shift) - 1;
        int slot = 0, loads = 0, tail = 0;
        uint32_t phase = 1;                 // of the slot's last use: none is waited for at first
        TcPlace<NT> tp;
        bool ok = true;
        while (ok) {
            ok = wait(&item_full[ip.s], ip.phase);
            if (!ok || items[ip.s].take == 0) break;
            const TcItem& I = items[ip.s];
            const int take = I.take, len = item_len(I), x0 = I.h * D, part0 = item_part0(I);
            const int32_t* table = a.table + static_cast<int64_t>(I.b) * a.table_stride;
            // Pages of a step, one a lane, looked up a step ahead; bad ones (and
            // those behind the item's tokens) are past the cache: TMA reads zeros.
            int k0 = I.tile * kTcKeys;
            auto look = [&](int key) {
                return lane < boxes && key < len ? __ldg(table + (key >> a.shift)) : a.num_pages;
            };
            int ahead = look(k0 + (lane << box_shift));
            for (int j = 0; j < take; ++j, k0 += kTcKeys) {
                const int key = k0 + (lane << box_shift);
                const bool bad = (ahead < 0 || ahead >= a.num_pages) && lane < boxes && key < len;
                const int page = bad ? a.num_pages : ahead;
                if (j + 1 < take) ahead = look(key + kTcKeys);
                if (loads >= ring) ok = wait(&empties[slot], phase);
                if (!ok) break;
                uint64_t* bar = &fulls[slot];
                if (lane == 0) mbar_arrive_expect_tx(bar, S::kSlotBytes);
                __syncwarp();
                if (lane < boxes) {
                    uint8_t* dst = base + slot * S::kSlotBytes + (lane << box_shift) * 128;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(dst + c * 16384, tm, bar, x0 + 64 * c, key & page_mask, page);
                }
                if (++slot == ring) {
                    slot = 0;
                    phase ^= 1u;
                }
                ++loads;
                if (is_k) {
                    const uint32_t m = __ballot_sync(0xffffffffu, bad);
                    if (lane == 0) {
                        if (m) raise_error(kErrBadInput);
                        bads[tp.s] = m;
                        mbar_arrive(&tk_full[tp.s]);
                    }
                    if (use_time) {
#pragma unroll 1
                        for (int r = lane; r < kTcKeys; r += 32) {
                            const int pg = __shfl_sync(0xffffffffu, page, r >> box_shift);
                            if (k0 + r < len && pg < a.num_pages)
                                cp_async8(tks + tp.s * kTcKeys + r,
                                          a.tsc + pg * a.tsc_page + ((k0 + r) & page_mask));
                        }
                    }
                    cp_async_arrive(&tk_full[tp.s]);
                    tp.next();
                } else if (k0 + kTcKeys > part0) {
                    if (lane == 0) mbar_arrive(&v_loading[tail & 3]);
                    ++tail;
                }
            }
            ip.next();
        }
        // every copy has landed before the block ends: the ring's last loads
        // (place s took the loads s, s + ring, ...)
        for (int s = 0; s < ring && s < loads; ++s)
            if (!warp_wait_far(&fulls[s], ((loads - 1 - s) / ring) & 1, nullptr) && lane == 0)
                raise_error(kErrTimeout);
        cp_async_wait_all();
    } else if (warp == kWarpTab) {
        // ------------------------------------------------------------ Q and the tables
        int16_t* parent = reinterpret_cast<int16_t*>(trees + 2);
        int it = 0, queries = 0;            // items, loads of Q
        for (;; ++it) {
            if (!wait(&item_full[ip.s], ip.phase) || items[ip.s].take == 0) break;
            const TcItem& I = items[ip.s];
            const int q0 = I.q0, rows = item_rows(I);
            auto load_q = [&]() {
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, S::kQBytes);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_2d(smem + S::kOffQ + c * NQ * 128, &tmQ, q_full, I.h * D + 64 * c,
                                    static_cast<int>(I.row0));
                }
                ++queries;
            };
            if (it == 0) {
                load_q();
            } else if (lane == 0) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_prefetch_2d(&tmQ, I.h * D + 64 * c, static_cast<int>(I.row0));
            }
            if (it >= 2 && !wait(&tab_empty[it & 1], (it / 2 - 1) & 1)) break;
            // loads first: times and the head's time biases
            TcTables<NQ>& T = tabs[it & 1];
            const int64_t* tsq = a.ts + I.row0;
            const float* tbh = a.tb + static_cast<int64_t>(I.h) * a.NB;
            int64_t tq[NQ / 32] = {}, first = 0;
            float tb0 = 0.f, tb1 = 0.f;
            if (use_time) {
                first = __ldg(tsq);
#pragma unroll
                for (int u = 0; u < NQ / 32; ++u) tq[u] = __ldg(tsq + min(lane + 32 * u, rows - 1));
                tb0 = __ldg(tbh + min(lane, a.NB - 1));
                tb1 = __ldg(tbh + min(lane + 32, a.NB - 1));
            }
            TcTree<NQ>& tree = trees[it & 1];
            if (!chain) build_tile_tree<NQ>(a.parents + I.row0 - q0, I.n, q0, tree, parent);
            const int64_t lim = int64_t{1} << 30;
            bool close = true;
            int lo = 0, hi = 0;
#pragma unroll
            for (int u = 0; u < NQ / 32; ++u) {
                const int c = lane + 32 * u, m = min(c, rows - 1);
                const int d = static_cast<int>(tq[u] - first);
                close = close && tq[u] - first < lim && first - tq[u] < lim;
                lo = min(lo, d);
                hi = max(hi, d);
                T.tq[c] = tq[u];
                T.tqr[c] = d;
                T.qo[c] = 4 * (chain ? m : tree.depth[q0 + m]);
            }
            T.tb[lane] = tb0;
            T.tb[lane + 32] = tb1;
            if (lane < 8) T.odd[lane] = 0u;
            close = __all_sync(0xffffffffu, close);
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (lane == 0) {
                T.first = first;
                T.lo = lo;
                T.hi = hi;
                T.close = close;
                T.span = chain ? rows - 1 : tree.deepest;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_full[it & 1]);
            if (it > 0) {
                if (!wait(q_empty, (it - 1) & 1)) break;
                load_q();
            }
            ip.next();
        }
        if (queries > 0 && !warp_wait_far(q_full, (queries - 1) & 1, nullptr) && lane == 0)
            raise_error(kErrTimeout);
    } else if (warp == kWarpWin) {
        // ------------------------------------------------------------ position windows
        TcPlace<4> wp;
        int i = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ok = wait(&item_full[ip.s], ip.phase);
            if (!ok || items[ip.s].take == 0) break;
            // (a tree's window is as wide as its tree is deep)
            if (ok && !chain) ok = wait(&tab_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const TcItem& I = items[ip.s];
            const int span = chain ? item_rows(I) - 1 : tabs[it & 1].span;
            const int take = I.take, part0 = item_part0(I);
            const float* posh = use_pos ? a.pos + static_cast<int64_t>(I.h) * a.P : nullptr;
            for (int j = 0; j < take; ++j, ++i) {
                if (i >= 4) ok = wait(&win_empty[wp.s], wp.phase ^ 1u);
                if (!ok) break;
                if (use_pos) {
                    float* win = reinterpret_cast<float*>(smem + S::kOffWin) + wp.s * S::kWin;
                    const int k0 = (I.tile + j) * kTcKeys;
                    const int least = part0 - origin(I, k0);
                    const int n = (deep(I, k0) ? 1 : kTcKeys) + span;
#pragma unroll 1
                    for (int x = lane; x < n; x += 32)
                        cp_async4(win + x, posh + max(0, min(least + x, a.P - 1)));
                }
                cp_async_arrive(&win_full[wp.s]);
                wp.next();
            }
            ip.next();
        }
        cp_async_wait_all();
    } else if (warp == kWarpS) {
        // ------------------------------------------------------------ S^T = K Q^T
        if (lane == 0) {
            auto one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_far(bar, parity, abort_flag); };
            const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + S::kOffQ));
            const uint64_t dk0 = desc_kmajor_sw128(smem_u32(smem));
            TcPlace<NK> kp;
            bool ok = true;
            int i = 0;
            for (int it = 0; ok; ++it) {
                ok = one(&item_full[ip.s], ip.phase);
                if (!ok || items[ip.s].take == 0) break;
                ok = one(q_full, it & 1);
                if (!ok) break;
                const int take = items[ip.s].take;
                const uint32_t idesc =
                    idesc_bf16_f32(128, (item_rows(items[ip.s]) + 15) / 16 * 16, 0, 0);
                for (int j = 0; j < take; ++j, ++i) {
                    ok = one(&k_full[kp.s], kp.phase) &&
                         (i < 2 || one(&s_empty[i & 1], ((i >> 1) - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dk = dk0 + static_cast<uint64_t>(kp.s * (S::kSlotBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16_ss(tmem + (i & 1) * 128,
                                     dk + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                     dq + (((kk >> 2) * NQ * 128 + (kk & 3) * 32) >> 4), idesc,
                                     kk > 0 ? 1u : 0u);
                    umma_commit(&s_full[i & 1]);
                    umma_commit(&k_empty[kp.s]);
                    kp.next();
                }
                if (ok) umma_commit(q_empty);
                ip.next();
            }
            umma_commit(&drain[0]);
            if (!mbar_wait_far(&drain[0], 0, nullptr)) raise_error(kErrTimeout);
        }
        __syncwarp();
    } else if (warp == kWarpO) {
        // ------------------------------------------------------------ O^T += V^T P^T
        if (lane == 0) {
            auto one = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_far(bar, parity, abort_flag); };
            const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(smem + S::kOffV), D == 64 ? 0 : 16384);
            const uint64_t dp0 = desc_mnmajor_sw128(smem_u32(smem + S::kOffP), 16384);
            TcPlace<NV> vp;
            int i = 0, tail = 0;
            bool ok = true;
            for (int it = 0; ok; ++it) {
                ok = one(&item_full[ip.s], ip.phase);
                if (!ok || items[ip.s].take == 0) break;
                ok = it < 2 || one(&o_empty[it & 1], (it / 2 - 1) & 1);
                if (!ok) break;
                const TcItem& I = items[ip.s];
                const int take = I.take, part0 = item_part0(I);
                int k1 = (I.tile + 1) * kTcKeys;
                const uint32_t idesc = idesc_bf16_f32(128, (item_rows(I) + 15) / 16 * 16, 1, 1);
                const uint32_t dst = tmem + 256 + (it & 1) * 128;
                for (int j = 0; j < take; ++j, ++i, k1 += kTcKeys) {
                    ok = one(&v_full[vp.s], vp.phase) &&
                         (k1 <= part0 || one(&v_clean[tail & 3], (tail >> 2) & 1)) &&
                         one(&p_full[i & 1], (i >> 1) & 1);
                    if (!ok) break;
                    if (k1 > part0) ++tail;
                    tc_fence_after();
                    const uint64_t dv = dv0 + static_cast<uint64_t>(vp.s * (S::kSlotBytes >> 4));
                    const uint64_t dp = dp0 + static_cast<uint64_t>((i & 1) * (S::kPBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kTcKeys / 16; ++kk)
                        umma_bf16_ss(dst, dv + ((kk * 2048) >> 4), dp + ((kk * 2048) >> 4), idesc,
                                     j > 0 || kk > 0 ? 1u : 0u);
                    umma_commit(&p_empty[i & 1]);
                    umma_commit(&v_empty[vp.s]);
                    vp.next();
                }
                if (ok) umma_commit(&o_full[it & 1]);
                ip.next();
            }
            umma_commit(&drain[1]);
            if (!mbar_wait_far(&drain[1], 0, nullptr)) raise_error(kErrTimeout);
        }
        __syncwarp();
    } else if (warp < kTcPointWarps) {
        // ------------------------------------------------------------ pointwise stage
        const int grp = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;              // the step's key
        const uint32_t s_col = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + grp * 128;
        const uint32_t prow = smem_u32(smem + S::kOffP + grp * S::kPBytes) + r * 128;
        const int box_shift = min(7, a.shift);
        const int64_t lim = int64_t{1} << 30;
        int i = 0;                                      // first step of the item
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ok = wait(&item_full[ip.s], ip.phase);
            if (!ok || items[ip.s].take == 0) break;
            ok = wait(&tab_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const TcItem I = items[ip.s];
            const TcTables<NQ>& T = tabs[it & 1];
            const TcTree<NQ>& tree = trees[it & 1];
            const int len = item_len(I), part0 = item_part0(I), nc = (item_rows(I) + 7) / 8 * 8;
            const int64_t first = T.first;
            const int span = T.span;
            for (int j = (i & 1) == grp ? 0 : 1; j < I.take; j += 2) {
                const int st = i + j, k0 = (I.tile + j) * kTcKeys, key = k0 + r;
                const int m = key - I.ctx;              // new token's index, < 0: cached
                const int tp = st % NT, wb = st & 3;
                ok = wait(&tk_full[tp], (st / NT) & 1) && wait(&win_full[wb], (st >> 2) & 1);
                if (!ok) break;
                const bool paged = key < len && !((bads[tp] >> (r >> box_shift)) & 1u);
                const int64_t tk = use_time && paged ? tks[tp * kTcKeys + r] : first;
                const int pk = m < 0 || chain ? key : I.ctx + (m < I.n ? tree.depth[m] : 0);
                const float* wr = reinterpret_cast<const float*>(smem + S::kOffWin) + wb * S::kWin +
                                  (origin(I, k0) - pk);
                // Most keys are far from the new tokens: all queries fall into one
                // or two buckets, and one comparison replaces the table.
                const int tkr = static_cast<int>(tk - first);
                const uint32_t b_lo = bucket_bytes(T.lo - tkr), b_hi = bucket_bytes(T.hi - tkr);
                const bool two = __all_sync(0xffffffffu, T.close && first - tk < lim && tk - first < lim &&
                                                             b_hi - b_lo <= 4u);
                float add_lo = 0.f, add_hi = 0.f;
                int turn = 0;                           // first relative time of the upper bucket
                if (two && use_time) {
                    add_lo = table_at(T.tb, b_lo - kBucketBias);
                    add_hi = table_at(T.tb, b_hi - kBucketBias);
                    if (b_hi != b_lo) turn = tkr + (1 << ((b_hi - kBucketBias) >> 2));
                }
                const bool wide = use_pos && span > 0;
                const float same = use_pos && !wide ? wr[0] : 0.f;  // candidates side by side
                add_lo += same;
                add_hi += same;
                ok = wait(&s_full[grp], (st >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                auto scores = [&](int c0, float (&x)[8]) {
                    uint32_t sv[8];
                    tmem_ld8(s_col + c0, sv);
                    if (c0 + 8 >= nc) {                 // S has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[grp]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(sv[e]);
                };
                // 64 queries a 128-byte row, 16-byte pieces in the 128-byte swizzle
                auto store = [&](int c0, const uint32_t (&p)[4]) {
                    if (c0 == 0 && st >= 2)             // the product with P of two steps ago is done
                        ok = wait(&p_empty[grp], ((st >> 1) - 1) & 1);
                    st_shared_v4(prow + (c0 >> 6) * 16384 + ((((c0 & 63) >> 3) ^ (r & 7)) << 4), p[0], p[1],
                                 p[2], p[3]);
                };
                // entries of wr behind the last query's belong to columns nobody reads
                auto add_window = [&](int c0, float (&x)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const int4 qo = *reinterpret_cast<const int4*>(T.qo + c0 + e);
                        x[e] += table_at(wr, qo.x);
                        x[e + 1] += table_at(wr, qo.y);
                        x[e + 2] += table_at(wr, qo.z);
                        x[e + 3] += table_at(wr, qo.w);
                    }
                };
                auto add_two = [&](int c0, float (&x)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const int4 tq = *reinterpret_cast<const int4*>(T.tqr + c0 + e);
                        x[e] += tq.x >= turn ? add_hi : add_lo;
                        x[e + 1] += tq.y >= turn ? add_hi : add_lo;
                        x[e + 2] += tq.z >= turn ? add_hi : add_lo;
                        x[e + 3] += tq.w >= turn ? add_hi : add_lo;
                    }
                };
                auto weights = [](const float (&x)[8], uint32_t (&p)[4]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = pack_bf16x2(silu_exp(x[2 * e]), silu_exp(x[2 * e + 1]));
                };
                if (two && k0 + kTcKeys <= part0 && __all_sync(0xffffffffu, paged)) {
                    // every query sees the key
#pragma unroll 1
                    for (int c0 = 0; c0 < nc; c0 += 8) {
                        float x[8];
                        uint32_t p[4];
                        scores(c0, x);
                        if (wide) add_window(c0, x);
                        add_two(c0, x);
                        weights(x, p);
                        store(c0, p);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < nc; c0 += 8) {
                        float x[8];
                        uint32_t p[4];
                        scores(c0, x);
                        if (wide) add_window(c0, x);
                        if (two) {
                            add_two(c0, x);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int64_t dt = max(T.tq[c0 + e] - tk, int64_t{1});
                                x[e] += same + table_at(T.tb, ((__float_as_uint(__ll2float_rz(dt)) >> 21) &
                                                               0x7fcu) - kBucketBias);
                            }
                        }
                        uint32_t seen = 0xffu;
                        if (m >= I.n || !paged) {
                            seen = 0u;
                        } else if (m >= 0) {
                            const int d = m - I.q0 - c0;    // chain: the first query that sees the key
                            seen = chain ? (d <= 0 ? 0xffu : d < 8 ? 0xffu << d : 0u)
                                         : tree.seen[c0 >> 5][m] >> (c0 & 24);
                        }
                        weights(x, p);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p[e] &= ((seen >> (2 * e)) & 1u) * 0xffffu |
                                    ((seen >> (2 * e + 1)) & 1u) * 0xffff0000u;
                        store(c0, p);
                    }
                }
                if (!ok) break;
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[grp]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&win_empty[wb]);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&point_done[it & 1]);
            i += I.take;
            ip.next();
        }
    } else {
        // ------------------------------------------------------------ the items' rows
        const int quarter = warp & 3;
        const int d = quarter * 32 + lane;              // column of the output, TMEM lane; row of V
        const uint32_t o_col = tmem + 256 + (static_cast<uint32_t>(quarter * 32) << 16);
        int i = 0, tail = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ok = wait(&item_full[ip.s], ip.phase);
            if (!ok || items[ip.s].take == 0) break;
            ok = wait(&tab_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const TcItem I = items[ip.s];
            TcTables<NQ>& T = tabs[it & 1];
            const int rows = item_rows(I);
            // V of the steps with keys that some query does not see: those meet
            // zeros in P, so they have to be finite. Rows behind the sequence and
            // rows of new tokens that are not finite become zeros; the latter are
            // added alone to the queries that see them.
            const int part0 = item_part0(I), len = item_len(I);
            for (int j = max(0, part0 / kTcKeys - I.tile); ok && j < I.take; ++j, ++tail) {
                const int st = i + j, s = st % NV, key = (I.tile + j) * kTcKeys + d;
                // (its load has been issued, so the slot's barrier is at this load's phase)
                ok = wait(&v_loading[tail & 3], (tail >> 2) & 1) && wait(&v_full[s], (st / NV) & 1);
                if (!ok) break;
                uint8_t* vr = smem + S::kOffV + s * S::kSlotBytes + d * 128;
                bool clear = key >= len;
                if (key >= part0 && key < len) {
                    bool bad = false;
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            vr + (c >> 3) * 16384 + (((c & 7) ^ (d & 7)) << 4));
                        const uint32_t f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bad = bad || (f[e] & 0x7f80u) == 0x7f80u ||
                                  (f[e] & 0x7f800000u) == 0x7f800000u;
                    }
                    if (bad) {
                        const int o = key - part0;          // < 256: a tile's chain or a tree
                        atomicOr(&T.odd[o >> 5], 1u << (o & 31));
                        clear = true;
                    }
                }
                if (clear) {
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c)
                        *reinterpret_cast<uint4*>(vr + (c >> 3) * 16384 + ((c & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                mbar_arrive(&v_clean[tail & 3]);
                ok = wait(&v_clean[tail & 3], (tail >> 2) & 1);     // T.odd is complete
            }
            i += I.take;
            ok = ok && wait(&point_done[it & 1], (it >> 1) & 1) && wait(&o_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            uint32_t any_odd = 0u;
#pragma unroll
            for (int o = 0; o < 8; ++o) any_odd |= T.odd[o];
            // (with odd keys the rows go through the block's part, whole or not)
            const bool whole = I.whole && !any_odd;
            float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (it == 0 ? 0 : 1)) * a.part_rows * D +
                          d;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + I.row0 * a.out_stride +
                                 static_cast<int64_t>(I.h) * D + (d & ~1);
            const int odd_lane = lane & 1;
#pragma unroll 1
            for (int c0 = 0; c0 < rows && quarter * 32 < D; c0 += 8) {
                uint32_t ov[8];
                tmem_ld8(o_col + (it & 1) * 128 + c0, ov);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float x0 = __uint_as_float(ov[e]), x1 = __uint_as_float(ov[e + 1]);
                    if (whole) {
                        // even lanes write columns d, d + 1 of query e, odd ones of e + 1
                        const float other = __shfl_xor_sync(0xffffffffu, odd_lane ? x0 : x1, 1);
                        const float mine = odd_lane ? x1 : x0;
                        const int c = c0 + e + odd_lane;
                        if (c < rows)
                            *reinterpret_cast<uint32_t*>(out + c * a.out_stride) =
                                odd_lane ? pack_bf16x2(other * a.inv_n, mine * a.inv_n)
                                         : pack_bf16x2(mine * a.inv_n, other * a.inv_n);
                    } else {
                        if (c0 + e < rows) part[(c0 + e) * D] = x0;
                        if (c0 + e + 1 < rows) part[(c0 + e + 1) * D] = x1;
                    }
                }
            }
            if (any_odd && quarter * 32 < D)
                add_odd_keys<D, NQ>(a, T, trees[it & 1], I.row0, I.ctx, chain ? I.q0 : 0, I.q0, rows, I.h,
                                    I.b, d, part, I.whole != 0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&o_empty[it & 1]);
                mbar_arrive(&tab_empty[it & 1]);
                mbar_arrive(&item_empty[ip.s]);
            }
            ip.next();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) raise_error(kErrTimeout);
    if (warp == kWarpS) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace hstu
