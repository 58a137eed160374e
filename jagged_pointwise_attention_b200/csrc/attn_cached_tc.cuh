// attn_cached_tc.cuh -- attention of many new tokens (trees of dozens, rows of
// candidates, pieces of a prompt) over a paged cache, bf16 on tcgen05
// (attn_cached.cuh has the formula and the work line).
//
// Items are tiles of NQ queries of one head; a step is 128 keys:
//   S^T [128 keys x nq] = K Q^T            TMEM, two buffers
//   P^T = silu(S^T + biases), bf16         shared memory, two buffers
//   O [queries x D] += P V                 TMEM, two buffers (items)
// The long axis fills the 128 rows of the first product, so its width nq can
// be the item's own count (rounded up to 16) and few queries cost few columns.
// A thread of the pointwise stage owns one key: its position, timestamp and
// page are its own, the queries' come as broadcasts, and its row of P^T is
// what the second product reads as an A operand with the queries contiguous.
//
// Warp roles: eight pointwise warps in two groups that take turns at the
// steps; one warp loads K and V tiles by TMA, a page (or 128 tokens of one) a
// box, its lanes a page each; one loads Q; one issues the products and owns
// TMEM. K and V share one ring in the order K0 K1 V0 K2 V1 ..., which is the
// order their products run in, so the ring's depth serves both.
//
// Bound by the cache's bytes up to about 64 queries, above that by the
// pointwise stage (two SFU operations and about sixteen instructions a pair).
#pragma once

#include "attn_cached.cuh"
#include "attn_cached_mma.cuh"

namespace hstu {

constexpr int kTcKeys = 128;
constexpr int kTcPointThreads = 256;
constexpr int kTcThreads = kTcPointThreads + 96;

template <int D, int NQ>
struct CachedTcSmem {
    static constexpr int kSlotBytes = kTcKeys * D * 2;
    static constexpr int kSlots = D == 64 ? 6 : NQ == 64 ? 5 : 3;
    static constexpr int kPBytes = NQ / 64 * 16384;
    static constexpr int kQBytes = NQ * D * 2;
    static constexpr int kWin = 128 + kMaxTree + 8;         // positions of a step: 127 + span
    static constexpr int kOffQ = kSlots * kSlotBytes;
    static constexpr int kOffP = kOffQ + kQBytes;
    static constexpr int kOffWin = kOffP + 2 * kPBytes;     // [group][parity][kWin]
    static constexpr int kOffTq = kOffWin + 4 * kWin * 4;   // int64 [NQ]
    static constexpr int kOffTql = kOffTq + NQ * 8;         // their low words
    static constexpr int kOffQo = kOffTql + NQ * 4;         // 4 x position behind the tile's lowest
    static constexpr int kOffTb = kOffQo + NQ * 4;
    static constexpr int kOffBar = kOffTb + 64 * 4;
    static constexpr int kOffScratch = kOffBar + 64 * 8;
    static constexpr int kOffMisc = kOffScratch + (kTcThreads / 32 + 9) * 8;
    static constexpr int kOffTree = (kOffMisc + 96 + 15) / 16 * 16;
    static constexpr int kBytes = kOffTree + static_cast<int>(sizeof(TreeSmem));
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory per block");
    static_assert(2 * kSlots + 10 <= 64, "barriers");
};

// A key's contribution to one query, alone: the rare keys whose values are not
// finite and which some query of the tile does not see.
template <int D>
__device__ __forceinline__ float cached_weight(const CachedArgs& a, int h, int64_t qrow, int pq,
                                               int pk, int64_t tq, const __nv_bfloat16* krow,
                                               int64_t tk, const float* tbs) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + qrow * a.q_stride +
                             static_cast<int64_t>(h) * D;
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(q[c]), __bfloat162float(krow[c]), s);
    if (a.pos) s += a.pos[static_cast<int64_t>(h) * a.P + min(pq - pk, a.P - 1)];
    if (a.tsc) s += tbs[time_bucket64(tq - tk, 63)];
    return silu_exp(s);
}

template <int D, int NQ>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_cached_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CachedArgs a) {
    using S = CachedTcSmem<D, NQ>;
    using L = Line<kTcKeys, NQ>;
    constexpr int NS = S::kSlots;
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps seeing shared memory)
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t* tqs = reinterpret_cast<int64_t*>(smem + S::kOffTq);
    int* tql = reinterpret_cast<int*>(smem + S::kOffTql);
    int* qos = reinterpret_cast<int*>(smem + S::kOffQo);
    float* tbs = reinterpret_cast<float*>(smem + S::kOffTb);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    uint64_t* empty = full + NS;
    uint64_t* q_full = empty + NS;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;         // [2]
    uint64_t* p_full = s_full + 2;          // [2]
    uint64_t* p_empty = p_full + 2;         // [2]
    uint64_t* o_full = p_empty + 2;         // [2]
    uint64_t* o_empty = o_full + 2;         // [2]
    uint64_t* drain = o_empty + 2;
    int64_t* scratch = reinterpret_cast<int64_t*>(smem + S::kOffScratch);
    uint8_t* misc = smem + S::kOffMisc;
    int64_t* t_lim = reinterpret_cast<int64_t*>(misc);              // least and greatest of tqs
    uint32_t* odd = reinterpret_cast<uint32_t*>(misc + 16);         // [8] new keys to add alone
    int* q_span = reinterpret_cast<int*>(misc + 48);                // greatest of qos
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 56);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 64);
    TreeSmem& tree = *reinterpret_cast<TreeSmem*>(smem + S::kOffTree);
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
            mbar_init(&o_empty[s], kTcPointThreads);
        }
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
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: S at 0 and 128, O at 256 and 384

    // A walk over the block's steps, one for each use of them.
    struct Walk {
        LineAt at;
        int64_t left;           // steps from the item's first of this block on
        int take, j;            // the item's steps here, and how many are behind
        __device__ __forceinline__ void enter() {
            take = static_cast<int>(min(left, static_cast<int64_t>(L::tiles(at.s, at.qt) - at.j)));
            j = 0;
        }
        __device__ __forceinline__ void next(const CachedArgs& a) {
            if (++j < take) return;
            left -= take;
            if (left <= 0) return;
            L::next_item(a, at);
            enter();
        }
        __device__ __forceinline__ int key0() const { return (at.j + j) * kTcKeys; }
        __device__ __forceinline__ int rows() const { return min(NQ, at.s.n - at.qt * NQ); }
        __device__ __forceinline__ int len() const { return at.s.ctx + min(at.s.n, (at.qt + 1) * NQ); }
    };
    Walk w0;
    w0.at = at;
    w0.left = steps;
    w0.enter();

    if (warp == 8) {
        // ------------------------------------------------------------ K and V
        Walk kw = w0, vw = w0;
        const int box = min(kTcKeys, 1 << a.shift), boxes = kTcKeys / box;
        int64_t seq = 0;
        bool ok = true;
        auto load = [&](Walk& w, const CUtensorMap* tm, bool report) {
            const int s = static_cast<int>(seq % NS);
            const int key = w.key0() + lane * box;
            int page = a.num_pages;         // past the cache: zeros
            if (lane < boxes && key < w.len()) {
                page = __ldg(a.table + static_cast<int64_t>(w.at.b) * a.table_stride + (key >> a.shift));
                if (page < 0 || page >= a.num_pages) {
                    if (report) raise_error(kErrBadInput);
                    page = a.num_pages;
                }
            }
            if (seq >= NS && !warp_wait(&empty[s], (seq / NS - 1) & 1, abort_flag)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], S::kSlotBytes);
            __syncwarp();
            if (lane < boxes) {
                uint8_t* dst = smem + s * S::kSlotBytes + lane * box * 128;
                const int row = key & ((1 << a.shift) - 1);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(dst + c * 16384, tm, &full[s], w.at.h * D + 64 * c, row, page);
            }
            ++seq;
            w.next(a);
            return true;
        };
        ok = load(kw, &tmK, true);
        for (int64_t i = 0; ok && i < steps; ++i) {
            if (i + 1 < steps) ok = load(kw, &tmK, true);
            if (ok) ok = load(vw, &tmV, false);
        }
        // every copy has landed before the block ends
        for (int s = 0; s < NS; ++s) {
            const int64_t c = seq > s ? (seq - s + NS - 1) / NS : 0;
            if (c > 0 && !warp_wait(&full[s], (c - 1) & 1, nullptr) && lane == 0)
                raise_error(kErrTimeout);
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------ Q
        if (lane == 0) {
            Walk w = w0;
            int it = 0;
            while (true) {
                if (it > 0 && !mbar_wait(q_empty, (it - 1) & 1, abort_flag)) break;
                mbar_arrive_expect_tx(q_full, S::kQBytes);
                const int row = static_cast<int>(w.at.s.off) + w.at.qt * NQ;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_2d(smem + S::kOffQ + c * NQ * 128, &tmQ, q_full, w.at.h * D + 64 * c, row);
                ++it;
                w.j = w.take - 1;
                w.next(a);
                if (w.left <= 0) break;
            }
            if (it > 0 && !mbar_wait(q_full, (it - 1) & 1, nullptr)) raise_error(kErrTimeout);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            Walk sw = w0, ow = w0;
            int sit = 0, oit = 0;           // items
            bool ok = true;
            const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + S::kOffQ));
            const uint64_t dk0 = desc_kmajor_sw128(smem_u32(smem));
            const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(smem), 16384);
            // 64 queries: both halves of the 128 rows read the same P (the upper is not used)
            const uint64_t dp0 = desc_mnmajor_sw128(smem_u32(smem + S::kOffP), NQ == 64 ? 0 : 16384);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, 1, 1);
            auto scores = [&](int64_t i) {
                const int64_t seq = i == 0 ? 0 : 2 * i - 1;
                const int s = static_cast<int>(seq % NS);
                if ((sw.j == 0 && !mbar_wait(q_full, sit & 1, abort_flag)) ||
                    !mbar_wait(&full[s], (seq / NS) & 1, abort_flag))
                    return false;
                tc_fence_after();
                const uint32_t idesc = idesc_bf16_f32(128, (sw.rows() + 15) / 16 * 16, 0, 0);
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
                const uint64_t dv = dv0 + static_cast<uint64_t>(s * (S::kSlotBytes >> 4));
                const uint64_t dp = dp0 + static_cast<uint64_t>((i & 1) * (S::kPBytes >> 4));
                const uint32_t dst = tmem + 256 + (oit & 1) * 128;
#pragma unroll
                for (int kk = 0; kk < kTcKeys / 16; ++kk)
                    umma_bf16_ss(dst, dp + ((kk * 2048) >> 4), dv + ((kk * 2048) >> 4), idesc_o,
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
    } else {
        // ------------------------------------------------------------ pointwise stage
        const int grp = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;              // the step's key, later the query
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t s_col = tmem + lane_base + grp * 128;
        uint8_t* prow = smem + S::kOffP + grp * S::kPBytes + r * 128;
        auto all = [] { named_bar_sync(1, kTcPointThreads); };
        Walk w = w0;
        // After a wait that gave up, the walk goes on without waiting, so that
        // every thread still comes to every barrier.
        int64_t i = 0;                                  // step of the block
        int it = 0, mine = 0, tree_of = -1, head_of = -1;
        bool ok = true;
        while (w.left > 0) {
            const LineAt& I = w.at;
            const int q0 = I.qt * NQ, rows = w.rows(), len = w.len();
            const int nc = (rows + 15) / 16 * 16;
            all();                                      // the previous item is done with
            if (!chain && tree_of != I.b) {
                build_tree(a, I.s, tree, tid, kTcPointThreads, all);
                tree_of = I.b;
            }
            if (tid < NQ) {
                const int m = min(tid, rows - 1);
                qos[tid] = 4 * (chain ? m : tree.depth[q0 + m]);
                if (use_time) {
                    tqs[tid] = a.ts[I.s.off + q0 + m];
                    tql[tid] = static_cast<int>(tqs[tid]);
                }
            }
            if (tid < 8) odd[tid] = 0u;
            if (use_time && head_of != I.h && tid >= 192)
                tbs[tid - 192] = a.tb[static_cast<int64_t>(I.h) * a.NB + min(tid - 192, a.NB - 1)];
            head_of = I.h;
            all();
            if (warp == 0) {
                int64_t lo = INT64_MAX, hi = INT64_MIN;
                int span = 0;
                for (int c = lane; c < rows; c += 32) {
                    span = max(span, qos[c]);
                    if (use_time) {
                        lo = min(lo, tqs[c]);
                        hi = max(hi, tqs[c]);
                    }
                }
                for (int o = 16; o > 0; o >>= 1) {
                    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                    span = max(span, __shfl_xor_sync(0xffffffffu, span, o));
                }
                if (lane == 0) {
                    t_lim[0] = lo;
                    t_lim[1] = hi;
                    q_span[0] = span;
                }
            }
            all();
            const int pbase = I.s.ctx + (chain ? q0 : 0);   // position of qos == 0
            // keys from here on are seen by some queries and not by others
            const int part0 = pbase;
            const float* posh = use_pos ? a.pos + static_cast<int64_t>(I.h) * a.P : nullptr;
            const int span = q_span[0] / 4;
            // this thread's key of a step: its page (-1: none) and timestamp
            auto key_of = [&](int j, int& page) {
                const int key = (I.j + j) * kTcKeys + r;
                page = -1;
                if (j < w.take && key < len)
                    page = __ldg(a.table + static_cast<int64_t>(I.b) * a.table_stride + (key >> a.shift));
            };
            auto time_of = [&](int j, int page) -> int64_t {
                if (!use_time || page < 0 || page >= a.num_pages) return 0;
                const int key = (I.j + j) * kTcKeys + r;
                return __ldg(a.tsc + page * a.tsc_page + (key & ((1 << a.shift) - 1)));
            };
            int j0 = (i & 1) == grp ? 0 : 1;            // the group's first step of the item
            int page;
            key_of(j0, page);
            int64_t tk = time_of(j0, page);
            for (int j = j0; j < w.take; j += 2, ++mine) {
                const int64_t st = i + j;
                const int k0 = (I.j + j) * kTcKeys, key = k0 + r;
                int next_page;
                key_of(j + 2, next_page);
                const bool fast = k0 + kTcKeys <= part0;
                float* win = reinterpret_cast<float*>(smem + S::kOffWin) + (2 * grp + (mine & 1)) * S::kWin;
                if (use_pos && fast) {
                    // position biases of the step: distances from the lowest up
                    const int least = pbase - (k0 + kTcKeys - 1);
                    for (int x = r; x < kTcKeys + span; x += 128)
                        win[x] = __ldg(posh + min(least + x, a.P - 1));
                    named_bar_sync(2 + grp, 128);
                }
                ok = ok && warp_wait(&s_full[grp], (st >> 1) & 1, abort_flag) &&
                     (st < 2 || warp_wait(&p_empty[grp], ((st >> 1) - 1) & 1, abort_flag));
                tc_fence_after();
                const bool paged = page >= 0 && page < a.num_pages;
                const int m = key - I.s.ctx;            // new token's index, < 0: cached
                bool near = true;
                if (use_time) {
                    const int64_t lim = int64_t{1} << 31;
                    near = t_lim[1] - tk < lim && t_lim[0] - tk > -lim;
                    near = __all_sync(0xffffffffu, near);
                }
                const int tkl = static_cast<int>(tk);
                const int pk = m >= 0 && !chain && m < I.s.n ? I.s.ctx + tree.depth[m] : key;
                const float* wr = win + (kTcKeys - 1 - r);
#pragma unroll 1
                for (int c0 = 0; c0 < nc; c0 += 16) {
                    uint32_t sv[16];
                    tmem_ld16(s_col + c0, sv);
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(sv[e]);
                    // (entries behind the last query's belong to columns nobody reads)
                    if (use_pos) {
                        if (fast && chain) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] += wr[c0 + e];
                        } else if (fast) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 qo = *reinterpret_cast<const int4*>(qos + c0 + e);
                                x[e] += table_at(wr, qo.x);
                                x[e + 1] += table_at(wr, qo.y);
                                x[e + 2] += table_at(wr, qo.z);
                                x[e + 3] += table_at(wr, qo.w);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[e] += __ldg(posh + max(0, min(pbase + qos[c0 + e] / 4 - pk, a.P - 1)));
                        }
                    }
                    if (use_time) {
                        if (near) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const int4 tq = *reinterpret_cast<const int4*>(tql + c0 + e);
                                x[e] += table_at(tbs, bucket_bytes(tq.x - tkl) - kBucketBias);
                                x[e + 1] += table_at(tbs, bucket_bytes(tq.y - tkl) - kBucketBias);
                                x[e + 2] += table_at(tbs, bucket_bytes(tq.z - tkl) - kBucketBias);
                                x[e + 3] += table_at(tbs, bucket_bytes(tq.w - tkl) - kBucketBias);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[e] += tbs[time_bucket64(tqs[c0 + e] - tk, 63)];
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
                    if (seen != 0xffffu) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            pk2[e] &= ((seen >> (2 * e)) & 1u) * 0xffffu |
                                      ((seen >> (2 * e + 1)) & 1u) * 0xffff0000u;
                    }
                    // 64 queries a 128-byte row, 16-byte pieces in the 128-byte swizzle
                    const uint32_t base = smem_u32(prow) + (c0 >> 6) * 16384;
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
                    ok = ok && warp_wait(&full[s], (seq / NS) & 1, abort_flag);
                    uint8_t* vr = smem + s * S::kSlotBytes + r * 128;
                    bool clear = key >= len;
                    if (key >= part0 && key < len) {
                        bool bad = false;
#pragma unroll 1
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
                            atomicOr(&odd[o >> 5], 1u << (o & 31));
                            clear = true;
                        }
                    }
                    if (clear) {
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(vr + (c >> 3) * 16384 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&p_full[grp]);
                page = next_page;
                tk = time_of(j + 2, page);
            }
            // ---- the item's rows: thread r of group g has query r, columns g D/2 ..
            all();                                      // odd is complete
            ok = ok && warp_wait(&o_full[it & 1], (it >> 1) & 1, abort_flag);
            tc_fence_after();
            const bool whole = w.take == L::tiles(I.s, I.qt);
            float* part = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (it == 0 ? 0 : 1)) * NQ * D +
                          static_cast<int64_t>(r) * D;
            __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) +
                                  (I.s.off + q0 + r) * a.out_stride + static_cast<int64_t>(I.h) * D;
            uint32_t any_odd = 0u;
            for (int o = 0; o < 8; ++o) any_odd |= odd[o];
#pragma unroll 1
            for (int c0 = grp * (D / 2); c0 < (grp + 1) * (D / 2); c0 += 32) {
                uint32_t ov[32];
                __syncwarp();
                if (quarter * 32 < rows) tmem_ld32(tmem + 256 + (it & 1) * 128 + lane_base + c0, ov);
                if (r < rows) {
                    if (any_odd) {
#pragma unroll 1
                        for (int o = 0; o < kMaxTree; ++o) {
                            if (!((odd[o >> 5] >> (o & 31)) & 1u)) continue;
                            const int key = part0 + o, m = key - I.s.ctx, qi = q0 + r;
                            if (chain ? m > qi : !((tree.seen[qi >> 5][m] >> (qi & 31)) & 1u)) continue;
                            const int pg = a.table[static_cast<int64_t>(I.b) * a.table_stride +
                                                   (key >> a.shift)];
                            const int row = key & ((1 << a.shift) - 1);
                            const float p = cached_weight<D>(
                                a, I.h, I.s.off + qi, pbase + qos[r] / 4,
                                chain ? key : I.s.ctx + tree.depth[m], use_time ? tqs[r] : 0,
                                static_cast<const __nv_bfloat16*>(a.k) + pg * a.k_page + row * a.k_tok +
                                    static_cast<int64_t>(I.h) * D,
                                use_time ? a.tsc[pg * a.tsc_page + row] : 0, tbs);
                            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) +
                                                     pg * a.v_page + row * a.v_tok +
                                                     static_cast<int64_t>(I.h) * D + c0;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                ov[e] = __float_as_uint(
                                    fmaf(p, __bfloat162float(v[e]), __uint_as_float(ov[e])));
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t f[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                f[u] = pack_bf16x2(__uint_as_float(ov[8 * e + 2 * u]) * a.inv_n,
                                                   __uint_as_float(ov[8 * e + 2 * u + 1]) * a.inv_n);
                            *reinterpret_cast<uint4*>(orow + c0 + 8 * e) =
                                make_uint4(f[0], f[1], f[2], f[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<uint4*>(part + c0 + 4 * e) =
                                make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&o_empty[it & 1]);
            i += w.take;
            ++it;
            w.j = w.take - 1;
            w.next(a);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) raise_error(kErrTimeout);
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace hstu
