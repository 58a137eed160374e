// cache_plan.cuh -- the paged key/value cache: the plan of a step (block
// tables and slot maps from request lengths) and the append of new rows.
//
// A cache holds num_pages pages of page_size tokens (a power of two). Token p
// of a sequence lies in page table[p / page_size], row p % page_size; its slot
// is page * page_size + row. Sequence b has ctx_b tokens in the cache and gets
// n_b new ones, at positions ctx_b .. ctx_b + n_b - 1:
//   have_b = ceil(ctx_b / P)      pages it holds
//   need_b = ceil((ctx_b + n_b) / P) - have_b
//   base_b = free_start + sum_{c < b} need_c
//   table[b][have_b + k] = free_pages[base_b + k]          k < need_b
//   slot[o_b + i] = table[b][(ctx_b + i) / P] * P + (ctx_b + i) % P
// All of it is a scan of B small integers and then independent stores.
#pragma once

#include "common.cuh"

namespace hstu {

struct CachePlanArgs {
    const int32_t* ctx;         // [B]
    const int64_t* off;         // [B + 1], off[B] <= T: the rows behind are padding
    int B;
    int64_t T;
    int shift;                  // log2(page_size)
    const int32_t* free_pages;  // [num_free]
    int num_free;
    const int32_t* free_start;  // [1]
    int32_t* table;             // [B, max_pages], row stride table_stride
    int64_t table_stride;
    int max_pages;
    int64_t* slots;             // [T]
    int32_t* free_end;          // [1]
    int seqs_per_block;         // <= kPlanSeqs
};

constexpr int kPlanThreads = 256;
constexpr int kPlanSeqs = 256;

struct PlanSeq {
    int64_t off;
    int ctx, n, have, need;     // need: pages to take
};

constexpr int64_t kPlanNone = INT64_MIN;    // less than every offset

// One sequence's numbers; a sequence that cannot be (negative lengths, offsets
// outside [0, T], one below `top`, the greatest before it, more pages than a
// table row has) takes no pages, `ok` false.
__device__ __forceinline__ PlanSeq plan_seq(const CachePlanArgs& a, int b, int64_t top, bool& ok) {
    PlanSeq s;
    const int64_t o = a.off[b], e = a.off[b + 1];
    const int64_t c = a.ctx[b];
    ok = c >= 0 && o >= 0 && o >= top && e >= o && e <= a.T && (b > 0 || o == 0) &&
         ((c + (e - o) + (1 << a.shift) - 1) >> a.shift) <= a.max_pages;
    s.off = o;
    s.ctx = ok ? static_cast<int>(c) : 0;
    s.n = ok ? static_cast<int>(e - o) : 0;
    const int page = 1 << a.shift;
    s.have = static_cast<int>((static_cast<int64_t>(s.ctx) + page - 1) >> a.shift);
    s.need = static_cast<int>((static_cast<int64_t>(s.ctx) + s.n + page - 1) >> a.shift) - s.have;
    return s;
}

// Sum over the block, in every thread.
__device__ __forceinline__ int64_t plan_block_sum(int64_t v, int64_t* warp_sums) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();            // the previous sum has been read
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) t += warp_sums[w];
    return t;
}

// Greatest v of the threads before this one (kPlanNone for the first); `all`:
// of the whole block.
__device__ __forceinline__ int64_t plan_max_before(int64_t v, int64_t* warp_max, int64_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, u);
    }
    __syncthreads();            // what was in warp_max has been read
    if (lane == 31) warp_max[warp] = v;
    __syncthreads();
    int64_t before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = kPlanNone;
    all = kPlanNone;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before = max(before, warp_max[w]);
        all = max(all, warp_max[w]);
    }
    return before;
}

// Block (x, y): sequences x * S .. x * S + S - 1, part y of their pages and
// tokens. Every block adds up the pages of all sequences before its own (a
// few loads a thread for thousands of sequences), so one launch needs no
// ordering between blocks: a token's page is one the sequence holds already
// (never written here) or comes straight from the free list. Bound by the
// launch and two dependent loads: 2.9 us in a graph for 128 sequences.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CachePlanArgs a) {
    __shared__ int64_t warp_sums[kPlanThreads / 32];
    __shared__ int64_t s_off[kPlanSeqs];
    __shared__ int64_t s_base[kPlanSeqs];
    __shared__ int s_ctx[kPlanSeqs], s_n[kPlanSeqs], s_have[kPlanSeqs];
    const int tid = threadIdx.x;
    const int b0 = blockIdx.x * a.seqs_per_block;
    const int nb = min(a.seqs_per_block, a.B - b0);
    const bool last = b0 + nb == a.B;
    const int64_t start = a.free_start[0];
    bool all_ok = start >= 0 && start <= a.num_free;

    // the pages of the sequences before, this thread's sequence, and whether an
    // offset falls anywhere up to the block's last sequence
    bool ok = true, fall = false;
    int64_t before = 0;
    for (int b = tid; b < b0; b += kPlanThreads) {
        before += plan_seq(a, b, kPlanNone, ok).need;
        fall = fall || a.off[b + 1] < a.off[b];
    }
    PlanSeq s;
    s.need = 0;
    int64_t top = kPlanNone;    // greatest offset before this thread's sequence
    if (tid < nb) {
        s = plan_seq(a, b0 + tid, kPlanNone, ok);
        fall = fall || a.off[b0 + tid + 1] < a.off[b0 + tid];
    }
    if (__syncthreads_or(fall)) {
        // rare: once more, with the greatest offset before each sequence, so that
        // no row belongs to two of them
        const int per = (b0 + kPlanThreads - 1) / kPlanThreads;
        const int c0 = min(tid * per, b0), c1 = min(c0 + per, b0);
        int64_t m = kPlanNone, all, own;
        for (int b = c0; b < c1; ++b) m = max(m, a.off[b]);
        int64_t run = plan_max_before(m, warp_sums, all);
        before = 0;
        for (int b = c0; b < c1; ++b) {
            before += plan_seq(a, b, run, ok).need;
            run = max(run, a.off[b]);
        }
        top = max(all, plan_max_before(tid < nb ? a.off[b0 + tid] : kPlanNone, warp_sums, own));
        if (tid < nb) s = plan_seq(a, b0 + tid, top, ok);
    }
    before = plan_block_sum(before, warp_sums);

    // this block's sequences: numbers and the scan of their pages
    if (tid < nb) {
        all_ok = all_ok && ok;
        s_off[tid] = max(top, s.off);
        s_ctx[tid] = s.ctx;
        s_n[tid] = s.n;
        s_have[tid] = s.have;
    }
    int64_t scan = s.need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if ((tid & 31) >= o) scan += v;
    }
    __syncthreads();
    if ((tid & 31) == 31) warp_sums[tid >> 5] = scan;
    __syncthreads();
    int64_t mine = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < (tid >> 5)) scan += warp_sums[w];
        mine += warp_sums[w];
    }
    if (tid < nb) s_base[tid] = start + before + scan - s.need;
    __syncthreads();

    // a page of the free list, -1 where the list is short
    auto take = [&](int64_t i) -> int32_t {
        return i >= 0 && i < a.num_free ? a.free_pages[i] : -1;
    };

    // new block-table entries: (sequence, k) pairs of this block, part y
    const int64_t stride = static_cast<int64_t>(gridDim.y) * kPlanThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.y) * kPlanThreads + tid;
    const int64_t base0 = start + before;
    for (int64_t i = first; i < mine; i += stride) {
        int lo = 0, hi = nb - 1;            // last sequence whose base is <= base0 + i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_base[mid] <= base0 + i) lo = mid;
            else hi = mid - 1;
        }
        const int k = static_cast<int>(base0 + i - s_base[lo]);
        const int32_t page = take(base0 + i);
        all_ok = all_ok && page >= 0;
        a.table[static_cast<int64_t>(b0 + lo) * a.table_stride + s_have[lo] + k] = page;
    }

    // slots of the block's rows, part y: from its first offset (row 0 in the
    // first block) to the next block's (the end in the last): rows that belong to
    // no sequence get slot -1
    const int64_t end = a.off[a.B];
    int64_t t0 = b0 == 0 ? 0 : s_off[0], t1 = last ? a.T : max(s_off[nb - 1], a.off[b0 + nb]);
    t0 = t0 < 0 ? 0 : t0;
    t1 = t1 > a.T ? a.T : t1;
    const int page_mask = (1 << a.shift) - 1;
    for (int64_t t = t0 + first; t < t1; t += stride) {
        int lo = 0, hi = nb - 1;            // last sequence whose offset is <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_off[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        int64_t slot = -1;
        const int64_t i = t - s_off[lo];
        if (i >= 0 && i < s_n[lo]) {
            const int p = s_ctx[lo] + static_cast<int>(i);
            const int at = p >> a.shift;
            const int32_t page =
                at < s_have[lo] ? a.table[static_cast<int64_t>(b0 + lo) * a.table_stride + at]
                                : take(s_base[lo] + at - s_have[lo]);
            if (page >= 0) slot = (static_cast<int64_t>(page) << a.shift) | (p & page_mask);
        }
        all_ok = all_ok && (slot >= 0 || t >= end);
        a.slots[t] = slot;
    }
    if (last && blockIdx.y == 0 && tid == 0) {
        const int64_t taken = start + before + mine;
        a.free_end[0] = static_cast<int32_t>(taken < a.num_free ? taken : a.num_free);
    }
    if (!all_ok) raise_error(kErrBadInput);
}

// ------------------------------------------------------------------ append

struct CacheAppendArgs {
    const uint8_t* k;           // token rows, strides and lengths in bytes
    const uint8_t* v;
    int64_t k_stride, v_stride;
    uint8_t* kc;
    uint8_t* vc;
    int64_t kc_page, kc_tok, vc_page, vc_tok;
    int k_bytes, v_bytes;       // H * d * element size
    const int64_t* ts;          // [T] or null
    int64_t* tsc;
    int64_t tsc_page;
    const int64_t* slots;       // [T]
    int64_t T;
    int64_t num_slots;
    int shift;
};

constexpr int kAppendWarps = 8;

// Copies rows to their slots, a warp per token: V is the widest type that
// every address and length is a multiple of. Bound by HBM: four vectors a lane
// are loaded before the first is stored, so 2 KB of a token are in flight.
// 79,913 tokens of 2 x 4 heads of 128 in bf16: 56 us, 5.8 TB/s read and
// written, 0.89 of the measured copy (one vector at a time: 71 us).
template <typename V>
__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(const CacheAppendArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = a.k_bytes / static_cast<int>(sizeof(V));
    const int n = nk + a.v_bytes / static_cast<int>(sizeof(V));
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kAppendWarps;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
    int64_t ahead = t < a.T ? a.slots[t] : 0;   // the next token's slot
    for (; t < a.T; t += stride) {
        const int64_t slot = ahead;
        if (t + stride < a.T) ahead = a.slots[t + stride];
        if (slot < 0 || slot >= a.num_slots) {
            if (slot >= 0 && lane == 0) raise_error(kErrBadInput);
            continue;           // a padded row: nothing to keep
        }
        const int64_t page = slot >> a.shift, row = slot & ((1 << a.shift) - 1);
        const V* ks = reinterpret_cast<const V*>(a.k + t * a.k_stride);
        const V* vs = reinterpret_cast<const V*>(a.v + t * a.v_stride) - nk;
        V* kd = reinterpret_cast<V*>(a.kc + page * a.kc_page + row * a.kc_tok);
        V* vd = reinterpret_cast<V*>(a.vc + page * a.vc_page + row * a.vc_tok) - nk;
        for (int i0 = lane; i0 < n; i0 += 128) {
            V f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u;
                if (i < n) f[u] = i < nk ? ks[i] : vs[i];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u;
                if (i < n) (i < nk ? kd : vd)[i] = f[u];
            }
        }
        if (a.ts != nullptr && lane == 0) a.tsc[page * a.tsc_page + row] = a.ts[t];
    }
}

}  // namespace hstu
