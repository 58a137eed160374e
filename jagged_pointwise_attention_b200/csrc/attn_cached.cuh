// attn_cached.cuh -- attention of new tokens over a paged cache: the work
// line, the tree of new tokens and the join, shared by the kernels: bf16 on
// tcgen05 (attn_cached_tc.cuh) and, for short sequences and heads of 32, on
// warp products (attn_cached_mma.cuh), fp32 on CUDA cores
// (attn_cached_simt.cuh).
//
//   out_i = (1/N) sum_{j seen by i} silu(q_i.k_j + pos[p_i - p_j]
//                                        + time[bucket(t_i - t_j)]) v_j
// A sequence has ctx cached tokens and n new ones, whose keys and values lie
// in the cache at positions ctx .. ctx + n - 1. New token i sees the cached
// tokens, its ancestors among the new ones, and itself; p is ctx + depth for
// new tokens, the index for cached ones.
//
// Work line. An item is (sequence, query tile of NQ new tokens, head); it has
// ceil(len / KT) key tiles, len = ctx + min(n, (qt + 1) NQ) (no new token sees
// a later one). The key tiles of all items, in that order, form one line, and
// block c of the grid takes an equal, contiguous part of it, so long and short
// sequences and any batch load all blocks alike. (Where ending an item costs a
// block about as much as E tiles, the line has E more places behind each
// item's tiles, at which there is nothing to do.) There is no softmax, so an
// item that several blocks share is their plain sum: each writes its part (32
// bits) to the workspace and a second, small launch adds the parts in line
// order -- no atomics, the same bits on every run. Every block finds its part
// by itself: a scan over the B sequence lengths, which costs it about a
// microsecond and saves a planning launch; it leaves what it found (a
// PartHead) for the join.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace hstu {

// x / (1 + exp(-x)) by exp2 and a reciprocal, both to a few units in the last
// place of 32 bits. (The approximate tanh of the dense forward is off by more
// than a bf16 step of silu for scores below about -3.) Very negative x: the
// exponential overflows to infinity, its reciprocal is 0.
__device__ __forceinline__ float silu_exp(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return x * r;
}

// Byte offset of the bucket floor(log2(max(1, dt))) in a table of floats that
// starts kBucketBias bytes earlier: the exponent of dt as a float, rounded
// towards zero so that it never carries into the next power of two.
constexpr int kBucketBias = 127 * 4;
__device__ __forceinline__ uint32_t bucket_bytes(int dt) {
    return (__float_as_uint(__int2float_rz(max(dt, 1))) >> 21) & 0x7fcu;
}
__device__ __forceinline__ float table_at(const float* base, uint32_t bytes) {
    return *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(base) + bytes);
}

constexpr int kMaxTree = 256;       // new tokens of a sequence that come as a tree

struct CachedArgs {
    // queries: the new tokens
    const void* q;                  // [T, H, dqk]
    int64_t q_stride;
    const int64_t* ts;              // [T] or null
    const int32_t* parents;         // [T] or null (each sequence a chain)
    void* out;                      // [T, H, dv]
    int64_t out_stride;
    // the cache
    const void* k;
    const void* v;
    int64_t k_page, k_tok, v_page, v_tok;       // elements
    const int64_t* tsc;             // null without the time term
    int64_t tsc_page;
    int num_pages, shift;           // page_size = 1 << shift
    const int32_t* table;           // [B, max_pages]
    int64_t table_stride;
    int max_pages;
    // the batch
    const int32_t* ctx;             // [B]
    const int64_t* off;             // [B + 1]
    int B;
    int64_t T;
    int max_new, max_seqlen;
    int H, dqk, dv;
    const float* pos;
    int P;
    const float* tb;
    int NB;
    float inv_n;
    struct PartHead* heads;         // workspace: one a block
    float* parts;                   // then two parts a block
    int part_rows;                  // of part_rows x dv floats each
};

// What block c found at the start of its part of the line: the item there.
struct alignas(16) PartHead {
    int64_t total;                  // the line's length
    int64_t start;                  // where the item starts
    int64_t row;                    // its first row of q and out
    int32_t tiles;                  // its key tiles; 0: no item starts or goes on here
    int32_t rows, h, pad;
};

struct CachedSeq {
    int64_t off;
    int ctx, n;                     // n == 0: nothing to do
};

// Sequence b's numbers. A sequence that cannot be (negative lengths, offsets
// outside [0, T], more new tokens than max_new or a tree's limit, longer than
// max_seqlen or than a table row) is left out, `ok` false.
__device__ __forceinline__ CachedSeq cached_seq(const CachedArgs& a, int b, bool& ok) {
    const int64_t o = a.off[b], e = a.off[b + 1];
    const int64_t c = a.ctx[b], n = e - o;
    const int64_t room = static_cast<int64_t>(a.max_pages) << a.shift;
    ok = c >= 0 && o >= 0 && n >= 0 && e <= a.T && n <= a.max_new && c + n <= a.max_seqlen &&
         c + n <= room;
    CachedSeq s;
    s.off = o;
    s.ctx = ok ? static_cast<int>(c) : 0;
    s.n = ok ? static_cast<int>(n) : 0;
    return s;
}

// Position on the line.
struct LineAt {
    int b, qt, h, j;                // j: key tile within the item (from its tiles on: none)
    CachedSeq s;
};

// Where block c's part of a line begins (0 <= c <= blocks < 1024). Short lines
// spare the 64-bit division.
__device__ __forceinline__ int64_t line_cut(int64_t total, int c, int blocks) {
    if (total < (1 << 22))
        return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(blocks);
    return total * c / blocks;
}

template <int KT, int NQ, int E = 0>
struct Line {
    static __device__ __forceinline__ int tiles(const CachedSeq& s, int qt) {
        return (s.ctx + min(s.n, (qt + 1) * NQ) + KT - 1) / KT;
    }
    // places of one head of sequence s
    static __device__ __forceinline__ int64_t per_head(const CachedSeq& s) {
        int64_t w = 0;
        for (int qt = 0; qt * NQ < s.n; ++qt) w += tiles(s, qt) + E;
        return w;
    }
    static __device__ __forceinline__ int64_t cut(int64_t total, int c, int blocks) {
        return line_cut(total, c, blocks);
    }

    // Block-wide: finds the line's length and the position of cut c. THREADS
    // threads; `scratch` holds THREADS / 32 + 8 int64. Returns the length.
    template <int THREADS>
    static __device__ int64_t locate(const CachedArgs& a, int c, int blocks, int64_t* scratch,
                                     LineAt& at, bool report) {
        const int tid = threadIdx.x;
        const int chunk = (a.B + THREADS - 1) / THREADS;
        const int b0 = min(tid * chunk, a.B), b1 = min(b0 + chunk, a.B);
        int64_t mine = 0;
        bool all_ok = true;
        for (int b = b0; b < b1; ++b) {
            bool ok;
            const CachedSeq s = cached_seq(a, b, ok);
            all_ok = all_ok && ok && (b > 0 || s.off == 0);
            mine += per_head(s) * a.H;
        }
        if (report && !all_ok) raise_error(kErrBadInput);
        int64_t scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
            if ((tid & 31) >= o) scan += v;
        }
        if ((tid & 31) == 31) scratch[tid >> 5] = scan;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (tid >> 5)) scan += scratch[w];
            total += scratch[w];
        }
        const int64_t x = cut(total, c, blocks);
        int64_t lo = scan - mine;
        if (x >= lo && x < scan) {          // exactly one thread, when x < total
            int b = b0;
            CachedSeq s;
            int64_t w;
            while (true) {
                bool ok;
                s = cached_seq(a, b, ok);
                w = per_head(s) * a.H;
                if (x < lo + w) break;
                lo += w;
                ++b;
            }
            int64_t r = x - lo;
            int qt = 0;
            while (r >= static_cast<int64_t>(tiles(s, qt) + E) * a.H) {
                r -= static_cast<int64_t>(tiles(s, qt) + E) * a.H;
                ++qt;
            }
            const int nt = tiles(s, qt) + E;
            int64_t* f = scratch + THREADS / 32;
            f[0] = b;
            f[1] = qt;
            f[2] = static_cast<uint32_t>(r) / static_cast<uint32_t>(nt);   // r < tiles * H < 2^32
            f[3] = static_cast<uint32_t>(r) % static_cast<uint32_t>(nt);
            f[4] = s.off;
            f[5] = s.ctx;
            f[6] = s.n;
        }
        __syncthreads();
        if (x < total) {
            const int64_t* f = scratch + THREADS / 32;
            at.b = static_cast<int>(f[0]);
            at.qt = static_cast<int>(f[1]);
            at.h = static_cast<int>(f[2]);
            at.j = static_cast<int>(f[3]);
            at.s.off = f[4];
            at.s.ctx = static_cast<int>(f[5]);
            at.s.n = static_cast<int>(f[6]);
        }
        return total;
    }

    // The item after at's.
    static __device__ __forceinline__ void next_item(const CachedArgs& a, LineAt& at) {
        at.j = 0;
        if (++at.h < a.H) return;
        at.h = 0;
        if (++at.qt * NQ < at.s.n) return;
        at.qt = 0;
        do {
            if (++at.b >= a.B) return;
            bool ok;
            at.s = cached_seq(a, at.b, ok);
        } while (at.s.n == 0);
    }
};

// Called by one thread of every block, also of those without work.
template <int KT, int NQ, int E = 0>
__device__ __forceinline__ void write_head(const CachedArgs& a, const LineAt& at, int64_t total,
                                           int64_t begin) {
    PartHead p;
    p.total = total;
    p.tiles = 0;
    if (begin < total) {
        p.start = begin - at.j;
        p.row = at.s.off + at.qt * NQ;
        p.tiles = Line<KT, NQ, E>::tiles(at.s, at.qt);
        if (at.j >= p.tiles) p.tiles = 0;
        p.rows = min(NQ, at.s.n - at.qt * NQ);
        p.h = at.h;
    }
    a.heads[blockIdx.x] = p;
}

__device__ __forceinline__ void store_out(float* dst, const float (&v)[1], float f) { *dst = v[0] * f; }
__device__ __forceinline__ void store_out(__nv_bfloat16* dst, const float (&v)[4], float f) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0] * f, v[1] * f),
                                                pack_bf16x2(v[2] * f, v[3] * f));
}

// Parts: block c's first item at 2c, its last (when that is another) at 2c + 1,
// part_rows * dv floats each. An item is shared where a cut lies strictly behind its
// first tile; the first such cut stands for it. Every block of the join reads
// all heads at once and lists the shared items, those of up to kJoinFew parts
// and those of more, and takes every gridDim-th unit of work: of the former
// 32 V values a warp, of the latter 32 V values, of which each warp adds an
// eighth of the parts and one the eight sums. The order of the sums is fixed
// by the lengths.
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kJoinBlocks = 6 * 148;
constexpr int kJoinFew = 6;

// An item as the units of the join need it.
struct JoinItem {
    int64_t row;                                // first row of out
    int32_t c, parts;                           // the parts are those of blocks c - 1 ..
    int32_t first;                              // index of the part of block c - 1
    int32_t rows, h;
};

// E: as the line's.
template <int V, typename TOut, int BLOCKS, int E>
__global__ void __launch_bounds__(kJoinThreads) attn_cached_join_kernel(const CachedArgs a) {
    __shared__ JoinItem items[BLOCKS];          // few parts from the front, many from the back
    __shared__ int warp_n[2][kJoinWarps];
    __shared__ float sums[kJoinWarps][32 * V];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t total = a.heads[0].total;
    int n[2] = {0, 0};
    for (int c0 = 1; c0 < BLOCKS; c0 += kJoinThreads) {
        const int c = c0 + tid;
        bool is = false, many = false;
        JoinItem item;
        if (c < BLOCKS) {
            const PartHead p = a.heads[c];
            const int64_t before = line_cut(total, c - 1, BLOCKS);
            is = p.tiles > 0 && line_cut(total, c, BLOCKS) != p.start && before <= p.start;
            if (is) {
                // the last block whose part begins inside; c - 1's part is its last
                // item's, its first one's when it begins with this item (or in the
                // empty places right before it)
                const int64_t end = (p.start + p.tiles) * BLOCKS - 1;
                const int last = total < (1 << 20) ? static_cast<uint32_t>(end) / static_cast<uint32_t>(total)
                                                   : static_cast<int>(end / total);
                item.row = p.row;
                item.c = c;
                item.parts = min(BLOCKS - 1, last) - c + 2;
                item.first = 2 * (c - 1) + (before + E < p.start ? 1 : 0);
                item.rows = p.rows;
                item.h = p.h;
                many = item.parts > kJoinFew;
            }
        }
        const uint32_t m[2] = {__ballot_sync(0xffffffffu, is && !many),
                               __ballot_sync(0xffffffffu, many)};
        if (BLOCKS > kJoinThreads) __syncthreads();
        if (lane < 2) warp_n[lane][warp] = __popc(m[lane]);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            int at = n[k];
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                if (w < warp) at += warp_n[k][w];
                n[k] += warp_n[k][w];
            }
            at += __popc(m[k] & ((1u << lane) - 1u));
            if (is && many == (k == 1)) items[k == 0 ? at : BLOCKS - 1 - at] = item;
        }
    }
    __syncthreads();
    const int values = a.part_rows * a.dv;
    const int per_few = (values + kJoinThreads * V - 1) / (kJoinThreads * V);
    const int per_many = (values + 32 * V - 1) / (32 * V);
    const int few_units = n[0] * per_few, units = few_units + n[1] * per_many;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const bool many = u >= few_units;
        const int x = many ? u - few_units : u, per = many ? per_many : per_few;
        const int at = x / per, piece = x - at * per;
        const JoinItem& p = items[many ? BLOCKS - 1 - at : at];
        const int i = (many ? piece * 32 + lane : piece * kJoinThreads + tid) * V;
        const bool live = i < p.rows * a.dv;
        const int q0 = many ? p.parts * warp / kJoinWarps : 0;
        const int q1 = many ? p.parts * (warp + 1) / kJoinWarps : p.parts;
        float v[V] = {};
        const float* src = a.parts + i;
#pragma unroll 4
        for (int q = q0; q < q1; ++q) {
            // (with fewer tiles than blocks some blocks have none)
            const int b = p.c - 1 + q;
            const bool has = live && (total >= BLOCKS ||
                                      line_cut(total, b, BLOCKS) < line_cut(total, b + 1, BLOCKS));
            const float* s = src + static_cast<int64_t>(q == 0 ? p.first : 2 * b) * values;
            if constexpr (V == 4) {
                const float4 f = has ? *reinterpret_cast<const float4*>(s) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            } else {
                v[0] += has ? *s : 0.f;
            }
        }
        if (many) {
            __syncthreads();                // the previous unit's sums have been read
#pragma unroll
            for (int e = 0; e < V; ++e) sums[warp][lane * V + e] = v[e];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] += sums[w][lane * V + e];
            }
        }
        if (live && (!many || warp == 0)) {
            const int r = i / a.dv;
            store_out(static_cast<TOut*>(a.out) + (p.row + r) * a.out_stride +
                          static_cast<int64_t>(p.h) * a.dv + (i - r * a.dv),
                      v, a.inv_n);
        }
    }
}

// ------------------------------------------------------------------ the tree

// Who sees whom among a sequence's new tokens (word w of key m: which of the
// queries 32w .. 32w + 31 see m) and the depth of every new token.
struct alignas(16) TreeSmem {
    uint32_t seen[kMaxTree / 32][kMaxTree];     // [query / 32][key]: bit of the query
    int16_t depth[kMaxTree];
    int16_t parent[kMaxTree];
};

// Built by `nt` threads (index t), which `sync` holds together; a parent that
// is not before its token is an error and counts as -1.
template <typename Sync>
__device__ __forceinline__ void build_tree(const CachedArgs& a, const CachedSeq& s, TreeSmem& tree,
                                           int t, int nt, Sync sync) {
    sync();                                     // the previous tree is no longer read
    const int words = (s.n + 31) / 32;
    for (int m = t; m < s.n; m += nt) {
        const int p = a.parents[s.off + m];
        const bool ok = p >= -1 && p < m;
        if (!ok) raise_error(kErrBadInput);
        tree.parent[m] = static_cast<int16_t>(ok ? p : -1);
        for (int w = 0; w < words; ++w) tree.seen[w][m] = 0u;
    }
    sync();
    for (int m = t; m < s.n; m += nt) {
        int d = -1;
        for (int p = m; p >= 0; p = tree.parent[p]) {   // parents are smaller: ends
            atomicOr(&tree.seen[m >> 5][p], 1u << (m & 31));
            ++d;
        }
        tree.depth[m] = static_cast<int16_t>(d);
    }
    sync();
}

// The weight of one key for one query, alone, from global memory: for the rare
// keys whose values are not finite while some query of their tile does not see
// them. Kept out of line, like all that only they need.
template <int D>
__device__ __noinline__ float odd_weight(const CachedArgs& a, int h, int64_t qrow, int pq, int page,
                                         int row, int pk) {
    const int64_t hd = static_cast<int64_t>(h) * D;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + qrow * a.q_stride + hd;
    const __nv_bfloat16* k =
        static_cast<const __nv_bfloat16*>(a.k) + page * a.k_page + row * a.k_tok + hd;
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(q[c]), __bfloat162float(k[c]), s);
    if (a.pos) s += a.pos[static_cast<int64_t>(h) * a.P + min(pq - pk, a.P - 1)];
    if (a.tsc)
        s += a.tb[static_cast<int64_t>(h) * a.NB +
                  time_bucket64(a.ts[qrow] - a.tsc[page * a.tsc_page + row], a.NB - 1)];
    return silu_exp(s);
}

}  // namespace hstu
