// cache_api.cuh -- host side of the serving entry points: the paged cache
// (plan, append, attention over it) and projections with 4-bit weights.
// Included once, by hstu_api.cu, after its helpers.
#pragma once

#include "attn_cached.cuh"
#include "attn_cached_mma.cuh"
#include "attn_cached_simt.cuh"
#include "attn_cached_tc.cuh"
#include "cache_plan.cuh"
#include "linear_w4.cuh"

namespace {

// log2 of a supported page size, -1 otherwise
int page_shift(int32_t page_size) {
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// Addresses of arrays of `bytes`-byte elements (null counts as aligned).
template <typename... P>
bool aligned_to(uintptr_t bytes, const P*... p) {
    return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t{0}) & (bytes - 1)) == 0;
}

bool cache_size_ok(int32_t num_pages, int32_t page_size) {
    return num_pages >= 1 && page_size >= 1 &&
           static_cast<int64_t>(num_pages) * page_size <= 0x7fffffff;
}

hstu_status_t validate_cached(hstu_dtype_t dtype, const CachedArgs& c, int32_t page_size,
                              const void* ws, size_t ws_bytes, size_t need) {
    if (c.B < 0 || c.T < 0 || c.T > 0x7fffffff || c.H < 1 || c.dqk < 1 || c.dv < 1 ||
        c.max_new < 1 || c.max_seqlen < 1 || c.max_seqlen > kMaxSeqlen || c.max_pages < 1)
        return HSTU_ERR_INVALID_ARG;
    if (dtype != HSTU_DTYPE_F32 && dtype != HSTU_DTYPE_BF16) return HSTU_ERR_INVALID_ARG;
    if (c.shift < 0) return HSTU_ERR_UNSUPPORTED;
    if (!cache_size_ok(c.num_pages, page_size)) return HSTU_ERR_INVALID_ARG;
    if (c.pos && c.P < 1) return HSTU_ERR_INVALID_ARG;
    if (c.tb && (c.NB < 1 || c.NB > kMaxTimeBuckets)) return HSTU_ERR_INVALID_ARG;
    if (c.parents && c.max_new > kMaxTree) return HSTU_ERR_UNSUPPORTED;
    if (c.H > 65535) return HSTU_ERR_UNSUPPORTED;
    if (dtype == HSTU_DTYPE_BF16) {
        if (c.dqk != c.dv || (c.dqk != 32 && c.dqk != 64 && c.dqk != 128))
            return HSTU_ERR_UNSUPPORTED;
    } else if (c.dqk > 128 || c.dv > 128) {
        return HSTU_ERR_UNSUPPORTED;
    }
    if (c.B == 0 || c.T == 0) return HSTU_OK;
    const int64_t rq = static_cast<int64_t>(c.H) * c.dqk, rv = static_cast<int64_t>(c.H) * c.dv;
    if (!c.q || !c.k || !c.v || !c.out || !c.table || !c.ctx || !c.off) return HSTU_ERR_INVALID_ARG;
    if (c.q_stride < rq || c.out_stride < rv || c.k_tok < rq || c.v_tok < rv ||
        c.table_stride < c.max_pages)
        return HSTU_ERR_INVALID_ARG;
    if (c.k_page < (page_size - 1) * c.k_tok + rq || c.v_page < (page_size - 1) * c.v_tok + rv)
        return HSTU_ERR_INVALID_ARG;
    if (c.tsc && (c.tsc_page < page_size || reinterpret_cast<uintptr_t>(c.tsc) % 8))
        return HSTU_ERR_INVALID_ARG;
    if (!aligned_to(8, c.off, c.ts) || !aligned_to(4, c.table, c.ctx, c.parents, c.pos, c.tb) ||
        (dtype == HSTU_DTYPE_F32 && !aligned_to(4, c.q, c.k, c.v, c.out)))
        return HSTU_ERR_INVALID_ARG;
    if (dtype == HSTU_DTYPE_BF16) {
        if (!aligned16(c.q) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(c.out))
            return HSTU_ERR_INVALID_ARG;
        if (c.q_stride % 8 || c.out_stride % 8 || c.k_tok % 8 || c.v_tok % 8 || c.k_page % 8 ||
            c.v_page % 8)
            return HSTU_ERR_INVALID_ARG;
    }
    if (!ws || !aligned16(ws) || ws_bytes < need) return HSTU_ERR_INVALID_ARG;
    return HSTU_OK;
}

// The join of parts, as a programmatic dependent of the attention launch.
template <int V, typename TOut, int BLOCKS, int E = 0>
hstu_status_t launch_join(const CachedArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_cached_join_kernel<V, TOut, BLOCKS, E>, a);
    return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

template <int DMAX, int R, bool VEC>
hstu_status_t launch_cached_simt(const CachedArgs& a, cudaStream_t stream) {
    static int done[kMaxDevices] = {0};
    constexpr int smem = static_cast<int>(sizeof(CachedSimtSmem<DMAX, R>));
    if (!ensure_smem(attn_cached_simt_kernel<DMAX, R, VEC>, smem, done)) return HSTU_ERR_CUDA;
    attn_cached_simt_kernel<DMAX, R, VEC><<<kSimtBlocks, kSimtThreads, smem, stream>>>(a);
    const hstu_status_t st = launch_status();
    return st == HSTU_OK ? launch_join<1, float, kSimtBlocks>(a, stream) : st;
}

template <int DMAX, bool VEC>
hstu_status_t run_cached_simt_rows(const CachedArgs& a, cudaStream_t stream) {
    return a.max_new <= 8 ? launch_cached_simt<DMAX, 8, VEC>(a, stream)
                          : launch_cached_simt<DMAX, 16, VEC>(a, stream);
}

template <bool VEC>
hstu_status_t run_cached_simt(const CachedArgs& a, cudaStream_t stream) {
    const int d = a.dqk > a.dv ? a.dqk : a.dv;
    if (d <= 32) return run_cached_simt_rows<32, VEC>(a, stream);
    if (d <= 64) return run_cached_simt_rows<64, VEC>(a, stream);
    return run_cached_simt_rows<128, VEC>(a, stream);
}

// bf16 [pages, page_size, H d] of a cache, boxes of `rows` tokens x 64 (32) columns.
bool make_tmap_cache(CUtensorMap* tm, const void* base, const CachedArgs& a, int64_t page,
                     int64_t tok, int rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const int d = a.dqk;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.H) * d, cuuint64_t{1} << a.shift,
                          static_cast<cuuint64_t>(a.num_pages)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(tok) * 2, static_cast<cuuint64_t>(page) * 2};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(d >= 64 ? 64 : 32),
                         static_cast<cuuint32_t>(rows), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          d >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

constexpr int kMmaBlocks = 148;
// Sequences are taken whole, a block each, where they are short enough: up to
// 256 tokens always, up to 1024 when the items fill the device twice. (Heads of
// 128, one new token, four heads: 128 sequences of 256 take 22 us whole and 33
// along the line, of 1024 50 and 52; one sequence of 1000 26 and 15.)
constexpr int kWholeLen = 256, kWholeLenFull = 1024;

template <int D, int NT, bool WHOLE>
hstu_status_t launch_cached_mma(const CachedArgs& a, int64_t items, cudaStream_t stream) {
    using S = CachedMmaSmem<D, NT, WHOLE>;
    static int done[kMaxDevices] = {0};
    CUtensorMap tk, tv;
    if (!make_tmap_cache(&tk, a.k, a, a.k_page, a.k_tok, kMmaKeys) ||
        !make_tmap_cache(&tv, a.v, a, a.v_page, a.v_tok, kMmaKeys) ||
        !ensure_smem(attn_cached_mma_kernel<D, NT, WHOLE>, S::kAlloc, done))
        return HSTU_ERR_CUDA;
    attn_cached_mma_kernel<D, NT, WHOLE>
        <<<WHOLE ? static_cast<unsigned>(items) : kMmaBlocks, S::kThreads, S::kAlloc, stream>>>(
            tk, tv, a, (a.max_new + 8 * NT - 1) / (8 * NT));
    const hstu_status_t st = launch_status();
    if (WHOLE || st != HSTU_OK) return st;
    return launch_join<4, __nv_bfloat16, kMmaBlocks>(a, stream);
}

template <int D, int NQ>
hstu_status_t launch_cached_tc(const CachedArgs& a, cudaStream_t stream) {
    using S = CachedTcSmem<D, NQ>;
    static int done[kMaxDevices] = {0};
    CUtensorMap tq, tk, tv;
    const int page = 1 << a.shift, rows = page < kTcKeys ? page : kTcKeys;
    if (!make_tmap_cache(&tk, a.k, a, a.k_page, a.k_tok, rows) ||
        !make_tmap_cache(&tv, a.v, a, a.v_page, a.v_tok, rows) ||
        !make_tmap_bf16(&tq, a.q, static_cast<uint64_t>(a.H) * D, a.T, a.q_stride * 2, NQ))
        return HSTU_ERR_CUDA;
    if (!ensure_smem(attn_cached_tc_kernel<D, NQ>, S::kAlloc, done)) return HSTU_ERR_CUDA;
    attn_cached_tc_kernel<D, NQ><<<kMmaBlocks, kTcThreads, S::kAlloc, stream>>>(tq, tk, tv, a);
    const hstu_status_t st = launch_status();
    return st == HSTU_OK ? launch_join<4, __nv_bfloat16, kMmaBlocks, kTcEnd>(a, stream) : st;
}

// Rows of a part: the most that an item of the kernels below can have.
int cached_part_rows(hstu_dtype_t dtype, int32_t max_new, int32_t d) {
    const int most = dtype == HSTU_DTYPE_F32 ? 16 : d == 32 ? 32 : 128;
    return max_new >= most ? most : (max_new + 7) / 8 * 8;
}

// Items of query tiles of `rows` where every sequence may be taken whole, else 0.
int64_t cached_whole_items(const CachedArgs& a, int rows) {
    const int64_t items = static_cast<int64_t>(a.B) * ((a.max_new + rows - 1) / rows) * a.H;
    const bool whole = a.max_seqlen <= kWholeLen ||
                       (a.max_seqlen <= kWholeLenFull && items >= 2 * kMmaBlocks);
    return whole && items <= 0x7fffffff ? items : 0;
}

// Heads of 64 and 128: the tcgen05 kernel, but for up to eight new tokens over
// sequences that are taken whole, and up to sixteen over those of up to 256
// tokens. (300 sequences of 200, 12 new tokens, 2 heads of 128: 34 us against
// 43, 4 of 64: 36 and 61; of 900, 16 new tokens, heads of 128: 61 and 46.)
template <int D>
hstu_status_t run_cached_bf16(const CachedArgs& a, cudaStream_t stream) {
    const int64_t items = cached_whole_items(a, a.max_new <= 8 ? 8 : 16);
    if (a.max_new <= 8 && items) return launch_cached_mma<D, 1, true>(a, items, stream);
    if (a.max_new <= 16 && a.max_seqlen <= kWholeLen && items)
        return launch_cached_mma<D, 2, true>(a, items, stream);
    return a.max_new <= 64 ? launch_cached_tc<D, 64>(a, stream) : launch_cached_tc<D, 128>(a, stream);
}

template <int NT>
hstu_status_t run_cached_bf16_d32(const CachedArgs& a, cudaStream_t stream) {
    const int64_t items = cached_whole_items(a, 8 * NT);
    return items ? launch_cached_mma<32, NT, true>(a, items, stream)
                 : launch_cached_mma<32, NT, false>(a, 0, stream);
}

template <>
hstu_status_t run_cached_bf16<32>(const CachedArgs& a, cudaStream_t stream) {
    return a.max_new <= 8    ? run_cached_bf16_d32<1>(a, stream)
           : a.max_new <= 16 ? run_cached_bf16_d32<2>(a, stream)
                             : run_cached_bf16_d32<4>(a, stream);
}

template <int MT, int NT, int G>
hstu_status_t launch_linear_w4(const LinearW4Args& a, int warps, cudaStream_t stream) {
    static int done[kMaxDevices] = {0};
    constexpr int ring = kW4Stages * w4_stage_bytes<MT>(), sums = 16 * MT * 8 * NT * 4;
    constexpr int per_warp = ring > sums ? ring : sums;
    if (!ensure_smem(linear_w4_kernel<MT, NT, G>, 8 * per_warp, done)) return HSTU_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>((a.N + 16 * MT - 1) / (16 * MT)),
                    static_cast<unsigned>((a.M + 8 * NT - 1) / (8 * NT)));
    linear_w4_kernel<MT, NT, G><<<grid, warps * 32, warps * per_warp, stream>>>(a);
    return launch_status();
}

template <int MT, int NT>
hstu_status_t launch_linear_w4_g(const LinearW4Args& a, int warps, cudaStream_t stream) {
    if (a.G == 32) return launch_linear_w4<MT, NT, 32>(a, warps, stream);
    if (a.G == 64) return launch_linear_w4<MT, NT, 64>(a, warps, stream);
    return launch_linear_w4<MT, NT, 128>(a, warps, stream);
}

// Two row tiles of W a block where they still fill the device twice (x is read
// half as often), else one; K split over at most eight warps. More than 32 rows
// of x: blocks of 64 and two row tiles where K is long enough to hide their start
// and their waves leave at most a third of the SMs idle (64 rows, us, that and
// blocks of 32: 4096 x 4096 19.5 and 21.5, 2048 x 8192 23.0 and 25.5; but 512 x
// 4096 9.7 and 7.2, 2048 x 6000 22.5 and 20.5, 8192 x 2048 31 and 19.5).
hstu_status_t run_linear_w4(const LinearW4Args& a, cudaStream_t stream) {
    const int nkb = a.K / 128;
    const bool wide = a.N >= 2 * 148 * 32;
    const int most = wide ? 4 : 8, warps = nkb < most ? nkb : most;
    const int64_t blocks = (static_cast<int64_t>(a.N) + 31) / 32 * ((a.M + 63) / 64);
    const bool tall = a.M > 32 && nkb >= 8 && (blocks + 147) / 148 * 148 * 2 <= blocks * 3;
    if (a.M <= 8)
        return wide ? launch_linear_w4_g<2, 1>(a, warps, stream)
                    : launch_linear_w4_g<1, 1>(a, warps, stream);
    if (a.M <= 16)
        return wide ? launch_linear_w4_g<2, 2>(a, warps, stream)
                    : launch_linear_w4_g<1, 2>(a, warps, stream);
    if (tall) return launch_linear_w4_g<2, 8>(a, warps, stream);
    return wide ? launch_linear_w4_g<2, 4>(a, warps, stream)
                : launch_linear_w4_g<1, 4>(a, warps, stream);
}

// Each of the calls below is in two parts, what it refuses and what it launches,
// so that the layer step refuses all its parts' arguments before the first launch.

// Checks an append (nothing to do where total_new is 0) and lays out its
// arguments; `mix`: every address and length in bytes, or-ed.
hstu_status_t make_append(hstu_dtype_t dtype, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int64_t* timestamps, const int64_t* slots,
                          int64_t total_new, int32_t H, int32_t d_qk, int32_t d_v, void* k_cache,
                          int64_t k_page_stride, int64_t k_tok_stride, void* v_cache,
                          int64_t v_page_stride, int64_t v_tok_stride, int64_t* ts_cache,
                          int64_t ts_page_stride, int32_t num_pages, int32_t page_size,
                          CacheAppendArgs& a, uint64_t& mix) {
    if (dtype != HSTU_DTYPE_F32 && dtype != HSTU_DTYPE_BF16) return HSTU_ERR_INVALID_ARG;
    if (total_new < 0 || H < 1 || d_qk < 1 || d_v < 1) return HSTU_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0) return HSTU_ERR_UNSUPPORTED;
    if (!cache_size_ok(num_pages, page_size)) return HSTU_ERR_INVALID_ARG;
    const int64_t rk = static_cast<int64_t>(H) * d_qk, rv = static_cast<int64_t>(H) * d_v;
    if (rk > (1 << 28) || rv > (1 << 28)) return HSTU_ERR_UNSUPPORTED;
    if (k_tok_stride < rk || v_tok_stride < rv ||
        k_page_stride < (page_size - 1) * k_tok_stride + rk ||
        v_page_stride < (page_size - 1) * v_tok_stride + rv)
        return HSTU_ERR_INVALID_ARG;
    if ((timestamps == nullptr) != (ts_cache == nullptr)) return HSTU_ERR_INVALID_ARG;
    if (ts_cache && (ts_page_stride < page_size || reinterpret_cast<uintptr_t>(ts_cache) % 8))
        return HSTU_ERR_INVALID_ARG;
    if (total_new == 0) return HSTU_OK;
    if (!k || !v || !slots || !k_cache || !v_cache) return HSTU_ERR_INVALID_ARG;
    if (total_new > 1 && (k_stride < rk || v_stride < rv)) return HSTU_ERR_INVALID_ARG;
    const int e = dtype == HSTU_DTYPE_BF16 ? 2 : 4;
    a = {static_cast<const uint8_t*>(k), static_cast<const uint8_t*>(v), k_stride * e, v_stride * e,
         static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_page_stride * e,
         k_tok_stride * e, v_page_stride * e, v_tok_stride * e, static_cast<int>(rk * e),
         static_cast<int>(rv * e), timestamps, ts_cache, ts_page_stride, slots, total_new,
         static_cast<int64_t>(num_pages) * page_size, shift};
    mix = reinterpret_cast<uint64_t>(k) | reinterpret_cast<uint64_t>(v) |
          reinterpret_cast<uint64_t>(k_cache) | reinterpret_cast<uint64_t>(v_cache) | a.k_stride |
          a.v_stride | a.kc_page | a.kc_tok | a.vc_page | a.vc_tok | a.k_bytes | a.v_bytes;
    return mix % e || !aligned_to(8, timestamps, slots) ? HSTU_ERR_INVALID_ARG : HSTU_OK;
}

hstu_status_t launch_append(const CacheAppendArgs& a, uint64_t mix, cudaStream_t s) {
    const int64_t blocks = (a.T + kAppendWarps - 1) / kAppendWarps;
    const unsigned grid = static_cast<unsigned>(blocks < 8 * 148 ? blocks : 8 * 148);
    if (mix % 16 == 0) cache_append_kernel<uint4><<<grid, kAppendWarps * 32, 0, s>>>(a);
    else if (mix % 4 == 0) cache_append_kernel<uint32_t><<<grid, kAppendWarps * 32, 0, s>>>(a);
    else cache_append_kernel<uint16_t><<<grid, kAppendWarps * 32, 0, s>>>(a);
    return launch_status();
}

// Checks a call of the attention (nothing to do without sequences or new tokens)
// and lays out its arguments.
hstu_status_t make_cached(hstu_dtype_t dtype, const void* q, int64_t q_tok_stride, const void* k_cache,
                          int64_t k_page_stride, int64_t k_tok_stride, const void* v_cache,
                          int64_t v_page_stride, int64_t v_tok_stride, const int64_t* ts_cache,
                          int64_t ts_page_stride, int32_t num_pages, int32_t page_size,
                          const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                          const int32_t* ctx_lens, const int64_t* new_offsets, int32_t B,
                          int64_t total_new, int32_t max_new, int32_t H, int32_t d_qk, int32_t d_v,
                          const int64_t* timestamps, const int32_t* parents, const float* pos_bias,
                          int32_t num_pos, const float* time_bias, int32_t num_time_buckets,
                          int32_t max_seqlen, void* out, int64_t out_tok_stride, void* workspace,
                          size_t workspace_bytes, CachedArgs& a) {
    const bool use_time = ts_cache && timestamps && time_bias;
    a = CachedArgs{};
    a.q = q;
    a.q_stride = q_tok_stride;
    a.ts = use_time ? timestamps : nullptr;
    a.parents = parents;
    a.out = out;
    a.out_stride = out_tok_stride;
    a.k = k_cache;
    a.v = v_cache;
    a.k_page = k_page_stride;
    a.k_tok = k_tok_stride;
    a.v_page = v_page_stride;
    a.v_tok = v_tok_stride;
    a.tsc = use_time ? ts_cache : nullptr;
    a.tsc_page = ts_page_stride;
    a.num_pages = num_pages;
    a.shift = page_shift(page_size);
    a.table = block_table;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.ctx = ctx_lens;
    a.off = new_offsets;
    a.B = B;
    a.T = total_new;
    a.max_new = max_new;
    a.max_seqlen = max_seqlen;
    a.H = H;
    a.dqk = d_qk;
    a.dv = d_v;
    a.pos = pos_bias;
    a.P = num_pos;
    a.tb = use_time ? time_bias : nullptr;
    a.NB = num_time_buckets;
    a.inv_n = 1.0f / static_cast<float>(max_seqlen);
    a.heads = static_cast<PartHead*>(workspace);
    a.parts = reinterpret_cast<float*>(a.heads + (dtype == HSTU_DTYPE_F32 ? kSimtBlocks : kMmaBlocks));
    a.part_rows = cached_part_rows(dtype, max_new, d_v);
    const hstu_status_t st = validate_cached(dtype, a, page_size, workspace, workspace_bytes,
                                             hstu_attn_cached_workspace_bytes(dtype, max_new, d_v));
    // No sequence brings more: a generous bound picks no other kernel, adds no
    // blocks and overflows no count of tiles.
    if (a.max_new > max_seqlen) a.max_new = max_seqlen;
    return st;
}

hstu_status_t launch_cached(hstu_dtype_t dtype, const CachedArgs& a, cudaStream_t s) {
    if (dtype == HSTU_DTYPE_BF16) {
        if (a.dqk == 32) return run_cached_bf16<32>(a, s);
        if (a.dqk == 64) return run_cached_bf16<64>(a, s);
        return run_cached_bf16<128>(a, s);
    }
    const bool vec = aligned16(a.k) && aligned16(a.v) && a.k_page % 4 == 0 && a.k_tok % 4 == 0 &&
                     a.v_page % 4 == 0 && a.v_tok % 4 == 0 && a.dqk % 4 == 0 && a.dv % 4 == 0;
    return vec ? run_cached_simt<true>(a, s) : run_cached_simt<false>(a, s);
}

// Checks a 4-bit projection (nothing to do where M is 0) and lays out its arguments.
hstu_status_t make_linear_w4(const void* x, int64_t ldx, int64_t M, int32_t K, const void* codes,
                             int64_t ldc, const void* scales, int64_t lds, int32_t group, int32_t N,
                             const float* bias, hstu_epilogue_t epilogue, const void* residual,
                             int64_t ldr, void* y, int64_t ldy, LinearW4Args& a) {
    if (M < 0 || K < 1 || N < 1) return HSTU_ERR_INVALID_ARG;
    if (epilogue != HSTU_EPI_NONE && epilogue != HSTU_EPI_SILU && epilogue != HSTU_EPI_RESIDUAL)
        return HSTU_ERR_INVALID_ARG;
    if ((group != 32 && group != 64 && group != 128) || K % 128 || M > 65535 * 8 || N > 0x7fffffff - 64)
        return HSTU_ERR_UNSUPPORTED;
    if (M == 0) return HSTU_OK;
    if (!x || !codes || !scales || !y || (epilogue == HSTU_EPI_RESIDUAL && !residual))
        return HSTU_ERR_INVALID_ARG;
    if (ldx < K || ldc < K / 2 || lds < K / group || ldy < N ||
        (epilogue == HSTU_EPI_RESIDUAL && ldr < N))
        return HSTU_ERR_INVALID_ARG;
    if (!aligned16(x) || ldx % 8 || !aligned16(codes) || ldc % 16) return HSTU_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(scales) % 2 || reinterpret_cast<uintptr_t>(y) % 2 ||
        reinterpret_cast<uintptr_t>(residual) % 2 || reinterpret_cast<uintptr_t>(bias) % 4)
        return HSTU_ERR_INVALID_ARG;
    a = {static_cast<const __nv_bfloat16*>(x), ldx, static_cast<int>(M), K, N, group,
         static_cast<const uint8_t*>(codes), ldc, static_cast<const __nv_bfloat16*>(scales), lds, bias,
         static_cast<const __nv_bfloat16*>(residual), ldr, static_cast<__nv_bfloat16*>(y), ldy,
         static_cast<int>(epilogue)};
    return HSTU_OK;
}

// workspace of a layer step: [LayerNorm(x)][U|V|Q|K][attention][gated rows][attention's own]
struct LayerStepWs {
    size_t xn, uvqk, attn, y, own, total;
};

LayerStepWs layer_step_ws(int64_t T, int32_t D, int32_t H, int32_t d, int32_t max_new) {
    const size_t t = static_cast<size_t>(T), F = static_cast<size_t>(H) * d;
    LayerStepWs w;
    w.xn = 0;
    w.uvqk = round_up(w.xn + t * D * 2, 256);
    w.attn = round_up(w.uvqk + t * 4 * F * 2, 256);
    w.y = round_up(w.attn + t * F * 2, 256);
    w.own = round_up(w.y + t * F * 2, 256);
    w.total = w.own + hstu_attn_cached_workspace_bytes(HSTU_DTYPE_BF16, max_new, d);
    return w;
}

bool layer_step_sizes_ok(int64_t T, int32_t D, int32_t H, int32_t d, int32_t max_new) {
    return T >= 0 && T <= 0x7fffffff && D >= 1 && H >= 1 && d >= 1 && max_new >= 1;
}

}  // namespace

extern "C" {

hstu_status_t hstu_cache_plan(const int32_t* ctx_lens, const int64_t* new_offsets, int32_t B,
                              int64_t total_new, int32_t page_size, const int32_t* free_pages,
                              int32_t num_free, const int32_t* free_start, int32_t* block_table,
                              int64_t table_stride, int32_t max_pages, int64_t* slots,
                              int32_t* free_end, void* stream) {
    if (B < 1 || total_new < 0 || total_new > 0x7fffffff || num_free < 0 || max_pages < 1 ||
        table_stride < max_pages)
        return HSTU_ERR_INVALID_ARG;
    const int shift = page_shift(page_size);
    if (shift < 0) return HSTU_ERR_UNSUPPORTED;
    if (!cache_size_ok(max_pages, page_size)) return HSTU_ERR_UNSUPPORTED;
    if (!ctx_lens || !new_offsets || !free_start || !block_table || !free_end || free_end == free_start ||
        (num_free > 0 && !free_pages) || (total_new > 0 && !slots))
        return HSTU_ERR_INVALID_ARG;
    if (!aligned_to(8, new_offsets, slots) ||
        !aligned_to(4, ctx_lens, free_pages, free_start, block_table, free_end))
        return HSTU_ERR_INVALID_ARG;
    CachePlanArgs a{ctx_lens, new_offsets, B, total_new, shift, free_pages, num_free, free_start,
                    block_table, table_stride, max_pages, slots, free_end, 1};
    // up to two blocks an SM over the sequences, then over each block's tokens
    const int64_t s = (static_cast<int64_t>(B) + 295) / 296;
    a.seqs_per_block = static_cast<int>(s > kPlanSeqs ? kPlanSeqs : s);
    const unsigned gx = static_cast<unsigned>((static_cast<int64_t>(B) + a.seqs_per_block - 1) /
                                              a.seqs_per_block);
    const int64_t per = (total_new / gx + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    const int64_t most = gx >= 296 ? 1 : 296 / gx;
    const unsigned gy = static_cast<unsigned>(per < 1 ? 1 : per < most ? per : most);
    cache_plan_kernel<<<dim3(gx, gy), kPlanThreads, 0, as_stream(stream)>>>(a);
    return launch_status();
}

hstu_status_t hstu_cache_append(hstu_dtype_t dtype, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int64_t* timestamps, const int64_t* slots,
                                int64_t total_new, int32_t H, int32_t d_qk, int32_t d_v,
                                void* k_cache, int64_t k_page_stride, int64_t k_tok_stride,
                                void* v_cache, int64_t v_page_stride, int64_t v_tok_stride,
                                int64_t* ts_cache, int64_t ts_page_stride, int32_t num_pages,
                                int32_t page_size, void* stream) {
    CacheAppendArgs a;
    uint64_t mix;
    const hstu_status_t st = make_append(dtype, k, k_stride, v, v_stride, timestamps, slots, total_new, H,
                                         d_qk, d_v, k_cache, k_page_stride, k_tok_stride, v_cache,
                                         v_page_stride, v_tok_stride, ts_cache, ts_page_stride,
                                         num_pages, page_size, a, mix);
    return st != HSTU_OK || total_new == 0 ? st : launch_append(a, mix, as_stream(stream));
}

size_t hstu_attn_cached_workspace_bytes(hstu_dtype_t dtype, int32_t max_new, int32_t d_v) {
    if ((dtype != HSTU_DTYPE_F32 && dtype != HSTU_DTYPE_BF16) || max_new < 1 || d_v < 1 ||
        d_v > 128)
        return 0;
    const size_t blocks = dtype == HSTU_DTYPE_F32 ? kSimtBlocks : kMmaBlocks;
    return blocks * (sizeof(PartHead) +
                     static_cast<size_t>(2) * cached_part_rows(dtype, max_new, d_v) * d_v * 4);
}

hstu_status_t hstu_attn_cached_fwd(hstu_dtype_t dtype, const void* q, int64_t q_tok_stride,
                                   const void* k_cache, int64_t k_page_stride,
                                   int64_t k_tok_stride, const void* v_cache,
                                   int64_t v_page_stride, int64_t v_tok_stride,
                                   const int64_t* ts_cache, int64_t ts_page_stride,
                                   int32_t num_pages, int32_t page_size,
                                   const int32_t* block_table, int64_t table_stride,
                                   int32_t max_pages, const int32_t* ctx_lens,
                                   const int64_t* new_offsets, int32_t B, int64_t total_new,
                                   int32_t max_new, int32_t H, int32_t d_qk, int32_t d_v,
                                   const int64_t* timestamps, const int32_t* parents,
                                   const float* pos_bias, int32_t num_pos, const float* time_bias,
                                   int32_t num_time_buckets, int32_t max_seqlen, void* out,
                                   int64_t out_tok_stride, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    CachedArgs a;
    const hstu_status_t st = make_cached(
        dtype, q, q_tok_stride, k_cache, k_page_stride, k_tok_stride, v_cache, v_page_stride,
        v_tok_stride, ts_cache, ts_page_stride, num_pages, page_size, block_table, table_stride,
        max_pages, ctx_lens, new_offsets, B, total_new, max_new, H, d_qk, d_v, timestamps, parents,
        pos_bias, num_pos, time_bias, num_time_buckets, max_seqlen, out, out_tok_stride, workspace,
        workspace_bytes, a);
    return st != HSTU_OK || B == 0 || total_new == 0 ? st : launch_cached(dtype, a, as_stream(stream));
}

hstu_status_t hstu_quant_groups_w4(const void* W, int64_t ldw, int64_t N, int32_t K, int32_t group,
                                   void* codes, int64_t ldc, void* scales, int64_t lds,
                                   void* stream) {
    if (N < 0 || K < 1) return HSTU_ERR_INVALID_ARG;
    if ((group != 32 && group != 64 && group != 128) || K % group) return HSTU_ERR_UNSUPPORTED;
    if (N == 0) return HSTU_OK;
    if (!W || !codes || !scales || ldw < K || ldc < K / 2 || lds < K / group)
        return HSTU_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(W) % 2 || reinterpret_cast<uintptr_t>(scales) % 2)
        return HSTU_ERR_INVALID_ARG;
    const QuantW4Args a{static_cast<const __nv_bfloat16*>(W), ldw, N, K,
                        static_cast<uint8_t*>(codes), ldc, static_cast<__nv_bfloat16*>(scales),
                        lds};
    const int64_t warps = (N * (K / group) * (group / (group == 128 ? 4 : 2)) + 31) / 32;
    const int64_t blocks = (warps + 7) / 8;
    const unsigned grid = static_cast<unsigned>(blocks < 16 * 148 ? blocks : 16 * 148);
    cudaStream_t s = as_stream(stream);
    if (group == 32) quant_w4_kernel<32><<<grid, 256, 0, s>>>(a);
    else if (group == 64) quant_w4_kernel<64><<<grid, 256, 0, s>>>(a);
    else quant_w4_kernel<128><<<grid, 256, 0, s>>>(a);
    return launch_status();
}

hstu_status_t hstu_linear_w4_fwd(const void* x, int64_t ldx, int64_t M, int32_t K, const void* codes,
                                 int64_t ldc, const void* scales, int64_t lds, int32_t group,
                                 int32_t N, const float* bias, hstu_epilogue_t epilogue,
                                 const void* residual, int64_t ldr, void* y, int64_t ldy,
                                 void* stream) {
    LinearW4Args a;
    const hstu_status_t st = make_linear_w4(x, ldx, M, K, codes, ldc, scales, lds, group, N, bias,
                                            epilogue, residual, ldr, y, ldy, a);
    return st != HSTU_OK || M == 0 ? st : run_linear_w4(a, as_stream(stream));
}

size_t hstu_layer_step_workspace_bytes(int64_t total_new, int32_t D, int32_t H, int32_t d,
                                       int32_t max_new) {
    if (!layer_step_sizes_ok(total_new, D, H, d, max_new) || (d != 64 && d != 128)) return 0;
    return layer_step_ws(total_new, D, H, d, max_new).total;
}

hstu_status_t hstu_layer_step_fwd(const void* x, int64_t total_new, int32_t D, const void* W1,
                                  const void* s1, const float* b1, const void* W2, const void* s2,
                                  const float* b2, int32_t w4_group, const float* ln_gamma,
                                  const float* ln_beta, float ln_eps, int32_t input_norm,
                                  const float* in_gamma, const float* in_beta, void* k_cache,
                                  int64_t k_page_stride, int64_t k_tok_stride, void* v_cache,
                                  int64_t v_page_stride, int64_t v_tok_stride, int64_t* ts_cache,
                                  int64_t ts_page_stride, int32_t num_pages, int32_t page_size,
                                  const int32_t* block_table, int64_t table_stride,
                                  int32_t max_pages, const int32_t* ctx_lens,
                                  const int64_t* new_offsets, int32_t B, const int64_t* slots,
                                  int32_t max_new, int32_t H, int32_t d, const int64_t* timestamps,
                                  const int32_t* parents, const float* pos_bias, int32_t num_pos,
                                  const float* time_bias, int32_t num_time_buckets,
                                  int32_t max_seqlen, void* out, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    const int64_t T = total_new;
    if (!layer_step_sizes_ok(T, D, H, d, max_new) || B < 0) return HSTU_ERR_INVALID_ARG;
    if (H > 65535 || (d != 64 && d != 128)) return HSTU_ERR_UNSUPPORTED;
    const int32_t F = H * d;
    if (D % 128 || F % 256 || F > 2048) return HSTU_ERR_UNSUPPORTED;
    if (input_norm && (D % 256 || D > 2048)) return HSTU_ERR_UNSUPPORTED;
    if (w4_group && w4_group != 32 && w4_group != 64 && w4_group != 128) return HSTU_ERR_UNSUPPORTED;
    if ((timestamps == nullptr) != (ts_cache == nullptr)) return HSTU_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return HSTU_OK;
    if (!x || !W1 || !W2 || !out || !slots || !workspace || (w4_group && (!s1 || !s2)))
        return HSTU_ERR_INVALID_ARG;
    const LayerStepWs w = layer_step_ws(T, D, H, d, max_new);
    if (workspace_bytes < w.total || !aligned16(workspace)) return HSTU_ERR_INVALID_ARG;
    cudaStream_t s = as_stream(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    __nv_bfloat16* uvqk = reinterpret_cast<__nv_bfloat16*>(ws + w.uvqk);
    __nv_bfloat16* attn = reinterpret_cast<__nv_bfloat16*>(ws + w.attn);
    __nv_bfloat16* ygate = reinterpret_cast<__nv_bfloat16*>(ws + w.y);
    // 1. [LayerNorm(x) ->] f1 with the SiLU epilogue
    // 2. the new keys and values into the cache, then the attention over it
    // 3. gate, f2 with the residual
    // All is checked before the first launch: a refused call leaves the cache as it was.
    const void* xin = input_norm ? ws + w.xn : x;
    CacheAppendArgs put;
    CachedArgs att;
    LinearW4Args f1, f2;
    uint64_t mix;
    hstu_status_t st = ln_eps >= 0.0f && aligned16(x) ? HSTU_OK : HSTU_ERR_INVALID_ARG;
    if (st == HSTU_OK)
        st = w4_group ? make_linear_w4(xin, D, T, D, W1, D / 2, s1, D / w4_group, w4_group, 4 * F, b1,
                                       HSTU_EPI_SILU, nullptr, 0, uvqk, 4 * F, f1)
                      : check_linear(false, xin, D, nullptr, T, D, W1, D, nullptr, 4 * F, HSTU_EPI_SILU,
                                     nullptr, 0, uvqk, 4 * F);
    if (st == HSTU_OK)
        st = make_append(HSTU_DTYPE_BF16, uvqk + 3 * F, 4 * F, uvqk + F, 4 * F, timestamps, slots, T, H, d,
                         d, k_cache, k_page_stride, k_tok_stride, v_cache, v_page_stride, v_tok_stride,
                         ts_cache, ts_page_stride, num_pages, page_size, put, mix);
    if (st == HSTU_OK)
        st = make_cached(HSTU_DTYPE_BF16, uvqk + 2 * F, 4 * F, k_cache, k_page_stride, k_tok_stride, v_cache,
                         v_page_stride, v_tok_stride, ts_cache, ts_page_stride, num_pages, page_size,
                         block_table, table_stride, max_pages, ctx_lens, new_offsets, B, T, max_new, H, d,
                         d, timestamps, parents, pos_bias, num_pos, time_bias, num_time_buckets,
                         max_seqlen, attn, F, ws + w.own, w.total - w.own, att);
    if (st == HSTU_OK)
        st = w4_group ? make_linear_w4(ygate, F, T, F, W2, F / 2, s2, F / w4_group, w4_group, D, b2,
                                       HSTU_EPI_RESIDUAL, x, D, out, D, f2)
                      : check_linear(false, ygate, F, nullptr, T, F, W2, F, nullptr, D, HSTU_EPI_RESIDUAL,
                                     x, D, out, D);
    if (st != HSTU_OK) return st;
    if (input_norm)
        st = run_ln_gate_any(false, false, x, D, nullptr, 0, T, D, in_gamma, in_beta, ln_eps, ws + w.xn, D,
                             nullptr, 0, nullptr, s);
    if (st == HSTU_OK)
        st = w4_group ? run_linear_w4(f1, s)
                      : run_linear(xin, D, T, D, W1, D, 4 * F, b1, HSTU_EPI_SILU, nullptr, 0, uvqk, 4 * F, s);
    if (st == HSTU_OK) st = launch_append(put, mix, s);
    if (st == HSTU_OK) st = launch_cached(HSTU_DTYPE_BF16, att, s);
    if (st == HSTU_OK)
        st = run_ln_gate(attn, F, uvqk, 4 * F, T, F, ln_gamma, ln_beta, ln_eps, ygate, F, s);
    if (st == HSTU_OK)
        st = w4_group ? run_linear_w4(f2, s)
                      : run_linear(ygate, F, T, F, W2, F, D, b2, HSTU_EPI_RESIDUAL, x, D, out, D, s);
    return st;
}

}  // extern "C"
