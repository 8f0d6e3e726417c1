// streaming.cuh -- host side of the streaming entry points (see
// include/vggt_attn.h): plan and append of the paged cache, attention over
// it, and the gated residual + norm.  Part of vggt_attn.cu, whose helpers it
// uses.
#pragma once

namespace {

bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

bool stride_ok(int64_t s, int64_t least)
{
    return s >= least && s % 8 == 0 && s < (int64_t{1} << 38);
}

// Elements from the first to behind the last of a strided [rows, heads, 64].
int64_t span(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride)
{
    return (rows - 1) * row_stride + (heads - 1) * head_stride + vggt::kHeadDim;
}

vggt_status check_tables(const vggt_cache &c)
{
    if (c.n_seqs < 1 || c.page_size < 1 || c.n_pages < 1 || c.max_pages < 1)
        return VGGT_ERR_INVALID_ARG;
    if (c.n_seqs > vggt::kCacheMaxSeqs || c.page_size % 8 != 0 ||
        static_cast<int64_t>(c.n_pages) * c.page_size > INT32_MAX ||
        static_cast<int64_t>(c.max_pages) * c.page_size > INT32_MAX - 1024)
        return VGGT_ERR_UNSUPPORTED;
    return VGGT_OK;
}

vggt_status check_cache(const vggt_cache &c)
{
    const vggt_status st = check_tables(c);
    if (st != VGGT_OK)
        return st;
    if (c.n_heads < 1 || c.n_kv_heads < 1 || c.n_heads % c.n_kv_heads != 0 || c.head_dim < 1)
        return VGGT_ERR_INVALID_ARG;
    if (c.head_dim != vggt::kHeadDim || c.n_heads > 64)
        return VGGT_ERR_UNSUPPORTED;
    if (!stride_ok(c.page_stride, vggt::kHeadDim) || !stride_ok(c.head_stride, vggt::kHeadDim) ||
        !stride_ok(c.token_stride, vggt::kHeadDim))
        return VGGT_ERR_INVALID_ARG;
    return VGGT_OK;
}

size_t pool_bytes(const vggt_cache &c)
{
    return 2 * static_cast<size_t>((c.n_pages - 1) * c.page_stride + (c.page_size - 1) * c.token_stride +
                                   (c.n_kv_heads - 1) * c.head_stride + vggt::kHeadDim);
}

vggt_status launched()
{
    return cudaGetLastError() == cudaSuccess ? VGGT_OK : VGGT_ERR_CUDA;
}

constexpr int64_t kFewAppendVecs = 1 << 20;

} // namespace

VGGT_API vggt_status vggt_cache_plan(vggt_cache cache, const int32_t *cached_lens, const int32_t *new_lens,
                                     const int32_t *free_pages, int32_t free_capacity, const int32_t *n_free,
                                     int32_t *block_table, int32_t n_rows, int32_t *cu_rows, int32_t *kv_lens,
                                     int32_t *slots, int32_t *counts, void *stream)
{
    vggt_status st = check_tables(cache);
    if (st != VGGT_OK)
        return st;
    if (n_rows < 0 || free_capacity < 0)
        return VGGT_ERR_INVALID_ARG;
    if (n_rows > INT32_MAX - 1024)
        return VGGT_ERR_UNSUPPORTED;
    const size_t B = static_cast<size_t>(cache.n_seqs);
    const void *in[4] = {cached_lens, new_lens, n_free, free_pages};
    const size_t in_bytes[4] = {4 * B, 4 * B, 4, 4 * static_cast<size_t>(free_capacity)};
    const void *out[5] = {block_table, cu_rows, kv_lens, counts, slots};
    const size_t out_bytes[5] = {4 * B * cache.max_pages, 4 * (B + 1), 4 * B, 8, 4 * static_cast<size_t>(n_rows)};
    for (int i = 0; i < 4; ++i)
        if ((!in[i] && in_bytes[i] > 0) || !aligned4(in[i]))
            return VGGT_ERR_INVALID_ARG;
    for (int i = 0; i < 5; ++i) {
        if ((!out[i] && out_bytes[i] > 0) || !aligned4(out[i]))
            return VGGT_ERR_INVALID_ARG;
        for (int j = 0; j < 4; ++j)
            if (overlaps(out[i], out_bytes[i], in[j], in_bytes[j]))
                return VGGT_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], out_bytes[i], out[j], out_bytes[j]))
                return VGGT_ERR_INVALID_ARG;
    }
    vggt::PlanParams p;
    p.n_seqs = cache.n_seqs;
    p.page_size = cache.page_size;
    p.n_pages = cache.n_pages;
    p.max_pages = cache.max_pages;
    p.n_rows = n_rows;
    p.free_capacity = free_capacity;
    p.by_page.set(static_cast<uint32_t>(cache.page_size));
    p.cached = cached_lens;
    p.fresh = new_lens;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.table = block_table;
    p.cu_rows = cu_rows;
    p.kv_lens = kv_lens;
    p.slots = slots;
    p.counts = counts;
    const int64_t want = (static_cast<int64_t>(n_rows) + 4 * vggt::kPlanThreads - 1) / (4 * vggt::kPlanThreads);
    const int grid = static_cast<int>(want < 1 ? 1 : (want > 592 ? 592 : want));
    const size_t smem = 4 * B * sizeof(int);
    if (smem > 40 * 1024 &&  // with the static part above 48 KB
        cudaFuncSetAttribute(vggt::cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * vggt::kCacheMaxSeqs * static_cast<int>(sizeof(int))) != cudaSuccess)
        return VGGT_ERR_CUDA;
    vggt::cache_plan_kernel<<<grid, vggt::kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}

VGGT_API vggt_status vggt_cache_append(vggt_cache cache, const void *k, const void *v, int64_t row_stride,
                                       int64_t in_head_stride, const int32_t *slots, int32_t n_rows, void *k_pages,
                                       void *v_pages, void *stream)
{
    vggt_status st = check_cache(cache);
    if (st != VGGT_OK)
        return st;
    if (n_rows < 0 || !stride_ok(row_stride, vggt::kHeadDim) || !stride_ok(in_head_stride, vggt::kHeadDim))
        return VGGT_ERR_INVALID_ARG;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages) || k_pages == v_pages)
        return VGGT_ERR_INVALID_ARG;
    if (n_rows == 0)
        return VGGT_OK;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || !aligned4(slots))
        return VGGT_ERR_INVALID_ARG;
    const size_t pool = pool_bytes(cache), sb = 4 * static_cast<size_t>(n_rows);
    const size_t rows = 2 * static_cast<size_t>(span(n_rows, row_stride, cache.n_kv_heads, in_head_stride));
    for (const void *out : {k_pages, v_pages})
        if (overlaps(out, pool, k, rows) || overlaps(out, pool, v, rows) || overlaps(out, pool, slots, sb))
            return VGGT_ERR_INVALID_ARG;
    vggt::AppendParams p;
    p.n_rows = n_rows;
    p.vecs = cache.n_kv_heads * 8;
    p.page_size = cache.page_size;
    p.n_slots = cache.n_pages * cache.page_size;
    p.row_stride = row_stride / 8;
    p.in_head_stride = in_head_stride / 8;
    p.page_stride = cache.page_stride / 8;
    p.head_stride = cache.head_stride / 8;
    p.token_stride = cache.token_stride / 8;
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.k_pages = static_cast<uint4 *>(k_pages);
    p.v_pages = static_cast<uint4 *>(v_pages);
    p.slots = slots;
    p.by_vecs.set(static_cast<uint32_t>(p.vecs));
    p.by_page.set(static_cast<uint32_t>(cache.page_size));
    // One vector per thread, then four.  Measured both sides: 703 thousand
    // vectors (four frames of 1374 tokens, 16 heads), 8.7 us against 10.0; 1.4
    // million, 16.2 against 15.0.
    const int64_t total = static_cast<int64_t>(n_rows) * p.vecs;
    if (total <= kFewAppendVecs) {
        const int64_t blocks = (total + 255) / 256;
        vggt::cache_append_kernel<1><<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    } else {
        const int64_t blocks = (total + 1023) / 1024;
        if (blocks > INT32_MAX)
            return VGGT_ERR_UNSUPPORTED;
        vggt::cache_append_kernel<4><<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    }
    return launched();
}

namespace {

// Rows of a workspace slot: those of a pair of query tiles.
int64_t part_rows(const vggt_cache &c, int64_t n_rows)
{
    const int64_t group = c.n_heads / c.n_kv_heads, pair = 2 * (vggt::kBlockM / group);
    return group * (n_rows < pair ? n_rows : pair);
}

// Workspace: one vggt::Join per CTA, (m, l) of every row of every slot,
// float2 [2 * 148][part_rows], and its sum of P V, float [2 * 148][part_rows][64].
struct CachedLayout {
    size_t ml, po, total;
};

CachedLayout cached_layout(const vggt_cache &c, int64_t n_rows)
{
    const size_t rows = 2 * static_cast<size_t>(vggt::kMaxCtas) * static_cast<size_t>(part_rows(c, n_rows));
    CachedLayout l;
    l.ml = align256(vggt::kMaxCtas * sizeof(vggt::Join));
    l.po = align256(l.ml + rows * 8);
    l.total = align256(l.po + rows * vggt::kHeadDim * 4);
    return l;
}

// Key tiles of the longest sequence that the block table can hold.
int64_t most_key_tiles(const vggt_cache &c)
{
    return (static_cast<int64_t>(c.max_pages) * c.page_size + vggt::kBlockN - 1) / vggt::kBlockN;
}

// Query rows [n_rows, H, 64] with their strides; a box holds the G heads of
// one key head for F tokens.
bool make_query_map(CUtensorMap *map, const void *q, const vggt_cache &c, int64_t n_rows, int64_t row_stride,
                    int64_t head_stride, int group, int tokens)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(vggt::kHeadDim), static_cast<cuuint64_t>(c.n_heads),
                                static_cast<cuuint64_t>(n_rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(vggt::kHeadDim), static_cast<cuuint32_t>(group),
                               static_cast<cuuint32_t>(tokens)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pages as (64, page_size, n_kv_heads, n_pages); a box is box_rows positions
// of one head of one page.
bool make_pages_map(CUtensorMap *map, const void *pages, const vggt_cache &c, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(vggt::kHeadDim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.n_kv_heads), static_cast<cuuint64_t>(c.n_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride) * 2,
                                   static_cast<cuuint64_t>(c.head_stride) * 2,
                                   static_cast<cuuint64_t>(c.page_stride) * 2};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(vggt::kHeadDim), static_cast<cuuint32_t>(box_rows), 1u, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pages), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace

VGGT_API size_t vggt_attn_cached_workspace_bytes(vggt_cache cache, int32_t n_rows)
{
    // one key tile: no unit can be cut
    if (check_cache(cache) != VGGT_OK || n_rows < 1 || most_key_tiles(cache) == 1)
        return 0;
    return cached_layout(cache, n_rows).total;
}

VGGT_API vggt_status vggt_attn_cached(vggt_cache cache, const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                      const void *k_pages, const void *v_pages, const int32_t *block_table,
                                      const int32_t *cu_rows, const int32_t *kv_lens, int32_t n_rows,
                                      int32_t causal_unit, void *o, float *lse, void *workspace,
                                      size_t workspace_bytes, float scale, void *stream)
{
    vggt_status st = check_cache(cache);
    if (st != VGGT_OK)
        return st;
    if (n_rows < 0 || causal_unit < 0 || !scale_ok(scale) || !stride_ok(q_row_stride, vggt::kHeadDim) ||
        !stride_ok(q_head_stride, vggt::kHeadDim))
        return VGGT_ERR_INVALID_ARG;
    if (n_rows > INT32_MAX - 1024)
        return VGGT_ERR_UNSUPPORTED;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages) || !block_table || !cu_rows || !kv_lens ||
        !aligned4(block_table) || !aligned4(cu_rows) || !aligned4(kv_lens))
        return VGGT_ERR_INVALID_ARG;
    if (n_rows == 0)
        return VGGT_OK;
    if (!q || !o || !aligned16(q) || !aligned16(o) || !aligned4(lse))
        return VGGT_ERR_INVALID_ARG;
    const size_t need = vggt_attn_cached_workspace_bytes(cache, n_rows);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return VGGT_ERR_INVALID_ARG;
    if (workspace_bytes < need)
        return VGGT_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(n_rows) * cache.n_heads, B = static_cast<size_t>(cache.n_seqs);
    const void *in[6] = {q, k_pages, v_pages, block_table, cu_rows, kv_lens};
    const size_t in_bytes[6] = {2 * static_cast<size_t>(span(n_rows, q_row_stride, cache.n_heads, q_head_stride)),
                                pool_bytes(cache), pool_bytes(cache), 4 * B * cache.max_pages, 4 * (B + 1), 4 * B};
    const void *out[3] = {o, lse, workspace};
    const size_t out_bytes[3] = {rows * vggt::kHeadDim * 2, lse ? rows * 4 : 0, need};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 6; ++j)
            if (out_bytes[i] > 0 && overlaps(out[i], out_bytes[i], in[j], in_bytes[j]))
                return VGGT_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out_bytes[i] > 0 && out_bytes[j] > 0 && overlaps(out[i], out_bytes[i], out[j], out_bytes[j]))
                return VGGT_ERR_INVALID_ARG;
    }
    int num_sms = 0;
    if ((st = prepare_device(num_sms)) != VGGT_OK)
        return st;
    vggt::CachedParams p;
    std::memset(&p, 0, sizeof p);
    p.n_seqs = cache.n_seqs;
    p.n_rows = n_rows;
    p.H = cache.n_heads;
    p.Hkv = cache.n_kv_heads;
    p.group = cache.n_heads / cache.n_kv_heads;
    p.tile_tokens = vggt::kBlockM / p.group;
    p.page_size = cache.page_size;
    p.n_pages = cache.n_pages;
    p.max_pages = cache.max_pages;
    p.unit = causal_unit;
    p.by_group.set(static_cast<uint32_t>(p.group));
    p.by_tile.set(static_cast<uint32_t>(p.tile_tokens));
    p.by_page.set(static_cast<uint32_t>(p.page_size));
    p.by_unit.set(static_cast<uint32_t>(causal_unit > 0 ? causal_unit : 1));
    p.box_rows = cache.page_size & -cache.page_size;
    if (p.box_rows > vggt::kBlockN)
        p.box_rows = vggt::kBlockN;
    // The most that the units can cost: every unit as a pair of tiles over the longest sequence.
    const int64_t units = cache.n_kv_heads * ((n_rows + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens) +
                                              static_cast<int64_t>(cache.n_seqs));
    const int64_t most = 2 * most_key_tiles(cache) + vggt::kUnitCost;
    while ((units * ((most >> p.cost_shift) + 1)) > INT32_MAX)
        ++p.cost_shift;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.table = block_table;
    p.cu_rows = cu_rows;
    p.kv_lens = kv_lens;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.wait_limit_ns = vggt::kWaitLimitNs;
    if (need > 0) {
        const CachedLayout l = cached_layout(cache, n_rows);
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        p.part_rows = static_cast<int>(part_rows(cache, n_rows));
        p.join = reinterpret_cast<vggt::Join *>(ws);
        p.part_ml = reinterpret_cast<float2 *>(ws + l.ml);
        p.part_o = reinterpret_cast<float *>(ws + l.po);
    }
    CUtensorMap tq, tk, tv;
    if (!make_query_map(&tq, q, cache, n_rows, q_row_stride, q_head_stride, p.group, p.tile_tokens) ||
        !make_pages_map(&tk, k_pages, cache, p.box_rows) || !make_pages_map(&tv, v_pages, cache, p.box_rows))
        return VGGT_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>(num_sms < vggt::kMaxCtas ? num_sms : vggt::kMaxCtas);
    // Both launches are set up while the one before them runs and wait for its
    // end on the device.
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(vggt::kAttnThreads);
    cfg.dynamicSmemBytes = vggt::cached_smem_bytes(cache.n_seqs);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, vggt::cached_attn_kernel, tq, tk, tv, p);
    if ((st = launched()) != VGGT_OK || need == 0)
        return st;
    cfg.gridDim = dim3(grid, static_cast<unsigned>((p.part_rows + vggt::kJoinRows - 1) / vggt::kJoinRows));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchKernelEx(
        &cfg, p.part_rows <= vggt::kJoinRows ? vggt::cached_combine_kernel<12> : vggt::cached_combine_kernel<4>, p);
    return launched();
}

namespace {

template <typename X, int kWarps, bool kAhead>
void launch_norm(const vggt::NormParams &p, cudaStream_t s)
{
    constexpr int rows = kWarps == 1 ? 4 : 1;
    const unsigned threads = kWarps == 1 ? 128 : 32 * ((static_cast<unsigned>(p.n_cols) + 255) / 256);
    vggt::norm_residual_kernel<X, kWarps, kAhead>
        <<<static_cast<unsigned>((p.n_rows + rows - 1) / rows), threads, 0, s>>>(p);
}

// Measured both sides: 128 rows, 8.2 us ahead against 8.2-10.2 (256 to 4096
// channels); 600 rows, 8.2-20.5 against 8.2-16.4.
constexpr int64_t kFewNormRows = 256;

template <typename X, int kWarps>
void launch_norm_rows(const vggt::NormParams &p, cudaStream_t s)
{
    if (p.n_rows <= kFewNormRows)
        launch_norm<X, kWarps, true>(p, s);
    else
        launch_norm<X, kWarps, false>(p, s);
}

template <typename X>
void launch_norm_cols(const vggt::NormParams &p, cudaStream_t s)
{
    if (p.n_cols <= 256)
        launch_norm_rows<X, 1>(p, s);
    else if (p.n_cols <= 1024)
        launch_norm_rows<X, 4>(p, s);
    else if (p.n_cols <= 2048)
        launch_norm_rows<X, 8>(p, s);
    else if (p.n_cols <= 4096)
        launch_norm_rows<X, 16>(p, s);
    else
        launch_norm_rows<X, 32>(p, s);
}

} // namespace

VGGT_API vggt_status vggt_norm_residual(vggt_norm norm, const void *x, const void *y, const float *post_w,
                                        const float *post_b, const float *scale, const void *gate, const float *w,
                                        const float *b, void *x_out, void *h, void *stream)
{
    if (norm.n_rows < 0 || norm.n_cols < 1 || (norm.kind != VGGT_NORM_LAYER && norm.kind != VGGT_NORM_RMS) ||
        (norm.x_fp32 != 0 && norm.x_fp32 != 1) || (norm.post_norm != 0 && norm.post_norm != 1) ||
        !std::isfinite(norm.eps) || norm.eps < 0.f)
        return VGGT_ERR_INVALID_ARG;
    if (norm.n_cols % 8 != 0 || norm.n_cols > vggt::kNormMaxCols || norm.n_rows > INT32_MAX - 1024)
        return VGGT_ERR_UNSUPPORTED;
    if (norm.n_rows == 0)
        return VGGT_OK;
    if (!y && (post_w || post_b || scale || gate || x_out || norm.post_norm))
        return VGGT_ERR_INVALID_ARG;
    if ((!norm.post_norm && (post_w || post_b)) || (!h && (w || b)) || (!x_out && !h))
        return VGGT_ERR_INVALID_ARG;
    if (gate && norm.rows_per_gate < 1)
        return VGGT_ERR_INVALID_ARG;
    const int64_t C = norm.n_cols, R = norm.n_rows;
    if (!stride_ok(norm.x_stride, C) || (y && !stride_ok(norm.y_stride, C)) ||
        (x_out && !stride_ok(norm.out_stride, C)) || (h && !stride_ok(norm.h_stride, C)))
        return VGGT_ERR_INVALID_ARG;
    if (!x)
        return VGGT_ERR_INVALID_ARG;
    const size_t xw = norm.x_fp32 ? 4 : 2;
    auto bytes = [&](const void *ptr, int64_t stride, size_t width) {
        return ptr ? static_cast<size_t>((R - 1) * stride + C) * width : size_t{0};
    };
    const size_t cb = static_cast<size_t>(C) * 4;
    const int64_t gates = gate ? (R + norm.rows_per_gate - 1) / norm.rows_per_gate : 0;
    const void *in[8] = {x, y, post_w, post_b, scale, gate, w, b};
    const size_t in_bytes[8] = {bytes(x, norm.x_stride, xw), bytes(y, norm.y_stride, 2), cb, cb, cb,
                                static_cast<size_t>(gates * C) * 2, cb, cb};
    const void *out[2] = {x_out, h};
    const size_t out_bytes[2] = {bytes(x_out, norm.out_stride, xw), bytes(h, norm.h_stride, 2)};
    for (int i = 0; i < 8; ++i)
        if (!aligned16(in[i]))
            return VGGT_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (!aligned16(out[i]))
            return VGGT_ERR_INVALID_ARG;
        for (int j = 0; j < 8; ++j) {
            if (!out[i] || !in[j] || (i == 0 && j == 0 && x_out == x && norm.out_stride == norm.x_stride))
                continue;
            if (overlaps(out[i], out_bytes[i], in[j], in_bytes[j]))
                return VGGT_ERR_INVALID_ARG;
        }
    }
    if (x_out && h && overlaps(x_out, out_bytes[0], h, out_bytes[1]))
        return VGGT_ERR_INVALID_ARG;
    vggt::NormParams p;
    p.n_rows = R;
    p.n_cols = norm.n_cols;
    p.rows_per_gate = gate ? norm.rows_per_gate : 1;
    p.layer = norm.kind == VGGT_NORM_LAYER;
    p.post_norm = norm.post_norm;
    p.eps = norm.eps;
    p.inv_cols = 1.f / static_cast<float>(C);
    p.x_stride = norm.x_stride;
    p.y_stride = norm.y_stride;
    p.out_stride = norm.out_stride;
    p.h_stride = norm.h_stride;
    p.gate_stride = C;
    p.x = x;
    p.y = static_cast<const __nv_bfloat16 *>(y);
    p.gate = static_cast<const __nv_bfloat16 *>(gate);
    p.post_w = post_w;
    p.post_b = post_b;
    p.scale = scale;
    p.w = w;
    p.b = b;
    p.x_out = x_out;
    p.h = static_cast<__nv_bfloat16 *>(h);
    if (norm.x_fp32)
        launch_norm_cols<float>(p, static_cast<cudaStream_t>(stream));
    else
        launch_norm_cols<__nv_bfloat16>(p, static_cast<cudaStream_t>(stream));
    return launched();
}
