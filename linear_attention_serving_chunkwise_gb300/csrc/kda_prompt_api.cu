// C ABI of the attention layers' prompt path and of the cache's upkeep: host-side validation and
// dispatch.  Declarations and contracts: include/kda.h.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_api_checks.h"
#include "kda_prompt_launch.h"

namespace {

using namespace kda::checks;

size_t element(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// a page of a cache, its stride and the whole cache, in elements that a pointer can count
bool page_stride_ok(int32_t num_pages, int64_t page, int64_t stride, int32_t dtype)
{
    const int64_t per16 = dtype == KDA_BF16 ? 8 : 4;
    return stride >= page && stride % per16 == 0 && (num_pages == 0 || stride <= (INT64_MAX >> 4) / num_pages);
}

kda::ChunkAttnArgs chunk_args(const kda_chunk_attention_desc& d)
{
    kda::ChunkAttnArgs a = {};
    a.batch = d.batch; a.tokens = d.total_tokens; a.heads = d.num_heads; a.kv_heads = d.num_kv_heads; a.dim = d.dim;
    a.num_pages = d.num_pages; a.page_size = d.page_size; a.table_cols = d.table_cols; a.bf16 = d.dtype == KDA_BF16;
    a.k_page_stride = (size_t)d.k_page_stride; a.v_page_stride = (size_t)d.v_page_stride; a.scale = d.scale;
    return a;
}

kda_status validate_chunk(const kda_chunk_attention_desc* d)
{
    if (!d || d->batch < 0 || d->total_tokens < 0 || d->num_heads < 1 || d->num_kv_heads < 1 || d->num_heads % d->num_kv_heads ||
        d->num_pages < 0 || d->page_size < 1 || d->table_cols < 0 ||
        !(fabsf(d->scale) <= 0x1p126f))     // (scores are kept in powers of two: scale / ln 2 is finite too)
        return KDA_ERR_INVALID_ARG;
    if (!known_dtype(d->dtype) || (d->dim != 64 && d->dim != 128) || d->num_heads / d->num_kv_heads > KDA_CHUNK_MAX_GROUP) return KDA_ERR_UNSUPPORTED;
    if ((size_t)d->total_tokens > 0x7fffffffull / d->num_heads) return KDA_ERR_INVALID_ARG;
    if ((size_t)d->page_size * d->num_kv_heads > 0x7fffffffull / d->dim) return KDA_ERR_INVALID_ARG;
    const int64_t page = (int64_t)d->page_size * d->num_kv_heads * d->dim;
    if (!page_stride_ok(d->num_pages, page, d->k_page_stride, d->dtype) || !page_stride_ok(d->num_pages, page, d->v_page_stride, d->dtype))
        return KDA_ERR_INVALID_ARG;
    return kda::chunk_attn_fits(chunk_args(*d)) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status validate_cache(const kda_cache_desc* d)
{
    if (!d || d->num_layers < 0 || d->num_pages < 0 || d->page_size < 1 || d->num_kv_heads < 1 || d->dim < 1) return KDA_ERR_INVALID_ARG;
    if (!known_dtype(d->dtype)) return KDA_ERR_UNSUPPORTED;
    if ((size_t)d->num_kv_heads > 0x7fffffffull / d->dim || (size_t)d->page_size > 0x7fffffffull / ((size_t)d->num_kv_heads * d->dim))
        return KDA_ERR_INVALID_ARG;
    const int64_t row = (int64_t)d->num_kv_heads * d->dim, per16 = d->dtype == KDA_BF16 ? 8 : 4, page = d->page_size * row;
    if (row % per16) return KDA_ERR_UNSUPPORTED;
    const int64_t layers[] = {d->k_layer_stride, d->v_layer_stride}, pages[] = {d->k_page_stride, d->v_page_stride};
    for (int i = 0; i < 2; ++i) {
        if (d->num_pages > 1 && !page_stride_ok(d->num_pages, page, pages[i], d->dtype)) return KDA_ERR_INVALID_ARG;
        if (d->num_layers > 1 && !page_stride_ok(d->num_layers, page, layers[i], d->dtype)) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

bool cache_empty(const kda_cache_desc& d) { return d.num_layers == 0 || d.num_pages == 0; }

kda::CacheArgs cache_args(const kda_cache_desc& d, void* k, void* v)
{
    const size_t e = element(d.dtype);
    return {d.num_layers, d.num_pages, d.page_size, (size_t)d.num_kv_heads * d.dim * e, static_cast<uint8_t*>(k), static_cast<uint8_t*>(v),
            d.num_layers > 1 ? d.k_layer_stride * e : 0, d.num_layers > 1 ? d.v_layer_stride * e : 0,
            d.num_pages > 1 ? d.k_page_stride * e : 0, d.num_pages > 1 ? d.v_page_stride * e : 0};
}

Span cache_span(const kda_cache_desc& d, const void* p, int64_t layer, int64_t page)
{
    if (cache_empty(d)) return {0, 0};
    const size_t one = (size_t)d.page_size * d.num_kv_heads * d.dim;
    return span(p, ((d.num_layers > 1 ? (size_t)(d.num_layers - 1) * layer : 0) + (d.num_pages > 1 ? (size_t)(d.num_pages - 1) * page : 0) + one) * element(d.dtype));
}

}  // namespace

extern "C" {

size_t kda_chunk_attention_workspace_bytes(const kda_chunk_attention_desc* desc)
{
    if (validate_chunk(desc) != KDA_OK || desc->batch == 0 || desc->total_tokens == 0) return 0;
    return kda::chunk_attn_workspace_bytes(chunk_args(*desc));
}

kda_status kda_chunk_attention(const kda_chunk_attention_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* context_lens, const int32_t* cu_seqlens, void* out,
                               void* workspace, size_t workspace_bytes, void* stream)
{
    const kda_status st = validate_chunk(desc);
    if (st != KDA_OK) return st;
    const kda_chunk_attention_desc d = *desc;
    const size_t need = kda_chunk_attention_workspace_bytes(desc);
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (d.batch == 0 || d.total_tokens == 0) return KDA_OK;
    const size_t B = (size_t)d.batch, e = element(d.dtype), cells = B * d.table_cols;
    if (!q || !context_lens || !cu_seqlens || !out || (need && !workspace)) return KDA_ERR_INVALID_ARG;
    if ((d.num_pages && (!k_cache || !v_cache)) || (cells && !block_table)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t rows = (size_t)d.total_tokens * d.num_heads * d.dim * e, page = (size_t)d.page_size * d.num_kv_heads * d.dim * e;
    const size_t more = d.num_pages ? (size_t)d.num_pages - 1 : 0;
    const Span s[] = {span(out, rows), span(workspace, need), span(q, rows),
                      span(d.num_pages ? k_cache : nullptr, more * d.k_page_stride * e + page),
                      span(d.num_pages ? v_cache : nullptr, more * d.v_page_stride * e + page),
                      span(block_table, cells * 4), span(context_lens, B * 4), span(cu_seqlens, (B + 1) * 4)};
    if (!apart(s, 2)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::ChunkAttnArgs a = chunk_args(d);
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    a.block_table = block_table; a.context_lens = context_lens; a.cu_seqlens = cu_seqlens;
    a.out = out; a.workspace = workspace; a.status = status;
    return of(kda::launch_chunk_attn(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_norm_rotate(const kda_norm_rotate_desc* desc, const void* q, const void* k, const void* v, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions, const int64_t* slots, void* q_out,
                           void* k_cache, void* v_cache, void* stream)
{
    if (!desc) return KDA_ERR_INVALID_ARG;
    const kda_norm_rotate_desc d = *desc;
    if (d.total_tokens < 0 || d.num_heads < 1 || d.num_kv_heads < 1 || d.num_pages < 0 || d.page_size < 1 || d.rot_dim < 0 || d.rot_dim > d.dim ||
        (d.flags & ~(KDA_ROTATE_INTERLEAVED | KDA_ROTATE_NO_NORM)) || !(d.eps >= 0.f) || !isfinite(d.eps))
        return KDA_ERR_INVALID_ARG;
    if (!known_dtype(d.dtype) || (d.dim != 64 && d.dim != 128) || d.rot_dim % 16) return KDA_ERR_UNSUPPORTED;
    if ((size_t)d.total_tokens > 0x7fffffffull / d.num_heads || (size_t)d.total_tokens > 0x7fffffffull / d.num_kv_heads || d.num_heads > (1 << 20) ||
        d.num_kv_heads > (1 << 20))
        return KDA_ERR_INVALID_ARG;
    if ((size_t)d.page_size * d.num_kv_heads > 0x7fffffffull / d.dim) return KDA_ERR_INVALID_ARG;
    const int64_t page = (int64_t)d.page_size * d.num_kv_heads * d.dim, per16 = d.dtype == KDA_BF16 ? 8 : 4;
    if (!page_stride_ok(d.num_pages, page, d.k_page_stride, d.dtype) || !page_stride_ok(d.num_pages, page, d.v_page_stride, d.dtype))
        return KDA_ERR_INVALID_ARG;
    const int64_t strides[] = {d.q_stride, d.k_stride, d.v_stride}, heads[] = {d.num_heads, d.num_kv_heads, d.num_kv_heads};
    for (int i = 0; i < 3; ++i)
        if (strides[i] < heads[i] * d.dim || strides[i] % per16 || (d.total_tokens > 0 && strides[i] > (INT64_MAX >> 4) / d.total_tokens))
            return KDA_ERR_INVALID_ARG;
    if (d.total_tokens == 0) return KDA_OK;
    if (!q || !k || !v || !slots || !q_out || (d.rot_dim && (!inv_freq || !positions)) || (d.num_pages && (!k_cache || !v_cache))) return KDA_ERR_INVALID_ARG;
    const void* wide[] = {q, k, v, q_out, k_cache, v_cache};
    for (const void* p : wide)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(inv_freq, 4) || !aligned(positions, 4) || !aligned(slots, 8)) return KDA_ERR_INVALID_ARG;
    const size_t T = (size_t)d.total_tokens, e = element(d.dtype), more = d.num_pages ? (size_t)d.num_pages - 1 : 0, D = (size_t)d.dim;
    const Span outs[] = {span(q_out, T * d.num_heads * D * e), span(d.num_pages ? k_cache : nullptr, (more * d.k_page_stride + page) * e),
                         span(d.num_pages ? v_cache : nullptr, (more * d.v_page_stride + page) * e)};
    const Span ins[] = {span(q, ((T - 1) * d.q_stride + d.num_heads * D) * e), span(k, ((T - 1) * d.k_stride + d.num_kv_heads * D) * e),
                        span(v, ((T - 1) * d.v_stride + d.num_kv_heads * D) * e), span(q_weight, D * 4), span(k_weight, D * 4),
                        span(inv_freq, (size_t)d.rot_dim * 2), span(positions, T * 4), span(slots, T * 8)};
    // (the two caches may be views of one tensor, as may q, k and v)
    if (meet(outs[0], outs[1]) || meet(outs[0], outs[2])) return KDA_ERR_INVALID_ARG;
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (meet(o, i)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::NormRotateArgs a = {};
    a.tokens = d.total_tokens; a.heads = d.num_heads; a.kv_heads = d.num_kv_heads; a.dim = d.dim; a.rot = d.rot_dim; a.page_size = d.page_size;
    a.num_slots = (long long)d.num_pages * d.page_size;
    a.bf16 = d.dtype == KDA_BF16; a.norm = !(d.flags & KDA_ROTATE_NO_NORM); a.interleaved = d.flags & KDA_ROTATE_INTERLEAVED; a.eps = d.eps;
    a.q = q; a.k = k; a.v = v;
    a.q_stride = (size_t)d.q_stride; a.k_stride = (size_t)d.k_stride; a.v_stride = (size_t)d.v_stride;
    a.q_weight = q_weight; a.k_weight = k_weight; a.inv_freq = inv_freq; a.positions = positions; a.slots = slots;
    a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
    a.k_page_stride = (size_t)d.k_page_stride; a.v_page_stride = (size_t)d.v_page_stride; a.status = status;
    return of(kda::launch_norm_rotate(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_page_fork(int32_t num_forks, int32_t rows, int32_t table_cols, int32_t num_pages, int32_t num_free, int32_t page_size,
                         const int32_t* parents, const int32_t* children, const int32_t* lens, const int32_t* pages_held, int32_t* block_table,
                         int32_t* shares, const int32_t* free_pages, int32_t* pages_held_out, int32_t* copies, int32_t* pages_taken, void* stream)
{
    if (num_forks < 0 || rows < 0 || num_forks > rows || table_cols < 0 || num_pages < 0 || num_free < 0 || page_size < 1) return KDA_ERR_INVALID_ARG;
    if (rows > KDA_PAGE_TABLES_MAX_BATCH) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)rows * table_cols > 0x7fffffff) return KDA_ERR_INVALID_ARG;
    const size_t n = (size_t)num_forks, R = (size_t)rows, cells = R * table_cols;
    if (!pages_taken || (rows && (!pages_held || !pages_held_out)) || (cells && !block_table) || (num_pages && !shares) || (num_free && !free_pages) ||
        (num_forks && (!parents || !children || !lens || !copies)))
        return KDA_ERR_INVALID_ARG;
    const void* words[] = {parents, children, lens, pages_held, block_table, shares, free_pages, pages_held_out, copies, pages_taken};
    for (const void* p : words)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const Span s[] = {span(block_table, cells * 4), span(shares, (size_t)num_pages * 4), span(pages_held_out, R * 4), span(copies, n * 12),
                      span(pages_taken, 4), span(parents, n * 4), span(children, n * 4), span(lens, n * 4), span(pages_held, R * 4),
                      span(free_pages, (size_t)num_free * 4)};
    if (!apart(s, 5)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const kda::PageForkArgs a = {num_forks, rows, table_cols, num_pages, num_free, page_size, parents, children, lens, pages_held, free_pages,
                                 block_table, shares, pages_held_out, copies, pages_taken, status};
    return of(kda::launch_page_fork(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_page_release(int32_t rows, int32_t table_cols, int32_t num_pages, int32_t page_size, const int32_t* keep_lens,
                            const int32_t* pages_held, const int32_t* block_table, int32_t* shares, int32_t* pages_held_out, int32_t* freed,
                            int32_t* num_freed, void* stream)
{
    if (rows < 0 || table_cols < 0 || num_pages < 0 || page_size < 1) return KDA_ERR_INVALID_ARG;
    if ((int64_t)rows * table_cols > 0x7fffffff) return KDA_ERR_INVALID_ARG;
    const size_t R = (size_t)rows, cells = R * table_cols, P = (size_t)num_pages;
    if (!num_freed || (rows && (!keep_lens || !pages_held || !pages_held_out)) || (cells && !block_table) || (num_pages && (!shares || !freed)))
        return KDA_ERR_INVALID_ARG;
    const void* words[] = {keep_lens, pages_held, block_table, shares, pages_held_out, freed, num_freed};
    for (const void* p : words)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const Span s[] = {span(shares, P * 4), span(pages_held_out, R * 4), span(freed, P * 4), span(num_freed, 4), span(keep_lens, R * 4),
                      span(pages_held, R * 4), span(block_table, cells * 4)};
    if (!apart(s, 4)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const kda::PageReleaseArgs a = {rows, table_cols, num_pages, page_size, keep_lens, pages_held, block_table, shares, pages_held_out, freed, num_freed, status};
    return of(kda::launch_page_release(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_cache_copy(const kda_cache_desc* desc, int32_t num_copies, const int32_t* copies, void* k_cache, void* v_cache, void* stream)
{
    const kda_status st = validate_cache(desc);
    if (st != KDA_OK) return st;
    if (num_copies < 0) return KDA_ERR_INVALID_ARG;
    const kda_cache_desc d = *desc;
    if (num_copies == 0 || d.num_layers == 0) return KDA_OK;
    if (!copies || (d.num_pages && (!k_cache || !v_cache)) || !aligned(copies, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return KDA_ERR_INVALID_ARG;
    const Span list = span(copies, (size_t)num_copies * 12);
    if (meet(list, cache_span(d, k_cache, d.k_layer_stride, d.k_page_stride)) || meet(list, cache_span(d, v_cache, d.v_layer_stride, d.v_page_stride)))
        return KDA_ERR_INVALID_ARG;
    kda::CacheCopyArgs a = {cache_args(d, k_cache, v_cache), num_copies, copies, nullptr};
    if (!kda::cache_copy_fits(a)) return KDA_ERR_UNSUPPORTED;
    a.status = kda::device_status_ptr();
    if (!a.status) return KDA_ERR_CUDA;
    return of(kda::launch_cache_copy(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_cache_keep_path(const kda_cache_desc* desc, int32_t batch, int32_t nodes, const int64_t* slots, const int32_t* path,
                               const int32_t* n_accept, void* k_cache, void* v_cache, void* stream)
{
    const kda_status st = validate_cache(desc);
    if (st != KDA_OK) return st;
    if (batch < 0 || nodes < 1 || nodes > KDA_TREE_MAX_NODES || batch > (1 << 24)) return KDA_ERR_INVALID_ARG;
    const kda_cache_desc d = *desc;
    if (batch == 0 || d.num_layers == 0) return KDA_OK;
    if (!slots || !path || !n_accept || (d.num_pages && (!k_cache || !v_cache)) || !aligned(slots, 8) || !aligned(path, 4) || !aligned(n_accept, 4) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return KDA_ERR_INVALID_ARG;
    const size_t n = (size_t)batch * nodes;
    const Span ins[] = {span(slots, n * 8), span(path, n * 4), span(n_accept, (size_t)batch * 4)};
    for (const Span& i : ins)
        if (meet(i, cache_span(d, k_cache, d.k_layer_stride, d.k_page_stride)) || meet(i, cache_span(d, v_cache, d.v_layer_stride, d.v_page_stride)))
            return KDA_ERR_INVALID_ARG;
    kda::KeepPathArgs a = {cache_args(d, k_cache, v_cache), batch, nodes, slots, path, n_accept, nullptr};
    if (!kda::keep_path_fits(a)) return KDA_ERR_UNSUPPORTED;
    a.status = kda::device_status_ptr();
    if (!a.status) return KDA_ERR_CUDA;
    return of(kda::launch_keep_path(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
