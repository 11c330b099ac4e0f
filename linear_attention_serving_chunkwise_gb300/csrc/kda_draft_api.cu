// C ABI of the draft-step operators: host-side validation and dispatch.  Declarations and
// contracts: include/kda.h.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/kda.h"
#include "kda_draft_launch.h"

namespace {

struct Span {
    uintptr_t lo, hi;   // [lo, hi); empty for a null pointer
};
Span span(const void* p, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p ? Span{lo, lo + bytes} : Span{0, 0};
}
bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// the outputs (the first `n_out` spans) overlap neither one another nor an input
template <int N>
bool apart(const Span (&s)[N], int n_out)
{
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < N; ++j)
            if (meet(s[i], s[j])) return false;
    return true;
}

bool known_dtype(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }
kda_status of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

kda_status validate_tree_shape(int32_t batch, int32_t nodes, int32_t heads, int32_t dk, int32_t dv, int32_t dtype, int32_t prologue)
{
    if (batch < 0 || nodes < 1 || nodes > KDA_TREE_MAX_NODES || heads < 1 || (prologue & ~KDA_PROLOGUE_ALL)) return KDA_ERR_INVALID_ARG;
    if (!known_dtype(dtype) || dk != dv || (dk != 64 && dk != 128)) return KDA_ERR_UNSUPPORTED;
    if ((size_t)batch * nodes > 0x7fffffffull / heads) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda_status validate_attn(const kda_tree_attention_desc* d)
{
    if (!d || d->batch < 0 || d->nodes < 1 || d->nodes > KDA_TREE_MAX_NODES || d->num_heads < 1 || d->num_kv_heads < 1 ||
        d->num_heads % d->num_kv_heads || d->num_pages < 0 || d->page_size < 1 || d->table_cols < 0 || !isfinite(d->scale))
        return KDA_ERR_INVALID_ARG;
    if (!known_dtype(d->dtype) || (d->dim != 64 && d->dim != 128)) return KDA_ERR_UNSUPPORTED;
    if ((size_t)d->batch * d->nodes > 0x7fffffffull / d->num_heads) return KDA_ERR_INVALID_ARG;
    if ((size_t)d->page_size * d->num_kv_heads > 0x7fffffffull / d->dim) return KDA_ERR_INVALID_ARG;
    const int64_t page = (int64_t)d->page_size * d->num_kv_heads * d->dim, per16 = d->dtype == KDA_BF16 ? 8 : 4;
    const int64_t strides[] = {d->k_page_stride, d->v_page_stride};
    for (const int64_t s : strides) {
        if (s < page || s % per16) return KDA_ERR_INVALID_ARG;
        if (d->num_pages > 0 && s > (INT64_MAX >> 4) / d->num_pages) return KDA_ERR_INVALID_ARG;
    }
    kda::TreeAttnArgs a = {};
    a.batch = d->batch; a.nodes = d->nodes; a.heads = d->num_heads; a.kv_heads = d->num_kv_heads;
    a.page_size = d->page_size; a.table_cols = d->table_cols; a.dim = d->dim; a.bf16 = d->dtype == KDA_BF16;
    return kda::tree_attn_fits(a) ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

kda_status kda_page_tables(int32_t batch, int32_t table_cols, int32_t num_free, int32_t page_size, int32_t max_tokens,
                           const int32_t* context_lens, const int32_t* new_lens, const int32_t* pages_held,
                           int32_t* block_table, const int32_t* free_pages, int64_t* slot_map, int32_t* cu_seqlens,
                           int32_t* pages_held_out, int32_t* pages_taken, void* stream)
{
    if (batch < 0 || table_cols < 0 || num_free < 0 || page_size < 1 || max_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (batch > KDA_PAGE_TABLES_MAX_BATCH) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)batch * table_cols > 0x7fffffff) return KDA_ERR_INVALID_ARG;
    const size_t B = (size_t)batch, cells = B * table_cols;
    if (!cu_seqlens || !pages_taken || (max_tokens && !slot_map) || (num_free && !free_pages)) return KDA_ERR_INVALID_ARG;
    if (batch && (!context_lens || !new_lens || !pages_held || !pages_held_out || (cells && !block_table))) return KDA_ERR_INVALID_ARG;
    const void* words[] = {context_lens, new_lens, pages_held, block_table, free_pages, cu_seqlens, pages_held_out, pages_taken};
    for (const void* p : words)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    if (!aligned(slot_map, 8)) return KDA_ERR_INVALID_ARG;
    const Span s[] = {span(block_table, cells * 4), span(slot_map, (size_t)max_tokens * 8), span(cu_seqlens, (B + 1) * 4),
                      span(pages_held_out, B * 4), span(pages_taken, 4), span(context_lens, B * 4), span(new_lens, B * 4),
                      span(pages_held, B * 4), span(free_pages, (size_t)num_free * 4)};
    if (!apart(s, 5)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const kda::PageTablesArgs a = {batch, table_cols, num_free, page_size, max_tokens, context_lens, new_lens, pages_held,
                                   free_pages, block_table, slot_map, cu_seqlens, pages_held_out, pages_taken, status};
    return of(kda::launch_page_tables(a, static_cast<cudaStream_t>(stream)));
}

size_t kda_tree_attention_workspace_bytes(const kda_tree_attention_desc* desc)
{
    if (validate_attn(desc) != KDA_OK || desc->batch == 0) return 0;
    return kda::tree_attn_workspace_bytes(desc->batch, desc->nodes, desc->num_heads, desc->num_kv_heads, desc->dim,
                                          desc->dtype == KDA_BF16);
}

kda_status kda_tree_attention(const kda_tree_attention_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* context_lens, const int32_t* parents, void* out,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    const kda_status st = validate_attn(desc);
    if (st != KDA_OK) return st;
    const kda_tree_attention_desc d = *desc;
    const size_t need = kda_tree_attention_workspace_bytes(desc);
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    if (d.batch == 0) return KDA_OK;
    const size_t B = (size_t)d.batch, e = d.dtype == KDA_BF16 ? 2 : 4, cells = B * d.table_cols;
    if (!q || !context_lens || !parents || !out || (need && !workspace)) return KDA_ERR_INVALID_ARG;
    if ((d.num_pages && (!k_cache || !v_cache)) || (cells && !block_table)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(parents, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t rows = B * d.nodes * d.num_heads * d.dim * e, page = (size_t)d.page_size * d.num_kv_heads * d.dim * e;
    const size_t more = d.num_pages ? (size_t)d.num_pages - 1 : 0;
    const Span s[] = {span(out, rows), span(workspace, need), span(q, rows),
                      span(d.num_pages ? k_cache : nullptr, more * d.k_page_stride * e + page),
                      span(d.num_pages ? v_cache : nullptr, more * d.v_page_stride * e + page),
                      span(block_table, cells * 4), span(context_lens, B * 4), span(parents, B * d.nodes * 4)};
    if (!apart(s, 2)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::TreeAttnArgs a = {};
    a.batch = d.batch; a.nodes = d.nodes; a.heads = d.num_heads; a.kv_heads = d.num_kv_heads; a.dim = d.dim;
    a.num_pages = d.num_pages; a.page_size = d.page_size; a.table_cols = d.table_cols; a.bf16 = d.dtype == KDA_BF16;
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    a.k_page_stride = (size_t)d.k_page_stride; a.v_page_stride = (size_t)d.v_page_stride;
    a.block_table = block_table; a.context_lens = context_lens; a.parents = parents;
    a.scale = d.scale; a.out = out; a.workspace = workspace; a.status = status;
    return of(kda::launch_tree_attn(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_tree_decode(int32_t batch, int32_t nodes, int32_t num_heads, int32_t dk, int32_t dv, int32_t qkv_dtype,
                           int32_t prologue, const void* q, const void* k, const void* v, const float* g,
                           const float* beta, const int32_t* parents, const float* gate, const float* state, float* out,
                           float* writes, void* stream)
{
    const kda_status st = validate_tree_shape(batch, nodes, num_heads, dk, dv, qkv_dtype, prologue);
    if (st != KDA_OK) return st;
    if (batch == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !parents || !state || !out || !writes) return KDA_ERR_INVALID_ARG;
    const void* wide[] = {q, k, v, g, gate, state, out, writes};
    for (const void* p : wide)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(beta, 4) || !aligned(parents, 4)) return KDA_ERR_INVALID_ARG;
    const size_t rows = (size_t)batch * nodes * num_heads, e = qkv_dtype == KDA_BF16 ? 2 : 4;
    const Span s[] = {span(out, rows * dv * 4), span(writes, rows * dv * 4), span(q, rows * dk * e), span(k, rows * dk * e),
                      span(v, rows * dv * e), span(g, rows * dk * 4), span(beta, rows * 4), span(gate, rows * dv * 4),
                      span(parents, (size_t)batch * nodes * 4), span(state, (size_t)batch * num_heads * dk * dv * 4)};
    if (!apart(s, 2)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::TreeDecodeArgs a = {};
    a.batch = batch; a.nodes = nodes; a.num_heads = num_heads; a.dk = dk; a.dv = dv; a.bf16 = qkv_dtype == KDA_BF16;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.parents = parents; a.state = state;
    a.out = out; a.writes = writes; a.status = status; a.prologue = prologue; a.gate = gate;
    return of(kda::launch_tree_decode(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_tree_commit(int32_t batch, int32_t nodes, int32_t num_heads, int32_t dk, int32_t dv, int32_t qkv_dtype,
                           int32_t prologue, const void* k, const float* g, const float* writes, const int32_t* path,
                           const int32_t* n_accept, float* state, void* stream)
{
    const kda_status st = validate_tree_shape(batch, nodes, num_heads, dk, dv, qkv_dtype, prologue);
    if (st != KDA_OK) return st;
    if (batch == 0) return KDA_OK;
    if (!k || !g || !writes || !path || !n_accept || !state) return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(g, 16) || !aligned(writes, 16) || !aligned(state, 16) || !aligned(path, 4) || !aligned(n_accept, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t rows = (size_t)batch * nodes * num_heads, e = qkv_dtype == KDA_BF16 ? 2 : 4;
    const Span s[] = {span(state, (size_t)batch * num_heads * dk * dv * 4), span(k, rows * dk * e), span(g, rows * dk * 4),
                      span(writes, rows * dv * 4), span(path, (size_t)batch * nodes * 4), span(n_accept, (size_t)batch * 4)};
    if (!apart(s, 1)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    kda::TreeCommitArgs a = {};
    a.batch = batch; a.nodes = nodes; a.num_heads = num_heads; a.dk = dk; a.dv = dv; a.bf16 = qkv_dtype == KDA_BF16;
    a.k = k; a.g = g; a.writes = writes; a.path = path; a.n_accept = n_accept; a.state = state; a.status = status;
    a.prologue = prologue;
    return of(kda::launch_tree_commit(a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_verify_drafts(int32_t batch, int32_t nodes, int32_t vocab, const float* target, const float* draft,
                             const int32_t* tokens, const int32_t* parents, const float* uniforms, const float* noise,
                             int32_t* path, int32_t* n_accept, int32_t* next_token, void* stream)
{
    if (batch < 0 || nodes < 1 || nodes > KDA_TREE_MAX_NODES || vocab < 1 || batch > (1 << 24)) return KDA_ERR_INVALID_ARG;
    if (vocab > KDA_VERIFY_MAX_VOCAB) return KDA_ERR_UNSUPPORTED;
    if (batch == 0) return KDA_OK;
    if (!target || !tokens || !parents || !uniforms || !noise || !path || !n_accept || !next_token) return KDA_ERR_INVALID_ARG;
    const void* words[] = {target, draft, tokens, parents, uniforms, noise, path, n_accept, next_token};
    for (const void* p : words)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t B = (size_t)batch, n = B * nodes;
    const Span s[] = {span(path, n * 4), span(n_accept, B * 4), span(next_token, B * 4),
                      span(target, B * (nodes + 1) * (size_t)vocab * 4), span(draft, n * (size_t)vocab * 4),
                      span(tokens, n * 4), span(parents, n * 4), span(uniforms, n * 4), span(noise, B * (size_t)vocab * 4)};
    if (!apart(s, 3)) return KDA_ERR_INVALID_ARG;
    int* status = kda::device_status_ptr();
    if (!status) return KDA_ERR_CUDA;
    const kda::VerifyArgs a = {batch, nodes, vocab, target, draft, tokens, parents, uniforms, noise, path, n_accept, next_token, status};
    return of(kda::launch_verify(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
