// Internal launchers of the attention layers' prompt path and of the cache's upkeep (host side).
// Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_draft_launch.h"

namespace kda {

struct PageForkArgs {
    int forks, rows, table_cols, num_pages, num_free, page_size;
    const int32_t *parents, *children, *lens, *pages_held, *free_pages;
    int32_t *block_table, *shares, *pages_held_out, *copies, *pages_taken;
    int* status;
};

struct PageReleaseArgs {
    int rows, table_cols, num_pages, page_size;
    const int32_t *keep_lens, *pages_held, *block_table;
    int32_t *shares, *pages_held_out, *freed, *num_freed;
    int* status;
};

// The caches of all layers; strides and rows in bytes (multiples of 16).
struct CacheArgs {
    int layers, num_pages, page_size;
    size_t row;                              // bytes of one token's heads
    uint8_t *k, *v;
    size_t k_layer, v_layer, k_page, v_page;
};

struct CacheCopyArgs {
    CacheArgs c;
    int n;
    const int32_t* copies;                   // [n, 3]: source page, target page, rows
    int* status;
};

struct KeepPathArgs {
    CacheArgs c;
    int batch, nodes;
    const int64_t* slots;                    // [B, K]
    const int32_t *path, *n_accept;          // [B, K], [B]
    int* status;
};

struct NormRotateArgs {
    int tokens, heads, kv_heads, dim, rot, page_size;
    long long num_slots;                     // slots of the cache
    bool bf16, norm, interleaved;
    float eps;
    const void *q, *k, *v;
    size_t q_stride, k_stride, v_stride;     // elements from token to token
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t* positions;
    const int64_t* slots;
    void *q_out, *k_cache, *v_cache;
    size_t k_page_stride, v_page_stride;     // elements
    int* status;
};

struct ChunkAttnArgs {
    int batch, tokens, heads, kv_heads, dim, num_pages, page_size, table_cols;
    bool bf16;
    const void *q, *k_cache, *v_cache;
    size_t k_page_stride, v_page_stride;     // elements
    const int32_t *block_table, *context_lens, *cu_seqlens;
    float scale;
    void* out;
    void* workspace;
    int* status;
};

cudaError_t launch_page_fork(const PageForkArgs& a, cudaStream_t stream);
cudaError_t launch_page_release(const PageReleaseArgs& a, cudaStream_t stream);
cudaError_t launch_cache_copy(const CacheCopyArgs& a, cudaStream_t stream);
cudaError_t launch_keep_path(const KeepPathArgs& a, cudaStream_t stream);
// whether a call's CTAs can be numbered
bool cache_copy_fits(const CacheCopyArgs& a);
bool keep_path_fits(const KeepPathArgs& a);
cudaError_t launch_norm_rotate(const NormRotateArgs& a, cudaStream_t stream);
// bf16 on the tensor cores (kda_chunk_attn_tc.cu), fp32 on the CUDA cores (kda_chunk_attn.cu)
cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t stream);
cudaError_t launch_chunk_attn_tc(const ChunkAttnArgs& a, cudaStream_t stream);
// whether the tables hold no more than the kernels count
bool chunk_attn_fits(const ChunkAttnArgs& a);
bool chunk_attn_tc_fits(const ChunkAttnArgs& a);
size_t chunk_attn_workspace_bytes(const ChunkAttnArgs& a);
size_t chunk_attn_tc_workspace_bytes(const ChunkAttnArgs& a);

}  // namespace kda
