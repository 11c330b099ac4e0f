// Internal launchers of the draft-step operators (host side).  Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct PageTablesArgs {
    int batch, table_cols, num_free, page_size, max_tokens;
    const int32_t *context_lens, *new_lens, *pages_held, *free_pages;
    int32_t* block_table;
    int64_t* slot_map;
    int32_t *cu_seqlens, *pages_held_out, *pages_taken;
    int* status;
};

struct VerifyArgs {
    int batch, nodes, vocab;
    const float *target, *draft;        // [B, K+1, V]; [B, K, V] or nullptr
    const int32_t *tokens, *parents;    // [B, K]
    const float *uniforms, *noise;      // [B, K]; [B, V]
    int32_t *path, *n_accept, *next_token;
    int* status;
};

struct TreeDecodeArgs {
    int batch, nodes, num_heads, dk, dv;
    bool bf16;
    const void *q, *k, *v;              // [B, K, H, d]
    const float *g, *beta;              // [B, K, H, dk], [B, K, H]
    const int32_t* parents;             // [B, K]
    const float* state;                 // [B, H, dk, dv], only read
    float *out, *writes;                // [B, K, H, dv] each
    int* status;
    int prologue;                       // KDA_PROLOGUE_* bits
    const float* gate;                  // output gate logits [B, K, H, dv], or nullptr
};

struct TreeCommitArgs {
    int batch, nodes, num_heads, dk, dv;
    bool bf16;
    const void* k;                      // [B, K, H, dk]
    const float *g, *writes;            // [B, K, H, dk], [B, K, H, dv]
    const int32_t *path, *n_accept;     // [B, K], [B]
    float* state;                       // [B, H, dk, dv] in place
    int* status;
    int prologue;                       // KDA_PROLOGUE_QK_L2NORM and G_LOGITS
};

struct TreeAttnArgs {
    int batch, nodes, heads, kv_heads, dim, num_pages, page_size, table_cols;
    bool bf16;
    const void *q, *k_cache, *v_cache;
    size_t k_page_stride, v_page_stride;   // elements
    const int32_t *block_table, *context_lens, *parents;
    float scale;
    void* out;
    void* workspace;
    int* status;
};

// Sets up a kernel on the current device at its first call there (its dynamic shared memory, and
// that it starts with `regs` registers a thread when that matters); later calls cost a lookup.
struct KernelSetup {
    unsigned long long done = 0;   // a bit per device; a race only repeats the set-up
    template <typename F>
    cudaError_t operator()(F* kernel, size_t smem, int regs = 0)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess || (dev < 64 && (__atomic_load_n(&done, __ATOMIC_RELAXED) >> dev & 1))) return e;
        if (regs) {
            cudaFuncAttributes at;
            if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
            if (at.numRegs != regs) return cudaErrorLaunchOutOfResources;
        }
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELAXED);
        return cudaSuccess;
    }
};

// the device status word of the current device (kda_api.cu)
int* device_status_ptr();

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);
// dk = 128 on the tensor cores (kda_tree_step_tc.cu), dk = 64 on the CUDA cores
cudaError_t launch_tree_decode(const TreeDecodeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_decode_tc(const TreeDecodeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t stream);
// bf16 on the tensor cores (kda_tree_attn_tc.cu), fp32 on the CUDA cores
cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t stream);
// whether the tables could hold no more than the kernels count
bool tree_attn_fits(const TreeAttnArgs& a);
bool tree_attn_tc_fits(const TreeAttnArgs& a);
cudaError_t launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t stream);
size_t tree_attn_tc_workspace_bytes(int nodes, int group, int dim);
size_t tree_attn_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int dim, bool bf16);

}  // namespace kda
