// What the tensor-core attention kernels (draft trees, chunks of prompts) share: the cache's rows into swizzled
// tiles, the rows' transpose before a store, the tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_draft_sm100.cuh"

namespace kda {
namespace attn {

using namespace sm100;

constexpr int kTileTokens = 128;

struct Maps {
    CUtensorMap k, v;       // [pages][page_size][kv_heads][D], boxes of box_rows x 64 channels
    int box_rows;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there)
{
    const int n = there ? 16 : 0;                   // 0: the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7f80u) != 0x7f80u; }

// Where a tile's tokens lie: lane l of producer warp w has token 32 w + l.
struct Rows {
    size_t koff, voff;      // elements from the caches' starts
    unsigned exists, lost;  // of the warp's 32 tokens: on a page; without one although the sequence has them
};

// token `pos` of a sequence whose keys end before `end`, on page `id`; a is the call's, hk the cache head
template <typename Args>
__device__ __forceinline__ Rows rows_of(const Args& a, int hk, int pos, int end, int id, size_t row_stride, int D)
{
    const bool there = id >= 0 && id < a.num_pages;
    const size_t in_page = (size_t)(pos % a.page_size) * row_stride + (size_t)hk * D;
    Rows r;
    r.lost = __ballot_sync(0xffffffffu, !there && pos < end);
    r.exists = __ballot_sync(0xffffffffu, there);
    r.koff = there ? (size_t)id * a.k_page_stride + in_page : 0;
    r.voff = there ? (size_t)id * a.v_page_stride + in_page : 0;
    return r;
}

__device__ __forceinline__ void note_row(uint32_t* bad_nodes, int i) { atomicOr(bad_nodes + (i >> 5), 1u << (i & 31)); }

// The warp's 32 rows of a tile through registers; rows that do not exist become zero.  In the
// rows that only some queries see (the first in row `node0`, which may be negative) non-finite values become
// zero too and are noted, a bit each from `node0` on.
template <int D>
__device__ __forceinline__ void copy_rows(uint8_t* dst, const __nv_bfloat16* src, size_t off, unsigned exists, int w, int lane,
                                          int node0, uint32_t* bad_nodes)
{
    constexpr int CH = D / 8, RPI = 32 / CH;        // 16-byte chunks of a row; rows a warp copies at once
    const int sub = lane / CH, chunk = lane % CH;
    uint32_t bad = 0;
    for (int i0 = 0; i0 < 32; i0 += 8 * RPI) {
        uint4 x[8];                                 // eight loads in flight
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = i0 + k * RPI + sub;
            const size_t o = __shfl_sync(0xffffffffu, off, r);
            x[k] = make_uint4(0, 0, 0, 0);
            if (exists >> r & 1) x[k] = *(reinterpret_cast<const uint4*>(src + o) + chunk);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = i0 + k * RPI + sub;
            if (32 * w + r >= node0) {
                uint32_t h[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool lo = finite_bf16(h[e]), hi = finite_bf16(h[e] >> 16);
                    if (!(lo && hi)) bad |= 1u << r;
                    h[e] = (lo ? h[e] & 0xffffu : 0u) | (hi ? h[e] & 0xffff0000u : 0u);
                }
                x[k] = make_uint4(h[0], h[1], h[2], h[3]);
            }
            *reinterpret_cast<uint4*>(dst + sw128_chunk(32 * w + r, chunk, 128)) = x[k];
        }
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad && lane == 0) {
        for (int r = 0; r < 32; ++r)
            if (bad >> r & 1) note_row(bad_nodes, 32 * w + r - node0);
    }
}

// The same for a V tile that came by TMA; rows past the last token (from row `rows` on) become zero.
constexpr int kCleanThreads = 96;

template <int D>
__device__ __forceinline__ void clean_rows(uint8_t* tile, int node0, int rows, int t, uint32_t* bad_nodes)
{
    constexpr int CH = D / 8, STEP = kCleanThreads / CH;
    const int chunk = t % CH;
#pragma unroll 4
    for (int r = max(0, node0) + t / CH; r < kTileTokens; r += STEP) {
        uint4* at = reinterpret_cast<uint4*>(tile + sw128_chunk(r, chunk, 128));
        if (r >= rows) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4 x = *at;
        uint32_t h[4] = {x.x, x.y, x.z, x.w};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool lo = finite_bf16(h[e]), hi = finite_bf16(h[e] >> 16);
            bad |= !(lo && hi);
            h[e] = (lo ? h[e] & 0xffffu : 0u) | (hi ? h[e] & 0xffff0000u : 0u);
        }
        if (bad) {
            *at = make_uint4(h[0], h[1], h[2], h[3]);
            note_row(bad_nodes, r - node0);
        }
    }
}

__device__ __forceinline__ float max_of(const float (&x)[32])
{
    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        a0 = fmaxf(a0, fmaxf(x[k], x[k + 1]));
        a1 = fmaxf(a1, fmaxf(x[k + 2], x[k + 3]));
    }
    return fmaxf(a0, a1);
}

// One step of the transpose of 4 x 4 pieces over four lanes: lanes that differ in bit `by`
// exchange the later of two pieces for the earlier one.
__device__ __forceinline__ void swap_pieces(uint4& lo, uint4& hi, bool upper, int by)
{
    uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
    uint32_t* h = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? l[e] : h[e], by);
        if (upper) l[e] = got;
        else h[e] = got;
    }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Whether the cache can be read in boxes: pages of a multiple of 8 tokens; a map holds strides below 2^40 bytes.
template <typename Args>
bool in_boxes(const Args& a)
{
    const size_t most = ((size_t)1 << 40) / 2 - 1;
    return a.page_size % 8 == 0 && a.num_pages > 0 && a.k_page_stride <= most && a.v_page_stride <= most;
}

template <typename Args>
bool make_map(CUtensorMap* m, const void* cache, size_t page_stride, const Args& a, int rows)
{
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = (cuuint64_t)a.dim, H = (cuuint64_t)a.kv_heads;
    const cuuint64_t dims[4] = {D, H, (cuuint64_t)a.page_size, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {D * 2, H * D * 2, (cuuint64_t)page_stride * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, a.dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace kda
