// Rows of the paged caches moved in place, in all layers at once: the filled part of a page that a fork
// copies, and the kept nodes' rows of a step of drafts.
#include "kda_common.cuh"
#include "kda_prompt_launch.h"

namespace kda {
namespace {

// ------------------------------------------------------------------ copies of pages
// A CTA moves 32 KB of one (copy, layer, K or V): eight 16-byte loads in flight a thread.  Bound: HBM (96 forks, 133 MB, with
// the forks themselves 23.5 us, 5.7 TB/s).
constexpr int kCopyThreads = 256, kCopyLoads = 8, kCopyBytes = kCopyThreads * kCopyLoads * 16;

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(CacheCopyArgs a, unsigned parts)
{
    const unsigned unit = blockIdx.x / parts, part = blockIdx.x - unit * parts;
    const int i = (int)(unit / (2u * a.c.layers)), x = (int)(unit - (unsigned)i * 2u * a.c.layers), layer = x >> 1;
    const int src = a.copies[3 * i], dst = a.copies[3 * i + 1], rows = a.copies[3 * i + 2];
    if (rows == 0) return;
    if (rows < 0 || rows > a.c.page_size || src < 0 || src >= a.c.num_pages || dst < 0 || dst >= a.c.num_pages) {
        if (x == 0 && part == 0 && threadIdx.x == 0) report_status(a.status, kDevBadSeqlens);
        return;
    }
    const size_t bytes = (size_t)rows * a.c.row, at = (size_t)part * kCopyBytes;
    if (at >= bytes || src == dst) return;
    const size_t page = x & 1 ? a.c.v_page : a.c.k_page;
    uint8_t* base = (x & 1 ? a.c.v : a.c.k) + (size_t)layer * (x & 1 ? a.c.v_layer : a.c.k_layer);
    const uint4* from = reinterpret_cast<const uint4*>(base + (size_t)src * page + at);
    uint4* to = reinterpret_cast<uint4*>(base + (size_t)dst * page + at);
    const int n = (int)(min(bytes - at, (size_t)kCopyBytes) / 16);
    uint4 y[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int j = threadIdx.x + k * kCopyThreads;
        if (j < n) y[k] = from[j];
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int j = threadIdx.x + k * kCopyThreads;
        if (j < n) to[j] = y[k];
    }
}

// ------------------------------------------------------------------ kept paths
// Entry e of a path is node path[e] >= e (a path goes up), so a row only moves towards the front, and a row
// that is written has been read by then: a thread owns 16 bytes of every row and goes through the
// entries in order, eight rows read before they are written.  Bound: HBM, or the launch and three dependent reads: 256 paths
// in eight layers (98 MB) 20.7 us, 4.7 TB/s (14.4 us where the rows are in L2), 4 paths 4.1 us.  Half the threads with two chunks
// each 21.1 us, a quarter with four 20.8, sixteen rows in flight 24.6.
constexpr int kKeepThreads = 128, kKeepLoads = 8, kMostNodes = 64;

__global__ void __launch_bounds__(kKeepThreads) keep_path_kernel(KeepPathArgs a, unsigned parts)
{
    __shared__ long long s_src[kMostNodes], s_dst[kMostNodes];   // rows that move: offsets of the two in the cache
    __shared__ int s_count;
    const int t = threadIdx.x;
    const unsigned unit = blockIdx.x / parts, part = blockIdx.x - unit * parts;
    const int b = (int)(unit / (2u * a.c.layers)), x = (int)(unit - (unsigned)b * 2u * a.c.layers), layer = x >> 1;
    const int n = a.n_accept[b];
    const size_t page = x & 1 ? a.c.v_page : a.c.k_page;
    if (t < 32) {
        // two entries to a lane; those that stay where they are need nothing
        int moved = 0;
        bool bad = n < 0 || n > a.nodes;
        for (int e0 = 0; e0 < (bad ? 0 : n); e0 += 32) {
            const int e = e0 + t;
            bool go = false;
            long long so = 0, to = 0;
            if (e < n) {
                const int p = a.path[(size_t)b * a.nodes + e], last = e ? a.path[(size_t)b * a.nodes + e - 1] : -1;
                bad |= p <= last || p >= a.nodes;
                if (p > last && p < a.nodes && p >= 0 && p != e) {
                    const long long all = (long long)a.c.num_pages * a.c.page_size;
                    const long long s = a.slots[(size_t)b * a.nodes + p], d = a.slots[(size_t)b * a.nodes + e];
                    bad |= s < 0 || s >= all || d < 0 || d >= all;
                    go = s != d;
                    so = s / a.c.page_size * (long long)page + s % a.c.page_size * (long long)a.c.row;
                    to = d / a.c.page_size * (long long)page + d % a.c.page_size * (long long)a.c.row;
                }
            }
            const unsigned gone = __ballot_sync(0xffffffffu, go);
            if (go) {
                const int at = moved + __popc(gone & ((1u << t) - 1u));
                s_src[at] = so;
                s_dst[at] = to;
            }
            moved += __popc(gone);
        }
        bad = __any_sync(0xffffffffu, bad);
        if (t == 0) {
            s_count = bad ? 0 : moved;
            if (bad && x == 0 && part == 0) report_status(a.status, kDevBadSeqlens);
        }
    }
    __syncthreads();
    const size_t at = ((size_t)part * kKeepThreads + t) * 16;
    if (at >= a.c.row) return;
    uint8_t* base = (x & 1 ? a.c.v : a.c.k) + (size_t)layer * (x & 1 ? a.c.v_layer : a.c.k_layer) + at;
    for (int e0 = 0; e0 < s_count; e0 += kKeepLoads) {
        uint4 y[kKeepLoads];
#pragma unroll
        for (int k = 0; k < kKeepLoads; ++k)
            if (e0 + k < s_count) y[k] = *reinterpret_cast<const uint4*>(base + s_src[e0 + k]);
#pragma unroll
        for (int k = 0; k < kKeepLoads; ++k)
            if (e0 + k < s_count) *reinterpret_cast<uint4*>(base + s_dst[e0 + k]) = y[k];
    }
}

}  // namespace

// CTAs of a call; their numbers are 31-bit
static double copy_ctas(const CacheCopyArgs& a, size_t& parts)
{
    parts = ((size_t)a.c.page_size * a.c.row + kCopyBytes - 1) / kCopyBytes;
    return 2.0 * parts * a.c.layers * a.n;
}
static double keep_ctas(const KeepPathArgs& a, size_t& parts)
{
    parts = (a.c.row / 16 + kKeepThreads - 1) / kKeepThreads;
    return 2.0 * parts * a.c.layers * a.batch;
}
bool cache_copy_fits(const CacheCopyArgs& a) { size_t parts; return copy_ctas(a, parts) < 2147483648.0; }
bool keep_path_fits(const KeepPathArgs& a) { size_t parts; return keep_ctas(a, parts) < 2147483648.0; }

cudaError_t launch_cache_copy(const CacheCopyArgs& a, cudaStream_t stream)
{
    size_t parts;
    const unsigned ctas = (unsigned)copy_ctas(a, parts);
    cache_copy_kernel<<<ctas, kCopyThreads, 0, stream>>>(a, (unsigned)parts);
    return cudaGetLastError();
}

cudaError_t launch_keep_path(const KeepPathArgs& a, cudaStream_t stream)
{
    size_t parts;
    const unsigned ctas = (unsigned)keep_ctas(a, parts);
    keep_path_kernel<<<ctas, kKeepThreads, 0, stream>>>(a, (unsigned)parts);
    return cudaGetLastError();
}

}  // namespace kda
