// Rows of a block table that share another row's first tokens, and rows cut short.
//
// shares[p] counts the rows that hold page p beyond the first, so a page that only page_tables
// handed out needs no entry.  A fork of `len` tokens adds the parent's floor(len / page_size) whole pages
// to the child by reference (shares + 1) and takes one page of its own for the rest, into which the
// parent's rows are to be copied: no row ever appends to a page that another holds.  A release gives
// back the entries from ceil(keep / page_size) on: shares - 1 each, and a page that nobody holds any more (its
// entry has become -1) is free.
#include <cooperative_groups.h>

#include "kda_common.cuh"
#include "kda_prompt_launch.h"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxRows = 16384;        // KDA_PAGE_TABLES_MAX_BATCH
constexpr int kBlock = 256;            // table columns that a warp takes at a time: eight reads in flight a lane

// (columns and pages go up to 2^31 - 1: what is added to them is added in 64 bits, or to an offset)
__host__ __device__ __forceinline__ int blocks_of(int cols) { return (int)((cols + (long long)kBlock - 1) / kBlock); }

// ------------------------------------------------------------------ forks
// As in page_tables, every CTA works the forks out for itself (12 bytes each, from L2) and then does
// its share of the table entries, so one launch does all.  Bound: latency, of the launch and of four dependent reads
// (the fork, its parent's pages held, the parent's entry, the share): 4 forks with the copies 8.3 us, 96 19.6 us (the copies' HBM).
constexpr int kForkThreads = 256, kForkWarps = kForkThreads / 32;
constexpr int kRefused = -2, kNoPage = -1;

struct ForkSmem {
    uint32_t child[kMaxRows / 32], twice[kMaxRows / 32];    // rows that are a child; of two forks or more
    int warp_need[kForkWarps];
    int taken;
    int page[1];                       // [forks]: index in free_pages, kNoPage or kRefused
};

__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(PageForkArgs a)
{
    extern __shared__ __align__(16) uint8_t raw[];
    ForkSmem& sm = *reinterpret_cast<ForkSmem*>(raw);
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, ps = a.page_size;
    const bool first = blockIdx.x == 0;
    const auto bit = [](const uint32_t* set, int i) { return set[i >> 5] >> (i & 31) & 1; };
    const int words = (a.rows + 31) / 32;
    for (int i = t; i < words; i += kForkThreads) sm.child[i] = sm.twice[i] = 0;
    if (t == 0) sm.taken = 0;
    __syncthreads();
    for (int i = t; i < a.forks; i += kForkThreads) {
        const int c = a.children[i];
        if (c < 0 || c >= a.rows) continue;
        const uint32_t m = 1u << (c & 31);
        if (atomicOr(&sm.child[c >> 5], m) & m) atomicOr(&sm.twice[c >> 5], m);
    }
    __syncthreads();

    int base = 0;                      // pages that the forks before this round need
    bool bad = false;
    for (int i0 = 0; i0 < a.forks; i0 += kForkThreads) {
        const int i = i0 + t;
        bool valid = false, need = false;
        if (i < a.forks) {
            const int p = a.parents[i], c = a.children[i], n = a.lens[i];
            valid = p >= 0 && p < a.rows && c >= 0 && c < a.rows && n >= 0;
            // a row that is forked in this call has no pages that could be forked from or written twice
            valid = valid && !bit(sm.child, p) && !bit(sm.twice, c) && a.pages_held[c] == 0;
            if (valid) {
                const int held = a.pages_held[p];
                valid = held >= 0 && held <= a.table_cols && (long long)held * ps >= n;
            }
            bad |= !valid;
            need = valid && n % ps != 0;
        }
        const unsigned ballot = __ballot_sync(0xffffffffu, need);
        if (lane == 0) sm.warp_need[w] = __popc(ballot);
        __syncthreads();
        int before = __popc(ballot & ((1u << lane) - 1u)), all = 0;
#pragma unroll
        for (int k = 0; k < kForkWarps; ++k) {
            if (k < w) before += sm.warp_need[k];
            all += sm.warp_need[k];
        }
        if (i < a.forks) {
            const int at = base + before;
            // first come, first served: past the last free page nobody takes any
            const bool got = need && at < a.num_free;
            sm.page[i] = !valid || (need && !got) ? kRefused : need ? at : kNoPage;
            if (got) atomicMax(&sm.taken, at + 1);
        }
        base += all;
        __syncthreads();               // before the next round writes the warps' counts
    }
    if (first) {
        if (bad) report_status(a.status, kDevBadSeqlens);
        if (t == 0) a.pages_taken[0] = sm.taken;
        for (int r = t; r < a.rows; r += kForkThreads)
            if (!bit(sm.child, r)) a.pages_held_out[r] = a.pages_held[r];
        for (int i = t; i < a.forks; i += kForkThreads) {
            const int page = sm.page[i], c = a.children[i], n = a.lens[i];
            int src = -1, dst = -1, rows = 0;
            if (page != kRefused) {
                a.pages_held_out[c] = n / ps + (page >= 0);
                if (page >= 0) {
                    const int s = a.block_table[(size_t)a.parents[i] * a.table_cols + n / ps], d = a.free_pages[page];
                    if (s >= 0 && s < a.num_pages && d >= 0 && d < a.num_pages) {
                        src = s;
                        dst = d;
                        rows = n % ps;
                    } else {
                        report_status(a.status, kDevBadSeqlens);
                    }
                }
            } else if (c >= 0 && c < a.rows) {
                a.pages_held_out[c] = a.pages_held[c];      // (the same value from every fork of this child)
            }
            a.copies[3 * i] = src;
            a.copies[3 * i + 1] = dst;
            a.copies[3 * i + 2] = rows;
        }
    }

    // the children's entries: a warp to kBlock columns of a fork
    const int blocks = blocks_of(a.table_cols);
    const long long items = (long long)a.forks * blocks;
    for (long long it = (long long)blockIdx.x * kForkWarps + w; it < items; it += (long long)gridDim.x * kForkWarps) {
        const int i = (int)(it / blocks), page = sm.page[i];
        if (page == kRefused) continue;
        const int full = a.lens[i] / ps, j0 = (int)(it % blocks) * kBlock;
        if (j0 > full) continue;
        const int32_t* src = a.block_table + (size_t)a.parents[i] * a.table_cols;
        int32_t* dst = a.block_table + (size_t)a.children[i] * a.table_cols;
        int id[kBlock / 32];
#pragma unroll
        for (int k = 0; k < kBlock / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            id[k] = j < full ? src[j] : j == full && page >= 0 ? a.free_pages[page] : -1;
        }
#pragma unroll
        for (int k = 0; k < kBlock / 32; ++k) {
            const int j = j0 + 32 * k + lane;
            if (j < full) {
                dst[j] = id[k];
                if (id[k] >= 0 && id[k] < a.num_pages) atomicAdd(a.shares + id[k], 1);
                else report_status(a.status, kDevBadSeqlens);
            } else if (j == full && page >= 0) {
                dst[j] = id[k];
            }
        }
    }
}

// ------------------------------------------------------------------ releases
// Three steps with a barrier of all threads between them:
//   1. what each row keeps (a row that would cut a page which others hold too is refused: appending to it would write
//      into their tokens; decided before any share changes);
//   2. shares - 1 for every entry given back;
//   3. the pages whose entry is below zero, in ascending order: each warp counts those of its stretch of pages, the counts
//      are exchanged, each warp writes its own behind those of the warps before it.
// Integer sums only, and no order of arrival shows in the outputs.
// One CTA for what it does in a few microseconds, else a cooperative grid: see kAlonePages.  Bound: latency, of the reads and
// of four grid barriers: 2048 rows in a pool of 600000 pages 15.5 us (pages given back twice 16.0; from call to call 18.4); a launch for each step, the last one a cluster of 16 CTAs, 27.
constexpr int kReleaseThreads = 1024, kReleaseWarps = kReleaseThreads / 32, kReleaseCtas = 152;
// One CTA alone up to these (GPU time): 4096 pages, 16 rows 8.4 us (a grid 13.9); 16384 pages, 64 rows of 128 14.0 (12.4), 512 rows
// 32.9 (12.7); 600000 pages, 2048 rows of 512 315 (18.6).
constexpr int kAlonePages = 8192;
constexpr long long kAloneEntries = 8192;

template <bool kGrid>
__global__ void __launch_bounds__(kReleaseThreads, 1) page_release_kernel(PageReleaseArgs a)
{
    __shared__ int warp_count[kReleaseWarps];
    __shared__ int s_before, s_total;
    const auto sync = [] {
        if constexpr (kGrid) cg::this_grid().sync();
        else __syncthreads();
    };
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, ps = a.page_size;
    const int ctas = kGrid ? gridDim.x : 1, cta = kGrid ? blockIdx.x : 0;
    const long long threads = (long long)ctas * kReleaseThreads, warps = (long long)ctas * kReleaseWarps;
    // (warp by warp over the CTAs, so that few items spread over all SMs)
    const int all_w = w * ctas + cta, all_t = all_w * 32 + lane;
    bool bad = false;

    for (long long r = all_t; r < a.rows; r += threads) {
        const int keep = a.keep_lens[r], held = a.pages_held[r];
        int left = held;
        if (keep < 0 || held < 0 || held > a.table_cols) {
            bad = true;
        } else {
            const int pages = (int)(((long long)keep + ps - 1) / ps);
            if (pages <= held) {
                left = pages;
                if (keep % ps) {       // (inside the last page that is held, too)
                    const int id = a.block_table[(size_t)r * a.table_cols + pages - 1];
                    if (id < 0 || id >= a.num_pages || a.shares[id] > 0) {
                        bad = true;
                        left = held;
                    }
                }
            }
        }
        a.pages_held_out[r] = left;
    }
    sync();

    // a warp to kBlock columns of a row
    const int blocks = blocks_of(a.table_cols);
    const long long items = (long long)a.rows * blocks;
    for (long long i = all_w; i < items; i += warps) {
        const int r = (int)(i / blocks), j0 = (int)(i % blocks) * kBlock, held = a.pages_held[r];
        if (held > a.table_cols || held <= j0) continue;
        const int from = max(__ldcg(a.pages_held_out + r), j0), n = min(held - j0, kBlock) - (from - j0);
        if (n <= 0) continue;
        const int32_t* row = a.block_table + (size_t)r * a.table_cols + from;
        int id[kBlock / 32];
#pragma unroll
        for (int x = 0; x < kBlock / 32; ++x) id[x] = 32 * x + lane < n ? row[32 * x + lane] : -1;
#pragma unroll
        for (int x = 0; x < kBlock / 32; ++x) {
            if (id[x] >= 0 && id[x] < a.num_pages) atomicSub(a.shares + id[x], 1);
            else bad |= 32 * x + lane < n;
        }
    }
    sync();

    // this warp's pages, `pages` from p0 on, in the order of the CTAs and of their warps
    const int each = (int)(((long long)a.num_pages + warps * 32 - 1) / (warps * 32)) * 32;
    const long long mine = (long long)cta * kReleaseWarps + w;
    const int p0 = (int)min((long long)a.num_pages, mine * each), pages = min(a.num_pages - p0, each);
    int32_t* const shares = a.shares + p0;
    int count = 0;
#pragma unroll 8
    for (int i = lane; i < pages; i += 32) count += __ldcg(shares + i) < 0;
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) warp_count[w] = count;
    __syncthreads();
    if (w == 0) {
        const int n = warp_count[lane];
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        warp_count[lane] = incl - n;
        if (lane == 31) {
            s_before = 0;
            s_total = incl;
            if (kGrid && cta < a.num_pages) a.freed[cta] = incl;    // (as scratch: the list is written once all have read it)
        }
    }
    if constexpr (kGrid) {
        sync();
        if (w == 0) {
            int before = 0, total = 0;
#pragma unroll
            for (int c = lane; c < kReleaseCtas; c += 32) {
                const int n = c < min(ctas, a.num_pages) ? __ldcg(a.freed + c) : 0;
                total += n;
                before += c < cta ? n : 0;
            }
            before = __reduce_add_sync(0xffffffffu, before);
            total = __reduce_add_sync(0xffffffffu, total);
            if (lane == 0) {
                s_before = before;
                s_total = total;
            }
        }
    }
    sync();
    int before = s_before + warp_count[w];
    const int total = s_total;
#pragma unroll 4
    for (int q = 0; q < pages; q += 32) {
        const int i = q + lane, s = i < pages ? __ldcg(shares + i) : 0;
        const unsigned gone = __ballot_sync(0xffffffffu, s < 0);
        if (s < 0) {
            a.freed[before + __popc(gone & ((1u << lane) - 1u))] = p0 + i;
            shares[i] = 0;
            bad |= s < -1;             // given back more often than it was held
        }
        before += __popc(gone);
    }
    for (long long i = total + (long long)cta * kReleaseThreads + t; i < a.num_pages; i += threads) a.freed[i] = -1;
    if (all_t == 0) a.num_freed[0] = total;
    // (one thread of a CTA reports: 150 thousand on one word took 20 us)
    if (__syncthreads_or(bad) && t == 0) report_status(a.status, kDevBadSeqlens);
}

}  // namespace

cudaError_t launch_page_fork(const PageForkArgs& a, cudaStream_t stream)
{
    static_assert(sizeof(ForkSmem) + kMaxRows * 4 <= 227 * 1024, "the forks fit shared memory");
    static KernelSetup setup;
    const cudaError_t e = setup(page_fork_kernel, sizeof(ForkSmem) + kMaxRows * sizeof(int));
    if (e != cudaSuccess) return e;
    const long long items = (long long)a.forks * blocks_of(a.table_cols), ctas = (items + kForkWarps - 1) / kForkWarps;
    const int grid = (int)(ctas < 1 ? 1 : ctas > 152 ? 152 : ctas);
    page_fork_kernel<<<grid, kForkThreads, sizeof(ForkSmem) + (size_t)a.forks * sizeof(int), stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_page_release(const PageReleaseArgs& a, cudaStream_t stream)
{
    if (a.num_pages <= kAlonePages && (long long)a.rows * a.table_cols <= kAloneEntries) {
        page_release_kernel<false><<<1, kReleaseThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_pages < kReleaseCtas ? (a.num_pages < 1 ? 1 : a.num_pages) : kReleaseCtas);   // (a word of scratch each)
    cfg.blockDim = dim3(kReleaseThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_release_kernel<true>, a);
}

}  // namespace kda
