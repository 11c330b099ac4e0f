// Pages and slots of the tokens a step appends to a paged cache, from request lengths.
//
// Request b has context_lens[b] tokens in the cache and appends new_lens[b]; it holds
// pages_held[b] pages and needs
//     need_b = max(0, ceil((context + new) / page_size) - held)
// more, which it takes from free_pages in request order, at the exclusive prefix sum of the
// needs.  Appended token t of request b lands in slot page * page_size + pos % page_size of
// logical position pos = context + t.
//
// Every CTA scans the requests by itself (16 bytes each, from L2) and then does its share of
// the slots and of the table entries: a page's id is read from the table where the request
// held it before the call and from free_pages where it is new, so no CTA needs another's
// writes and one launch does all.  Bound: latency, of the launch and of four dependent reads (the
// lengths, their scan, a page's id, the slot); the only stream is the slot map, 8 bytes a token.
// 48 requests of 16 tokens: 5.9 us a call inside a graph; 32 prompts of up to 16384 tokens (264 K
// slots, 2.1 MB): 10.7 us, 0.2 TB/s; 16384 requests of one token: 132 us, every CTA's scan and a warp to each
// request's entries.  2048 tokens a CTA: 129 CTAs for the prompts, one wave.
#include "kda_common.cuh"
#include "kda_draft_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kTokensPerCta = 2048;
constexpr int kPageTablesMaxBatch = 16384;   // KDA_PAGE_TABLES_MAX_BATCH: two words each in shared memory

__global__ void __launch_bounds__(kThreads) page_tables_kernel(PageTablesArgs a)
{
    // first appended token of each request, and its first index in free_pages (-1: refused)
    extern __shared__ int32_t sm[];
    int32_t* tok0 = sm;                    // [B + 1]
    int32_t* page0 = sm + a.batch + 1;     // [B]
    __shared__ long long warp_tok[kThreads / 32];
    __shared__ int warp_page[kThreads / 32];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const long long cap = (long long)a.table_cols * a.page_size;
    const bool first = blockIdx.x == 0;

    long long tok_base = 0;                // totals of the requests before this round's
    long long page_base = 0;
    int taken = 0;
    bool bad = false;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + t;
        int need = 0, held = 0, add = 0;
        bool fits = false;
        if (b < a.batch) {
            const int c = a.context_lens[b];
            add = a.new_lens[b];
            held = a.pages_held[b];
            const bool valid = c >= 0 && add >= 0 && held >= 0 && held <= a.table_cols && (long long)held * a.page_size >= c;
            bad |= !valid;
            if (!valid) add = 0;
            const long long total = (long long)c + add;
            fits = valid && total <= cap;
            if (fits) need = max(0, (int)((total + a.page_size - 1) / a.page_size) - held);
        }
        // inclusive scans over the round's requests
        long long ts = add;
        int ps = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long tu = __shfl_up_sync(0xffffffffu, ts, o);
            const int pu = __shfl_up_sync(0xffffffffu, ps, o);
            if (lane >= o) { ts += tu; ps += pu; }
        }
        if (lane == 31) { warp_tok[w] = ts; warp_page[w] = ps; }
        __syncthreads();
        long long tok_all = 0, tok_before = 0;
        int page_all = 0, page_before = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < w) { tok_before += warp_tok[i]; page_before += warp_page[i]; }
            tok_all += warp_tok[i];
            page_all += warp_page[i];
        }
        __syncthreads();                   // before the next round writes the warp totals
        if (b < a.batch) {
            const long long tok_incl = tok_base + tok_before + ts;
            const long long page_incl = page_base + page_before + ps;
            // first come, first served: past the last free page nobody takes any
            if (need > 0 && page_incl > a.num_free) fits = false;
            if (fits && need > 0) taken = max(taken, (int)page_incl);
            bad |= tok_incl > a.max_tokens;
            tok0[b + 1] = (int)min(tok_incl, (long long)INT32_MAX);
            page0[b] = fits ? (int)min(page_incl - need, (long long)a.num_free) : -1;
            if (first) a.pages_held_out[b] = fits ? held + need : held;
        }
        tok_base += tok_all;
        page_base += page_all;
    }
    if (t == 0) tok0[0] = 0;
    if (first) {
        if (bad) report_status(a.status, kDevBadSeqlens);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
        if (lane == 0) warp_page[w] = taken;
    }
    __syncthreads();
    if (first) {
        if (t == 0) {
            int m = 0;
            for (int i = 0; i < kThreads / 32; ++i) m = max(m, warp_page[i]);
            a.pages_taken[0] = m;
        }
        for (int b = t; b <= a.batch; b += kThreads) a.cu_seqlens[b] = tok0[b];
    }

    // table entries of the new pages: one warp per request
    for (int b = blockIdx.x * (kThreads / 32) + w; b < a.batch; b += gridDim.x * (kThreads / 32)) {
        const int p0 = page0[b];
        if (p0 < 0) continue;
        const int held = a.pages_held[b];
        // (its own new tokens: tok0's difference is not them where the sum has passed 32 bits)
        const int need = max(0, (int)(((long long)a.context_lens[b] + a.new_lens[b] + a.page_size - 1) / a.page_size) - held);
        for (int j = lane; j < need; j += 32) a.block_table[(size_t)b * a.table_cols + held + j] = a.free_pages[p0 + j];
    }

    // slots
    const long long end = min((long long)a.max_tokens, (long long)(blockIdx.x + 1) * kTokensPerCta);
    int lo = 0;
    for (long long i = (long long)blockIdx.x * kTokensPerCta + t; i < end; i += kThreads) {
        long long slot = -1;
        if (i < tok0[a.batch]) {
            int hi = a.batch;              // the request with tok0[b] <= i < tok0[b + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (tok0[mid] <= i) lo = mid; else hi = mid;
            }
            const int b = lo, p0 = page0[b];
            if (p0 >= 0) {
                // (a position may pass 31 bits where the context is near them, but not 32; its page does not)
                const uint32_t pos = (uint32_t)a.context_lens[b] + (uint32_t)(i - tok0[b]);
                const int pg = (int)(pos / (uint32_t)a.page_size), held = a.pages_held[b];
                const long long id = pg < held ? a.block_table[(size_t)b * a.table_cols + pg] : a.free_pages[p0 + pg - held];
                slot = id * a.page_size + (pos - (uint32_t)pg * (uint32_t)a.page_size);
            }
        }
        a.slot_map[i] = slot;
    }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream)
{
    const size_t smem = (size_t)(2 * a.batch + 1) * sizeof(int32_t);
    static_assert((2 * kPageTablesMaxBatch + 1) * 4 <= 227 * 1024 - 1024, "the scan fits shared memory");
    static KernelSetup setup;
    const cudaError_t e = setup(page_tables_kernel, (2 * kPageTablesMaxBatch + 1) * sizeof(int32_t));
    if (e != cudaSuccess) return e;
    const int grid = a.max_tokens > kTokensPerCta ? (int)(((long long)a.max_tokens + kTokensPerCta - 1) / kTokensPerCta) : 1;
    page_tables_kernel<<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
