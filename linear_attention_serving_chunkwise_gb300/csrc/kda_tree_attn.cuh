// How the tree-attention kernels share their work, and the join of what was split.
//
// A unit is one (sequence, key/value head, block of query rows); its tokens (the context and
// the draft nodes) are cut into tiles.  All tiles of all units form one line (sequence-major,
// then head, then row block), and CTA c of N takes the tiles [T c / N, T (c + 1) / N): every
// CTA gets the same number of tiles (one more or less) whatever the mix of lengths, a long sequence is
// split over many CTAs and a short one is not.  The context lengths live on the device, so
// each CTA works the cut out for itself from two passes over them.
//
// A unit that lies within one CTA's range is finished there.  Of any other, each CTA leaves
// its part (running maximum, sum and unnormalised output per row, fp32) in the workspace:
// slot 2 c when the unit began before the CTA's range, slot 2 c + 1 otherwise, so a CTA
// has at most two.  join_kernel then joins a unit's parts in the order of its tiles.
#pragma once

#include "kda_draft_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace attn {

struct Shape {
    int BM;        // query rows of a unit
    int BN;        // tokens of a tile
    int ctas;      // CTAs that share the line
};

// rows of a (sequence, head): K nodes x G query heads, row = node * G + head of the group
__host__ __device__ __forceinline__ int row_blocks(const TreeAttnArgs& a, int BM)
{
    return (a.nodes * (a.heads / a.kv_heads) + BM - 1) / BM;
}

// tokens of sequence b, or 0 for a length that its table cannot hold (the sequence is skipped)
__device__ __forceinline__ int seq_tokens(const TreeAttnArgs& a, int b, bool& ok)
{
    const int c = a.context_lens[b];
    ok = c >= 0 && (long long)c + a.nodes <= (long long)a.table_cols * a.page_size;
    return ok ? c + a.nodes : 0;
}
__device__ __forceinline__ int seq_tiles(const TreeAttnArgs& a, int b, int BN)
{
    bool ok;
    const int n = seq_tokens(a, b, ok);
    return n > 0 ? (n + BN - 1) / BN : 1;       // a skipped sequence still gets its zero rows
}

__device__ __forceinline__ long long line_start(long long T, int c, int N) { return T * c / N; }
// the CTA whose range holds tile s
__device__ __forceinline__ int line_owner(long long T, long long s, int N) { return (int)(((s + 1) * N - 1) / T); }

// One warp: the total number of tiles, and the sequence b that holds tile `want` (< total)
// with the line's position at b's start.  want < 0: the total alone.
__device__ __forceinline__ long long line_total(const TreeAttnArgs& a, int BN, int per_seq, int lane)
{
    long long sum = 0;
    for (int b = lane; b < a.batch; b += 32) sum += seq_tiles(a, b, BN);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum * per_seq;
}
__device__ __forceinline__ void line_find(const TreeAttnArgs& a, int BN, int per_seq, long long want, int lane, int& seq,
                                          long long& start)
{
    long long base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const long long n = b < a.batch ? (long long)seq_tiles(a, b, BN) * per_seq : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > want);
        if (past) {
            const int src = __ffs(past) - 1;
            seq = b0 + src;
            start = base + __shfl_sync(0xffffffffu, incl - n, src);
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    seq = a.batch;
    start = base;
}

// A CTA's part of one unit: tiles [first, last) of the unit's tiles.
struct Piece {
    int b, hk, r0;          // sequence, cache head, first query row
    int first, last;
    int n, ctx;             // tokens of the sequence (0: skipped) and how many of them are context
    bool seq_ok, whole;     // whole: the unit lies within this CTA's range
    int slot;               // workspace slot of the part, when not whole
};

// Walks a CTA's range piece by piece.  begin() needs a full warp; next() any thread.
struct Line {
    long long hi, lo, at, b0;
    int b, per_seq, rb;

    __device__ __forceinline__ void begin(const TreeAttnArgs& a, const Shape& sh, int cta, int lane)
    {
        rb = row_blocks(a, sh.BM);
        per_seq = rb * a.kv_heads;
        const long long T = line_total(a, sh.BN, per_seq, lane);
        lo = at = line_start(T, cta, sh.ctas);
        hi = line_start(T, cta + 1, sh.ctas);
        line_find(a, sh.BN, per_seq, lo, lane, b, b0);
    }
    __device__ __forceinline__ bool next(const TreeAttnArgs& a, const Shape& sh, int cta, Piece& p)
    {
        if (at >= hi) return false;
        long long tiles = seq_tiles(a, b, sh.BN);
        while (at >= b0 + tiles * per_seq) {
            b0 += tiles * per_seq;
            tiles = seq_tiles(a, ++b, sh.BN);
        }
        const int u = (int)((at - b0) / tiles);
        const long long us = b0 + u * tiles, ue = us + tiles;
        p.b = b;
        p.hk = u / rb;
        p.r0 = (u % rb) * sh.BM;
        p.first = (int)(at - us);
        p.last = (int)(min(hi, ue) - us);
        p.n = seq_tokens(a, b, p.seq_ok);
        p.ctx = p.n - a.nodes;
        p.whole = us >= lo && ue <= hi;
        p.slot = 2 * cta + (us < lo ? 0 : 1);
        at = us + p.last;
        return true;
    }
};

// workspace: for each of 2 * ctas slots, BM maxima, BM sums, then BM x D outputs
__host__ __device__ __forceinline__ size_t slot_floats(int BM, int D) { return (size_t)BM * (D + 2); }

// Joins the units that cross a boundary of the line: CTA (c, y) looks at the boundary at the
// start of range c and, if that is the first boundary inside its unit, joins rows
// [y * rows, ...) of the unit, a warp to a row.  Maxima, sums and outputs are joined in tile
// order: m = max m_i, o = sum e^{m_i - m} o_i / sum e^{m_i - m} l_i.
template <typename Tout, int D>
__global__ void __launch_bounds__(256) join_kernel(TreeAttnArgs a, Shape sh)
{
    constexpr int C = D / 32;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int G = a.heads / a.kv_heads, rb = row_blocks(a, sh.BM), per_seq = rb * a.kv_heads;
    const int c = blockIdx.x + 1;
    const long long T = line_total(a, sh.BN, per_seq, lane);
    const long long cut = line_start(T, c, sh.ctas);
    if (cut >= T || cut == line_start(T, c - 1, sh.ctas)) return;   // the end, or the same cut again
    int b;
    long long b0;
    line_find(a, sh.BN, per_seq, cut, lane, b, b0);
    const int tiles = seq_tiles(a, b, sh.BN);
    const int u = (int)((cut - b0) / tiles);
    const long long s = b0 + (long long)u * tiles, e = s + tiles;
    if (s == cut) return;                                            // between two units: nothing is split
    const int c0 = line_owner(T, s, sh.ctas);
    if (c != c0 + 1) return;                                         // not the unit's first cut
    const int c1 = line_owner(T, e - 1, sh.ctas);
    const int hk = u / rb, r0 = (u % rb) * sh.BM;
    const int rows = min(sh.BM, a.nodes * G - r0);
    const float* ws = static_cast<const float*>(a.workspace);
    const size_t sf = slot_floats(sh.BM, D);
    for (int r = blockIdx.y * (blockDim.x / 32) + w; r < rows; r += gridDim.y * (blockDim.x / 32)) {
        float m = -INFINITY, l = 0.f, o[C] = {};
        for (int x = c0; x <= c1; ++x) {
            const long long lo = line_start(T, x, sh.ctas);
            if (lo == line_start(T, x + 1, sh.ctas)) continue;       // an empty range
            const float* p = ws + sf * (2 * (size_t)x + (s < lo ? 0 : 1));
            const float pm = p[r], pl = p[sh.BM + r];
            const float nm = fmaxf(m, pm), base = nm == -INFINITY ? 0.f : nm;
            const float f0 = exp2f(m - base), f1 = exp2f(pm - base);
            l = l * f0 + pl * f1;
#pragma unroll
            for (int k = 0; k < C; ++k) o[k] = o[k] * f0 + p[2 * sh.BM + (size_t)r * D + lane + 32 * k] * f1;
            m = nm;
        }
        const int row = r0 + r;
        Tout* dst = static_cast<Tout*>(a.out) + (((size_t)b * a.nodes + row / G) * a.heads + hk * G + row % G) * D;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // nothing to attend to: zeros; NaN stays
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const float y = l == 0.f ? 0.f : o[k] * inv;
            if constexpr (sizeof(Tout) == 2) dst[lane + 32 * k] = __float2bfloat16_rn(y);
            else dst[lane + 32 * k] = y;
        }
    }
}

}  // namespace attn
}  // namespace kda
