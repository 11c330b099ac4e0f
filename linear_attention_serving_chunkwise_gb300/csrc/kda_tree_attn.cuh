// How the tree-attention kernels share their work, and the join of what was split.
//
// A unit is one (sequence, key/value head, block of query rows); its tokens (the context and
// the draft nodes) are cut into tiles.  All units' tiles form one line (sequence-major, then
// head, then row block; before a unit's tiles a few places stand for its fixed cost), and CTA
// c of N takes the places [start(c), start(c + 1)) with start(c) = floor(T c / N): every CTA
// gets the same share (a place more or less) whatever the mix of lengths, a long sequence
// is split over many CTAs and a short one is not.  The context lengths live on the device, so each
// CTA works its cut out for itself (one warp's scan over the lengths, about 1 us for 64).
//
// A unit that lies within one CTA's range is finished there.  Of any other, each CTA leaves
// its part (running maximum, sum and unnormalised output per row, fp32) in the workspace:
// slot 2 c when the unit began before the CTA's range, slot 2 c + 1 otherwise, so a CTA has
// at most two, and a record for the join.  join_kernel joins a unit's parts in tile order.
#pragma once

#include "kda_attn_join.cuh"
#include "kda_draft_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace attn {

// rows of a (sequence, head): K nodes x G query heads, row = node * G + head of the group
__host__ __device__ __forceinline__ int row_blocks(const TreeAttnArgs& a, int BM)
{
    return (a.nodes * (a.heads / a.kv_heads) + BM - 1) / BM;
}

// The line's positions are 32-bit: false for a call whose tables could hold more tiles (2^31
// tiles of 64 tokens would read a cache of terabytes).
__host__ __forceinline__ bool line_fits(const TreeAttnArgs& a, const Shape& sh)
{
    const double tiles = (double)a.table_cols * a.page_size / sh.BN + 1 + sh.head;
    return tiles * row_blocks(a, sh.BM) * a.kv_heads * a.batch < 2147483647.0;
}

// Tokens that a sequence may have: positions are 32-bit, and the last tile's go past the end by less than this
// leaves (a lane of the copies numbers up to 31 boxes of 128 tokens past the tile's first).
constexpr int kMostTokens = 0x7fffffff - 8191;

// tokens of sequence b, or 0 for a length that its table cannot hold (the sequence is skipped)
__device__ __forceinline__ int seq_tokens(const TreeAttnArgs& a, int b, bool& ok)
{
    const int c = __ldg(a.context_lens + b);
    ok = c >= 0 && c <= kMostTokens - a.nodes && (long long)c + a.nodes <= (long long)a.table_cols * a.page_size;
    return ok ? c + a.nodes : 0;
}
__device__ __forceinline__ int tiles_of(int n, int BN) { return n > 0 ? (n - 1) / BN + 1 : 1; }   // a skipped sequence still gets its zero rows
// places of one of its units
__device__ __forceinline__ int unit_places(int n, const Shape& sh) { return tiles_of(n, sh.BN) + sh.head; }
__device__ __forceinline__ int unit_places(const TreeAttnArgs& a, int b, const Shape& sh)
{
    bool ok;
    return unit_places(seq_tokens(a, b, ok), sh);
}

// floor(T c / N) without a product past 32 bits
__device__ __forceinline__ int line_start(int T, int c, int N)
{
    const int q = T / N, r = T - q * N;
    return q * c + r * c / N;
}

// A CTA's part of one unit: tiles [first, last) of the unit's tiles.
struct Piece {
    int b, hk, r0;          // sequence, cache head, first query row
    int first, last;
    int n, ctx;             // tokens of the sequence (0: skipped) and how many of them are context
    bool seq_ok;
    bool begins, ends;      // the unit's first, last tile is in this CTA's range
    int slot;               // workspace slot of the part, when it is not the whole unit
    int rest;               // the unit's tiles past this CTA's range
    __device__ __forceinline__ bool whole() const { return begins && ends; }
};

// Walks a CTA's range piece by piece.
struct Line {
    int hi, lo, at, b0;
    int b, per_seq, rb;
    int T, N;               // places, and CTAs that share them: no more than there are places

    // a full warp
    __device__ __forceinline__ void begin(const TreeAttnArgs& a, const Shape& sh, int cta, int lane)
    {
        rb = row_blocks(a, sh.BM);
        per_seq = rb * a.kv_heads;
        const int mine = lane < a.batch ? unit_places(a, lane, sh) : 0;    // of the first 32 sequences
        int sum = mine;
        for (int i = lane + 32; i < a.batch; i += 32) sum += unit_places(a, i, sh);
        T = __reduce_add_sync(0xffffffffu, sum) * per_seq;
        N = min(sh.ctas, T);
        if (cta >= N) {
            lo = hi = at = 0;
            return;
        }
        lo = at = line_start(T, cta, N);
        hi = line_start(T, cta + 1, N);
        // the sequence that holds place lo, and where it begins
        b = a.batch;
        b0 = 0;
        for (int i0 = 0; i0 < a.batch; i0 += 32) {
            const int i = i0 + lane, n = (i0 == 0 ? mine : i < a.batch ? unit_places(a, i, sh) : 0) * per_seq;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            const unsigned past = __ballot_sync(0xffffffffu, b0 + incl > lo);
            if (past) {
                const int src = __ffs(past) - 1;
                b = i0 + src;
                b0 += __shfl_sync(0xffffffffu, incl - n, src);
                break;
            }
            b0 += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    // any thread
    __device__ __forceinline__ bool next(const TreeAttnArgs& a, const Shape& sh, int cta, Piece& p)
    {
        while (at < hi) {
            p.n = seq_tokens(a, b, p.seq_ok);
            const int places = unit_places(p.n, sh);
            if (at >= b0 + places * per_seq) {
                b0 += places * per_seq;
                ++b;
                continue;
            }
            const int u = (at - b0) / places, us = b0 + u * places, ue = us + places;
            p.b = b;
            p.hk = rb == 1 ? u : u / rb;
            p.r0 = (u - p.hk * rb) * sh.BM;
            p.first = max(at - us - sh.head, 0);
            p.last = min(hi, ue) - us - sh.head;
            p.ctx = p.n - a.nodes;
            p.begins = us + sh.head >= lo;
            p.ends = ue <= hi;
            p.rest = max(ue - hi, 0);
            p.slot = 2 * cta + (p.begins ? 1 : 0);
            at = min(hi, ue);
            if (p.last > p.first) return true;      // (else only places of its head are here)
        }
        return false;
    }
};

// One thread of each CTA, piece by piece and once at the end.
struct Recorder {
    int R, BM;             // rows of a (sequence, head), and of a unit
    Record r = {};
    __device__ __forceinline__ Recorder(const TreeAttnArgs& a, const Shape& sh) : R(a.nodes * (a.heads / a.kv_heads)), BM(sh.BM) {}
    __device__ __forceinline__ void see(const Line& line, const Piece& p)
    {
        if (!p.begins || p.ends) return;
        // the CTA that holds the unit's last place
        const int end = line.hi + p.rest - 1;
        r.last = (int)((((long long)end + 1) * line.N - 1) / line.T);
        r.row0 = p.b * R + p.r0;
        r.hk = p.hk;
        r.rows = min(BM, R - p.r0);
    }
    __device__ __forceinline__ void leave(const TreeAttnArgs& a, int cta) { static_cast<Record*>(a.workspace)[cta] = r; }
};

}  // namespace attn
}  // namespace kda
