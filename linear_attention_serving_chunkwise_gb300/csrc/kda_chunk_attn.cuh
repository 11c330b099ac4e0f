// How the chunk-attention kernels share their work.
//
// A unit is one (sequence, key/value head, block of the chunk's tokens): its query rows are
// (token, head of the group), as many whole tokens as a block of rows holds.  It reads the context and the chunk
// up to its own last token, in tiles.  All units form one line (sequence-major, then head, then block),
// in which a unit has a place for every token that it reads and `head` tiles' worth for its fixed cost; range r of N
// is the places [start(r), start(r + 1)), start(r) = floor(T r / N), and its work the tiles whose first token lies
// there.  So every range is the same share whatever the mix of chunks and contexts, and a causal block counts
// what it reads.  Places before a block are a quadratic in its number, so a range's start is found with a scan over the
// sequences and a bisection; lengths are read on the device.
//
// CTA c of C works the ranges c, c + C, c + 2 C ... in turn, as many waves of them as keep what
// all CTAs read at a time within L2 (kResident): the blocks of a chunk read the same keys and values, and in a single
// wave the CTAs would be spread over the whole line, each behind another's reads by more than L2 holds.
//
// Units that several ranges share are joined as those of the tree attention are (kda_attn_join.cuh): a range leaves its part of
// a unit that began before it in slot 2 r, of one that goes on past it in slot 2 r + 1.
#pragma once

#include "kda_attn_join.cuh"
#include "kda_prompt_launch.h"

namespace kda {
namespace chunk {

using attn::Record;
using attn::Shape;

// Tokens that a sequence may have: positions are 32-bit, and the copies number a little past the last tile.
constexpr int kMostTokens = 0x7fffffff - 8191;
constexpr int kMaxWaves = 8;
// Bytes of keys and values that the CTAs may be at work on together (24, 48 and 96 MB: 3.03, 3.03, 3.32 ms for 2048 tokens after 131072;
// 4.29, 4.29, 4.25 for 12 sequences after up to 16384), and the least tiles to a range of several waves.
constexpr float kResident = 48e6f;
constexpr int kLeastTiles = 24;

// floor(a / b) for a >= 0, b > 0.  Not in line: the setting-up of a range has five of them, every CTA waits for it, and code
// that runs once costs its way from memory.
static __device__ __noinline__ long long quotient(long long a, long long b)
{
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// (tiles are powers of two)
__device__ __forceinline__ int tile_bits(const Shape& sh) { return 31 - __clz(sh.BN); }

// One sequence of the call: its chunk and context, and the line's numbers for one of its (sequence, head)s.
struct Seq {
    int tok0, n, ctx;       // first row of q, tokens of the chunk, cached tokens before it
    bool ok;                // false: a length that the table cannot hold; its rows become zero
    int blocks;
    // block j (from 0) has head + base + step (j + 1) places, the last head + last
    long long base, step, last;

    __device__ __forceinline__ void read(const ChunkAttnArgs& a, int b, int TB)
    {
        tok0 = __ldg(a.cu_seqlens + b);
        n = (int)((uint32_t)__ldg(a.cu_seqlens + b + 1) - (uint32_t)tok0);
        ctx = __ldg(a.context_lens + b);
        ok = ctx >= 0 && n >= 0 && ctx <= kMostTokens - n && (long long)ctx + n <= (long long)a.table_cols * a.page_size;
        blocks = n > 0 ? (n - 1) / TB + 1 : 0;
        base = ok ? ctx : 1;
        step = ok ? TB : 0;
        last = ok ? (long long)ctx + n : 1;
    }
    // places before block j < blocks
    __device__ __forceinline__ long long before(int j, long long head) const
    {
        return j * (head + base) + step * ((long long)j * (j + 1) / 2);
    }
    __device__ __forceinline__ long long per_head(long long head) const { return blocks ? before(blocks - 1, head) + head + last : 0; }
};

// A range's part of one unit: tiles [first, last) of `tiles`.
struct Piece {
    int b, hk;
    int tok, tokens;        // first token of the block within the chunk, and how many
    int row0;               // q's row of that token
    int ctx;                // of the sequence
    bool ok;
    int first, last, tiles;
    int range, slot;        // the range, and the workspace slot of the part when it is not the whole unit
    int seen, common;       // tokens that the block's last one sees, itself included, and those that all see
    long long at;           // the line's place of the unit's first token
    __device__ __forceinline__ bool begins() const { return first == 0; }
    __device__ __forceinline__ bool ends() const { return last == tiles; }
    __device__ __forceinline__ bool whole() const { return begins() && ends(); }
};

struct Line {
    long long T, lo, hi, us;    // places in all, of this range; the current unit's first place
    long long head;
    int N, range, TB, b, hk, j;
    Seq s;

    // the range with place x
    __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * N - 1) / T); }

    // A full warp, for one of sh.ctas ranges that `ctas` CTAs take; false: the sequences' ends are no sums of lengths, and nothing may be done.
    __device__ __forceinline__ bool begin(const ChunkAttnArgs& a, const Shape& sh, int ctas, int range_, int lane)
    {
        head = (long long)sh.head * sh.BN;
        TB = sh.BM / (a.heads / a.kv_heads);
        range = range_;
        long long sum = 0, mine = 0;            // places of a head: all sequences', of this lane's among the first 32
        float again = 0.f;                      // tokens that several blocks read
        bool good = true;
        for (int i = lane; i < a.batch; i += 32) {
            Seq x;
            x.read(a, i, TB);
            good = good && x.n >= 0 && x.tok0 >= 0 && (i > 0 || x.tok0 == 0) && (long long)x.tok0 + x.n <= a.tokens;   // (of each: n may have wrapped)
            const long long p = x.per_head(head);
            if (i == lane) mine = p;
            sum += p;
            again += x.blocks > 1 ? (float)x.last : 0.f;
        }
        lo = hi = us = 0;              // (nothing for a range of which this returns early: `next` ends at once)
        T = 0;
        if (!__all_sync(0xffffffffu, good)) return false;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            again += __shfl_xor_sync(0xffffffffu, again, o);
        }
        T = sum * a.kv_heads;
        // as many waves as their keys and values ask for, of kLeastTiles at least to a range
        const float bytes = again * a.kv_heads * a.dim * (a.bf16 ? 4.f : 8.f);
        int waves = 1;
        while ((waves + 1) * ctas <= sh.ctas && waves * kResident < bytes && (waves + 1ll) * ctas * kLeastTiles * sh.BN <= T) ++waves;
        // (at least a tile's places to a range, so that each one between a unit's first and last has a tile of it)
        N = (int)min((long long)ctas * waves, T >> tile_bits(sh));
        if (N < 1) N = 1;
        if (T == 0 || range >= N) return true;
        const long long q = quotient(T, N), over = T - q * N, c0 = quotient(over * range, N), c1 = quotient(over * (range + 1), N);
        lo = q * range + c0;
        hi = q * (range + 1) + c1;
        // the sequence that holds place lo, and where it begins
        long long b0 = 0;
        b = a.batch - 1;
        for (int i0 = 0; i0 < a.batch; i0 += 32) {
            long long m = mine;
            if (i0 > 0) {
                Seq x;
                m = 0;
                if (i0 + lane < a.batch) {
                    x.read(a, i0 + lane, TB);
                    m = x.per_head(head);
                }
            }
            m *= a.kv_heads;
            long long incl = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            const unsigned past = __ballot_sync(0xffffffffu, b0 + incl > lo);
            if (past) {
                const int src = __ffs(past) - 1;
                b = i0 + src;
                b0 += __shfl_sync(0xffffffffu, incl - m, src);
                break;
            }
            b0 += __shfl_sync(0xffffffffu, incl, 31);
        }
        s.read(a, b, TB);
        const long long per = s.per_head(head), in = lo - b0;
        hk = (int)quotient(in, per);
        const long long rest = in - hk * per;
        int l = 0, r = s.blocks - 1;    // the last block that begins at or before `rest`
        while (l < r) {
            const int mid = l + (r - l + 1) / 2;
            if (s.before(mid, head) <= rest) l = mid;
            else r = mid - 1;
        }
        j = l;
        us = b0 + hk * per + s.before(j, head);
        return true;
    }
    // any thread
    __device__ __forceinline__ bool next(const ChunkAttnArgs& a, const Shape& sh, Piece& p)
    {
        while (us < hi) {
            p.b = b;
            p.hk = hk;
            p.tok = j * TB;
            p.tokens = min(TB, s.n - p.tok);
            p.row0 = s.tok0 + p.tok;
            p.ctx = s.ctx;
            p.ok = s.ok;
            p.seen = s.ok ? s.ctx + p.tok + p.tokens : 0;
            p.common = s.ok ? s.ctx + p.tok + 1 : 0;
            p.range = range;
            p.tiles = s.ok ? ((p.seen - 1) >> tile_bits(sh)) + 1 : 1;
            p.at = us + head;
            const long long x = lo - p.at, y = hi - p.at;
            p.first = x <= 0 ? 0 : (int)min((long long)p.tiles, (x + sh.BN - 1) >> tile_bits(sh));
            p.last = y <= 0 ? 0 : (int)min((long long)p.tiles, (y + sh.BN - 1) >> tile_bits(sh));
            p.slot = 2 * range + (p.first == 0 ? 1 : 0);
            // on to the next unit
            const long long places = head + (j == s.blocks - 1 ? s.last : s.base + s.step * (j + 1));
            us += places;
            if (++j == s.blocks) {
                j = 0;
                if (++hk == a.kv_heads) {
                    hk = 0;
                    do {
                        if (++b < a.batch) s.read(a, b, TB);
                        else { us = hi; break; }
                    } while (s.blocks == 0);
                }
            }
            if (p.last > p.first) return true;
        }
        return false;
    }
};

// What the join reads, by one thread of each CTA: none of its ranges' records at first, then piece by piece.
__device__ __forceinline__ void clear_records(const ChunkAttnArgs& a, const Shape& sh, int ctas, int cta)
{
    for (int r = cta; r < sh.ctas; r += ctas) static_cast<Record*>(a.workspace)[r] = {0, 0, 0, 0};
}
__device__ __forceinline__ void record(const ChunkAttnArgs& a, const Shape& sh, const Line& line, const Piece& p)
{
    if (!p.begins() || p.ends()) return;
    const int G = a.heads / a.kv_heads;
    static_cast<Record*>(a.workspace)[p.range] = {line.owner(p.at + (long long)(p.tiles - 1) * sh.BN), p.row0 * G, p.hk, p.tokens * G};
}

// The line's places fit what its products count: false for tables of many terabytes.
__host__ __forceinline__ bool line_fits(const ChunkAttnArgs& a, const Shape& sh)
{
    const int TB = sh.BM / (a.heads / a.kv_heads);
    const double units = ((double)a.tokens / TB + a.batch) * a.kv_heads;
    const double most = (double)a.table_cols * a.page_size + (double)sh.head * sh.BN + 1;
    return units * (most < 2147483648.0 ? most : 2147483648.0) * sh.ctas < 4.0e18;
}

}  // namespace chunk
}  // namespace kda
