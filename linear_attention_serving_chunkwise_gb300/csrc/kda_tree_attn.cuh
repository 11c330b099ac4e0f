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

#include "kda_draft_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace attn {

struct Shape {
    int BM;        // query rows of a unit
    int BN;        // tokens of a tile
    int ctas;      // CTAs that share the line
    int head;      // places of the line before a unit's tiles: what a unit costs beyond them, in tiles
};

// What CTA c left for the join: the unit whose first part is in slot 2 c + 1 and the CTA with
// its last part (the CTAs between have one each, in their slots 2 x); last = 0: none.
struct Record {
    int last, b, hk, r0;
};

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
    Record r = {};
    __device__ __forceinline__ void see(const Line& line, const Piece& p)
    {
        if (!p.begins || p.ends) return;
        // the CTA that holds the unit's last place
        const int end = line.hi + p.rest - 1;
        r.last = (int)((((long long)end + 1) * line.N - 1) / line.T);
        r.b = p.b;
        r.hk = p.hk;
        r.r0 = p.r0;
    }
    __device__ __forceinline__ void leave(const TreeAttnArgs& a, int cta) { static_cast<Record*>(a.workspace)[cta] = r; }
};

// Workspace: the CTAs' records, then for each of 2 * ctas slots BM maxima, BM sums, and the
// outputs as [D / 4][BM] float4 -- a thread holds a row, so that order makes its stores
// (and the join's loads) contiguous across a warp.
__host__ __device__ __forceinline__ size_t slot_floats(int BM, int D) { return (size_t)BM * (D + 2); }
__host__ __device__ __forceinline__ size_t workspace_bytes(const Shape& sh, int D)
{
    return sh.ctas * sizeof(Record) + slot_floats(sh.BM, D) * 2 * sh.ctas * sizeof(float);
}
__device__ __forceinline__ float* slot_of(const TreeAttnArgs& a, const Shape& sh, int D, int slot)
{
    return reinterpret_cast<float*>(static_cast<Record*>(a.workspace) + sh.ctas) + slot_floats(sh.BM, D) * (size_t)slot;
}
__device__ __forceinline__ float4* slot_out(float* slot, int BM) { return reinterpret_cast<float4*>(slot + 2 * BM); }

// Joins the units that cross a boundary of the line: block (c, y, z) takes rows [32 y, 32 y + 32)
// and channels [32 z, 32 z + 32) of the unit whose first part CTA c left, if there is one.
// Lane = row.  m = max m_i, o = sum e^{m_i - m} o_i / sum e^{m_i - m} l_i, in an order set by the
// parts alone.
// Bound: latency, of a chain of dependent reads (the record, then the parts).  A unit in two parts
// (most, when there are more units than CTAs) has all its reads under way at once, a warp to four
// channels: 32 trees of 16 nodes took 253 us in all with the general form below, 247 with
// this one.  More parts are shared by the warps first and the channels second, as many to the parts as
// give each two, so that a unit in a hundred parts is as quick to join as one in two (this form
// for up to four parts: 30.4 -> 33.9 us for a small fp32 call).  Blocks of 64 channels, half as many,
// lost 5 us of 208 where the units are few and their parts many (2 x 131072 tokens).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinChannels = 32;

template <typename Tout, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(TreeAttnArgs a, Shape sh)
{
    constexpr int K = 2;                                     // chunks of 4 channels a warp takes at a time
    constexpr int C4 = kJoinChannels / 4;                    // chunks of a block
    static_assert(C4 == kJoinWarps, "a warp to a chunk");
    __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
    __shared__ float4 s_o[kJoinWarps][K][32];
    __shared__ float4 s_out[32][C4 + 1];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, c = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the parts are written
    const int4 raw = *(reinterpret_cast<const int4*>(a.workspace) + c);
    const Record rec = {raw.x, raw.y, raw.z, raw.w};
    const int G = a.heads / a.kv_heads, rows = min(sh.BM, a.nodes * G - rec.r0), r0 = 32 * blockIdx.y;
    if (rec.last == 0 || r0 >= rows) return;
    const int parts = rec.last - c + 1, r = min(r0 + lane, sh.BM - 1), first4 = C4 * blockIdx.z;
    const auto part = [&](int i) { return slot_of(a, sh, D, i == 0 ? 2 * c + 1 : 2 * (c + i)); };
    // nothing to attend to: zeros; NaN stays
    const auto over = [](float4 x, float sum) {
        const float inv = 1.f / sum;
        return sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    };
    if (parts == 2) {
        float pm[2], pl[2];
        float4 po[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float* p = part(i);
            pm[i] = p[r];
            pl[i] = p[sh.BM + r];
            po[i] = slot_out(p, sh.BM)[(size_t)(first4 + w) * sh.BM + r];
        }
        const float m = fmaxf(pm[0], pm[1]), base = m == -INFINITY ? 0.f : m;
        const float f0 = exp2f(pm[0] - base), f1 = exp2f(pm[1] - base);
        s_out[lane][w] = over(make_float4(fmaf(f1, po[1].x, f0 * po[0].x), fmaf(f1, po[1].y, f0 * po[0].y),
                                          fmaf(f1, po[1].z, f0 * po[0].z), fmaf(f1, po[1].w, f0 * po[0].w)),
                              fmaf(f1, pl[1], f0 * pl[0]));
        __syncthreads();
    } else {
        float m = -INFINITY;
#pragma unroll 4
        for (int i = w; i < parts; i += kJoinWarps) m = fmaxf(m, part(i)[r]);
        s_m[w][lane] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) m = fmaxf(m, s_m[k][lane]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        for (int i = w; i < parts; i += kJoinWarps) l = fmaf(exp2f(part(i)[r] - base), part(i)[sh.BM + r], l);
        s_l[w][lane] = l;
        const int pw = parts <= 4 ? 2 : parts <= 8 ? 4 : 8, cw = kJoinWarps / pw, pl = w % pw, cl = w / pw;
        for (int k0 = 0; k0 < C4; k0 += cw * K) {
            float4 o[K] = {};
#pragma unroll 4
            for (int i = pl; i < parts; i += pw) {
                float* p = part(i);
                const float f = exp2f(p[r] - base);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float4 x = slot_out(p, sh.BM)[(size_t)(first4 + k0 + cl * K + k) * sh.BM + r];
                    o[k].x = fmaf(f, x.x, o[k].x);
                    o[k].y = fmaf(f, x.y, o[k].y);
                    o[k].z = fmaf(f, x.z, o[k].z);
                    o[k].w = fmaf(f, x.w, o[k].w);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) s_o[w][k][lane] = o[k];
            __syncthreads();
            if (w < cw * K) {                                // a warp to a chunk
                const int k = w % K, first = (w / K) * pw;
                float4 x = s_o[first][k][lane];
                for (int i = 1; i < pw; ++i) {
                    const float4 y = s_o[first + i][k][lane];
                    x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                }
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kJoinWarps; ++i) sum += s_l[i][lane];
                s_out[lane][k0 + w] = over(x, sum);
            }
            __syncthreads();
        }
    }
    // 8 lanes to a row's 32 channels
    const int i = t >> 3, k = t & 7;
    if (r0 + i < rows) {
        const int row = rec.r0 + r0 + i;
        Tout* dst = static_cast<Tout*>(a.out) + (((size_t)rec.b * a.nodes + row / G) * a.heads + rec.hk * G + row % G) * D + 4 * (first4 + k);
        const float4 x = s_out[i][k];
        if constexpr (sizeof(Tout) == 2) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
            *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
            *reinterpret_cast<float4*>(dst) = x;
        }
    }
}

// The join's blocks may be launched while the last of the attention's still run (they wait for
// the whole grid before they read).
template <typename Tout, int D>
cudaError_t launch_join(const TreeAttnArgs& a, const Shape& sh, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    const int rows = a.nodes * (a.heads / a.kv_heads);
    cfg.gridDim = dim3(sh.ctas - 1, ((rows < sh.BM ? rows : sh.BM) + 31) / 32, D / kJoinChannels);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<Tout, D>, a, sh);
}

}  // namespace attn
}  // namespace kda
