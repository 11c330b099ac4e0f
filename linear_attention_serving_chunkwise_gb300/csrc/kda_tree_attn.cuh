// How the tree-attention kernels share their work, and the join of what was split.
//
// A unit is one (sequence, key/value head, block of query rows); its tokens (the context and
// the draft nodes) are cut into tiles.  All units' tiles form one line (sequence-major, then
// head, then row block; before a unit's tiles a few places stand for its fixed cost), and CTA
// c of N takes the places [start(c), start(c + 1)) with start(c) = floor(T c / N): every CTA
// gets the same share (a place more or less) whatever the mix of lengths, a long sequence
// is split over many CTAs and a short one is not.  The context lengths live on the device, so each CTA works its cut out for itself.
//
// A unit that lies within one CTA's range is finished there.  Of any other, each CTA leaves
// its part (running maximum, sum and unnormalised output per row, fp32) in the workspace:
// slot 2 c when the unit began before the CTA's range, slot 2 c + 1 otherwise, so a CTA has
// at most two, and a record of both.  join_kernel joins a unit's parts in tile order.
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

// What a CTA left for the join.
struct Record {
    int begins;    // slot 2 c + 1 holds the first part of a unit: this one
    int b, hk, r0;
    int goes_on;   // slot 2 c holds a later part of a unit: 1 a middle one, 2 its last; 0 none
    int pad[3];
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

// tokens of sequence b, or 0 for a length that its table cannot hold (the sequence is skipped)
__device__ __forceinline__ int seq_tokens(const TreeAttnArgs& a, int b, bool& ok)
{
    const int c = __ldg(a.context_lens + b);
    ok = c >= 0 && (long long)c + a.nodes <= (long long)a.table_cols * a.page_size;
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
    __device__ __forceinline__ bool whole() const { return begins && ends; }
};

// Walks a CTA's range piece by piece.
struct Line {
    int hi, lo, at, b0;
    int b, per_seq, rb;

    // a full warp
    __device__ __forceinline__ void begin(const TreeAttnArgs& a, const Shape& sh, int cta, int lane)
    {
        rb = row_blocks(a, sh.BM);
        per_seq = rb * a.kv_heads;
        const int mine = lane < a.batch ? unit_places(a, lane, sh) : 0;    // of the first 32 sequences
        int sum = mine;
        for (int i = lane + 32; i < a.batch; i += 32) sum += unit_places(a, i, sh);
        const int T = __reduce_add_sync(0xffffffffu, sum) * per_seq;
        lo = at = line_start(T, cta, sh.ctas);
        hi = line_start(T, cta + 1, sh.ctas);
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
    __device__ __forceinline__ void see(const Piece& p)
    {
        if (!p.begins) r.goes_on = p.ends ? 2 : 1;
        else if (!p.ends) { r.begins = 1; r.b = p.b; r.hk = p.hk; r.r0 = p.r0; }
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

// Joins the units that cross a boundary of the line: CTA (c, y) takes rows [32 y, 32 y + 32) of
// the unit whose first part CTA c left, if there is one.  Lane = row; the warps share the
// channels.  m = max m_i, o = sum e^{m_i - m} o_i / sum e^{m_i - m} l_i, in tile order.
constexpr int kJoinThreads = 256;

template <typename Tout, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(TreeAttnArgs a, Shape sh)
{
    constexpr int W = kJoinThreads / 32, C = D / 4 / W;      // chunks of 4 channels per warp
    extern __shared__ short s_parts[];                       // slots of the unit's parts, in order
    __shared__ float4 s_out[32][D / 4 + 1];
    __shared__ int s_n;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, c = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the parts are written
    const Record* recs = static_cast<const Record*>(a.workspace);
    const Record rec = recs[c];
    if (!rec.begins) return;
    const int G = a.heads / a.kv_heads, rows = min(sh.BM, a.nodes * G - rec.r0), r0 = 32 * blockIdx.y;
    if (r0 >= rows) return;
    if (w == 0) {
        int n = 0;
        if (lane == 0) s_parts[0] = (short)(2 * c + 1);
        for (int x0 = c + 1, more = 1; more && x0 < sh.ctas; x0 += 32) {
            const int x = x0 + lane, g = x < sh.ctas ? recs[x].goes_on : 0;
            const unsigned last = __ballot_sync(0xffffffffu, g == 2);
            const unsigned upto = last ? 0xffffffffu >> (32 - __ffs(last)) : 0xffffffffu;
            const unsigned on = __ballot_sync(0xffffffffu, g != 0) & upto;
            if (on >> lane & 1) s_parts[1 + n + __popc(on & ((1u << lane) - 1))] = (short)(2 * x);
            n += __popc(on);
            more = last == 0;
        }
        if (lane == 0) s_n = 1 + n;
    }
    __syncthreads();
    const int parts = s_n, r = min(r0 + lane, sh.BM - 1);
    float m = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) m = fmaxf(m, slot_of(a, sh, D, s_parts[i])[r]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o[C] = {};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        float* p = slot_of(a, sh, D, s_parts[i]);
        const float f = exp2f(p[r] - base);
        l = fmaf(f, p[sh.BM + r], l);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const float4 x = slot_out(p, sh.BM)[(size_t)(w + W * k) * sh.BM + r];
            o[k].x = fmaf(f, x.x, o[k].x);
            o[k].y = fmaf(f, x.y, o[k].y);
            o[k].z = fmaf(f, x.z, o[k].z);
            o[k].w = fmaf(f, x.w, o[k].w);
        }
    }
    const float inv = 1.f / l;                               // nothing to attend to: zeros; NaN stays
#pragma unroll
    for (int k = 0; k < C; ++k)
        s_out[lane][w + W * k] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv);
    __syncthreads();
    for (int i = w; i < 32 && r0 + i < rows; i += W) {
        const int row = rec.r0 + r0 + i;
        Tout* dst = static_cast<Tout*>(a.out) + (((size_t)rec.b * a.nodes + row / G) * a.heads + rec.hk * G + row % G) * D;
        for (int k = lane; k < D / 4; k += 32) {
            const float4 x = s_out[i][k];
            if constexpr (sizeof(Tout) == 2) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
                *reinterpret_cast<uint2*>(dst + 4 * k) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            } else {
                *reinterpret_cast<float4*>(dst + 4 * k) = x;
            }
        }
    }
}

// The join's blocks may be launched while the last of the attention's still run (they wait for
// the whole grid before they read).
template <typename Tout, int D>
cudaError_t launch_join(const TreeAttnArgs& a, const Shape& sh, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas - 1, (sh.BM + 31) / 32);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = (sh.ctas + 1) * sizeof(short);
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
