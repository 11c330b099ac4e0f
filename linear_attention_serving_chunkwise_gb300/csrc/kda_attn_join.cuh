// The parts that the attention kernels leave of units whose work several CTAs share, and their join.
#pragma once

#include "kda_common.cuh"

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
// Rows are numbered (token, head of the group) over the whole call: row r of cache head hk is query head hk G + r % G of
// out's token r / G.
struct Record {
    int last, row0, hk, rows;
};

struct JoinArgs {
    void *workspace, *out;
    int heads, kv_heads;
};

// Workspace: the CTAs' records, then for each of 2 * ctas slots BM maxima, BM sums, and the
// outputs as [D / 4][BM] float4 -- a thread holds a row, so that order makes its stores
// (and the join's loads) contiguous across a warp.
__host__ __device__ __forceinline__ size_t slot_floats(int BM, int D) { return (size_t)BM * (D + 2); }
__host__ __device__ __forceinline__ size_t workspace_bytes(const Shape& sh, int D)
{
    return sh.ctas * sizeof(Record) + slot_floats(sh.BM, D) * 2 * sh.ctas * sizeof(float);
}
__device__ __forceinline__ float* slot_of(void* workspace, const Shape& sh, int D, int slot)
{
    return reinterpret_cast<float*>(static_cast<Record*>(workspace) + sh.ctas) + slot_floats(sh.BM, D) * (size_t)slot;
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
__global__ void __launch_bounds__(kJoinThreads) join_kernel(JoinArgs a, Shape sh)
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
    const int G = a.heads / a.kv_heads, rows = rec.rows, r0 = 32 * blockIdx.y;
    if (rec.last == 0 || r0 >= rows) return;
    const int parts = rec.last - c + 1, r = min(r0 + lane, sh.BM - 1), first4 = C4 * blockIdx.z;
    const auto part = [&](int i) { return slot_of(a.workspace, sh, D, i == 0 ? 2 * c + 1 : 2 * (c + i)); };
    // no maximum at all: nothing to attend to, zeros; NaN stays, and a sum of 0 with a maximum (scores of -inf only) becomes it
    const auto over = [](float4 x, float sum, float m) {
        const float inv = 1.f / sum, none = m == -INFINITY ? 0.f : NAN;
        return sum == 0.f ? make_float4(none, none, none, none) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
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
                              fmaf(f1, pl[1], f0 * pl[0]), m);
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
                s_out[lane][k0 + w] = over(x, sum, m);
            }
            __syncthreads();
        }
    }
    // 8 lanes to a row's 32 channels
    const int i = t >> 3, k = t & 7;
    if (r0 + i < rows) {
        const int row = rec.row0 + r0 + i;
        Tout* dst = static_cast<Tout*>(a.out) + ((size_t)(row / G) * a.heads + rec.hk * G + row % G) * D + 4 * (first4 + k);
        const float4 x = s_out[i][k];
        if constexpr (sizeof(Tout) == 2) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
            *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
            *reinterpret_cast<float4*>(dst) = x;
        }
    }
}

// `most_rows`: of a unit.  The join's blocks may be launched while the last of the attention's still run (they wait for
// the whole grid before they read).
template <typename Tout, int D>
cudaError_t launch_join(const JoinArgs& a, const Shape& sh, int most_rows, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas - 1, ((most_rows < sh.BM ? most_rows : sh.BM) + 31) / 32, D / kJoinChannels);
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
