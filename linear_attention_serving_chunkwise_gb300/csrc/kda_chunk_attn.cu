// Softmax attention of chunks of new tokens over a paged fp32 key/value cache, on the CUDA cores
// (fp32 throughout).
//
// A thread has 8 query rows and BN / 16 tokens of a tile's scores, then 8 rows and D / 16 channels of
// the output: 12 shared-memory reads to 128 multiply-adds (scores at D = 128: 10 to 64).  One pass over the tiles with the running maximum
// and sum of the softmax.  A tile's values are zeroed where no row of the unit may see the token (past its last one, a page
// out of range); in the tiles that only some rows see whole, a token that the row does not see has the weight -1, which is skipped: 0
// times whatever lies there must not be NaN.  (A weight of 0 is not: what a row sees shows, infinities and NaN too.)
// Bound: the CUDA cores, half of their multiply-adds; without the scores' loop the kernel takes 0.62 of its time, without the values'
// 0.67, without either 0.32 (64 channels).  5 sequences of 1 to 701 tokens after up to 3001, 6 heads on 2, D = 64 200 us, 33 TFLOP/s; 2048 tokens after
// 2048, 32 heads on 8 1.28 ms (D = 64, 40 TFLOP/s), 2.71 ms (D = 128).  Two multiply-adds at a time took 198 us, 1.23 and 2.48 ms beside 197 us, 1.25
// and 2.68: 7 % at D = 128 and little at 64, not built in so far.  A second buffer for the tiles (226 instead of 201 us), other rows to a
// thread (216) and operands fetched a step ahead (204) lost.
#include <float.h>

#include "kda_chunk_attn.cuh"
#include "kda_draft_sm100.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128, kBM = 64, kTM = 8;
constexpr float kTame = 4096.f;        // largest maximum (in powers of two) of the quick form
// Most that a thread's weights of a tile's row may sum to before the maximum is set anew.  16 threads and 2^26 tiles of 32 tokens make a
// row's sum 2^45 at most, so sums with values up to 2^82 stay finite.  With 32 instead of 2^15 sharper scores cost 1 to 2 %.
constexpr float kMostSum = 32768.f;
// The maximum of a row that sees tokens whose scores are all -inf: its weights are 0 over 0, as by the definition, where a row that sees
// no token (maximum -inf) becomes zero.
constexpr float kLowest = -FLT_MAX;

template <int D>
struct Tile {
    static constexpr int BN = D == 128 ? 32 : 64, CD = D / 16, TN = BN / 16, LD = D + 4, LP = BN + 4;
    static constexpr size_t kSmem = (size_t)(kBM * LD + 2 * BN * LD + kBM * LP) * 4;
};

// o += p v over a tile: eight rows of weights from sp on, four channels of every 16 from sv on.  kSome: a weight below 0 is
// skipped (a test for each, so not where all rows see the whole tile).
template <int D, bool kSome>
__device__ __forceinline__ void add_values(float (&o)[kTM][Tile<D>::CD], const float* sp, const float* sv)
{
    using L = Tile<D>;
#pragma unroll 2
    for (int j = 0; j < L::BN; j += 4) {
        float4 p4[kTM];
#pragma unroll
        for (int i = 0; i < kTM; ++i) p4[i] = *reinterpret_cast<const float4*>(sp + i * L::LP + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v[L::CD];
#pragma unroll
            for (int k = 0; k < L::CD; k += 4) {
                const float4 v4 = *reinterpret_cast<const float4*>(sv + (j + e) * L::LD + 16 * k);
                v[k] = v4.x; v[k + 1] = v4.y; v[k + 2] = v4.z; v[k + 3] = v4.w;
            }
#pragma unroll
            for (int i = 0; i < kTM; ++i) {
                const float p = e == 0 ? p4[i].x : e == 1 ? p4[i].y : e == 2 ? p4[i].z : p4[i].w;
                if (kSome && p < 0.f) continue;
#pragma unroll
                for (int k = 0; k < L::CD; ++k) o[i][k] = fmaf(p, v[k], o[i][k]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3) chunk_attn_simt_kernel(ChunkAttnArgs a, attn::Shape sh)
{
    using L = Tile<D>;
    constexpr int BN = L::BN, CD = L::CD, TN = L::TN, LD = L::LD, LP = L::LP;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                   // [kBM][LD]
    float* sk = sq + kBM * LD;        // [BN][LD]
    float* sv = sk + BN * LD;         // [BN][LD]
    float* sp = sv + BN * LD;         // [kBM][LP]
    __shared__ unsigned char s_on[BN];     // the tile's tokens that exist

    const int t = threadIdx.x, lane = t & 31, ty = t >> 4, tx = t & 15;
    const int G = a.heads / a.kv_heads;
    const float sc = a.scale * 1.4426950408889634f;     // scores in powers of two

    chunk::Line line;
    const bool good = line.begin(a, sh, sh.ctas, blockIdx.x, lane);
    if (!good && blockIdx.x == 0 && t == 0) report_status(a.status, kDevBadSeqlens);
    chunk::Piece pc;
    if (t == 0) chunk::clear_records(a, sh, sh.ctas, blockIdx.x);
    bool bad = false;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    while (line.next(a, sh, pc)) {
        if (t == 0) chunk::record(a, sh, line, pc);
        const int rows = pc.tokens * G;
        bad |= !pc.ok;
        __syncthreads();              // the last unit's reads of shared memory are done
        for (int i = t; i < kBM * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) x = load4(static_cast<const float*>(a.q) + ((size_t)(pc.row0 + r / G) * a.heads + pc.hk * G + r % G) * D + c);
            *reinterpret_cast<float4*>(sq + r * LD + c) = x;
        }
        float m[kTM], l[kTM], o[kTM][CD];
        int seen[kTM];                // tokens that the row sees
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            const int r = ty * kTM + i;
            seen[i] = pc.ok && r < rows ? pc.ctx + pc.tok + r / G + 1 : 0;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int k = 0; k < CD; ++k) o[i][k] = 0.f;
        }
        for (int tile = pc.first; pc.ok && tile < pc.last; ++tile) {
            const int t0 = tile * BN;
            __syncthreads();
            // a thread has four channels of every kStep-th token; the page ids are read together, then four rows at a time
            constexpr int kStep = kThreads / (D / 4), kRows = BN / kStep;
            const int j0 = t / (D / 4), c = 4 * (t % (D / 4));
            int id[kRows];
            size_t at[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int pos = t0 + j0 + i * kStep, pg = pos / a.page_size;
                at[i] = ((size_t)(pos - pg * a.page_size) * a.kv_heads + pc.hk) * D + c;
                id[i] = pos < pc.seen ? __ldg(a.block_table + (size_t)pc.b * a.table_cols + pg) : -1;
            }
            bool there = true;        // all of this thread's tokens
#pragma unroll
            for (int i0 = 0; i0 < kRows; i0 += 4) {
                float4 k4[4], v4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = id[i0 + i];
                    k4[i] = v4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p >= 0 && p < a.num_pages) {
                        k4[i] = load4(static_cast<const float*>(a.k_cache) + (size_t)p * a.k_page_stride + at[i0 + i]);
                        v4[i] = load4(static_cast<const float*>(a.v_cache) + (size_t)p * a.v_page_stride + at[i0 + i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + (i0 + i) * kStep, p = id[i0 + i];
                    const bool on = p >= 0 && p < a.num_pages;
                    bad |= !on && t0 + j < pc.seen;
                    if (c == 0) s_on[j] = on;
                    there &= on;
                    *reinterpret_cast<float4*>(sk + j * LD + c) = k4[i];
                    *reinterpret_cast<float4*>(sv + j * LD + c) = v4[i];
                }
            }
            // (every row sees the whole tile)
            const bool all = __syncthreads_and(there) && t0 + BN <= pc.ctx + pc.tok + 1;
            float s[kTM][TN] = {};
#pragma unroll 2
            for (int ch = 0; ch < D; ch += 4) {
                float4 k4[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) k4[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + ch);
#pragma unroll
                for (int i = 0; i < kTM; ++i) {
                    const float4 q4 = *reinterpret_cast<const float4*>(sq + (ty * kTM + i) * LD + ch);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        s[i][j] = fmaf(q4.x, k4[j].x, fmaf(q4.y, k4[j].y, fmaf(q4.z, k4[j].z, fmaf(q4.w, k4[j].w, s[i][j]))));
                }
            }
            // The weights are formed from the last maximum, and stand unless one is past what may, which their sums tell: then, and in
            // tiles that some rows see in part, the row's maximum first.  (s sc - m in one operation: m's own rounding is a factor
            // that a row's weights share.)
            float p[kTM][TN], part[kTM];
            bool again = !all;
            if (!again) {
                bool wild = false;
#pragma unroll
                for (int i = 0; i < kTM; ++i) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        p[i][j] = ex2(fmaf(s[i][j], sc, -m[i]));
                        sum += p[i][j];
                    }
                    wild |= seen[i] && (sum > kMostSum || !(fabsf(m[i]) <= kTame));    // (what a row that is none gets goes nowhere)
                    part[i] = sum;
                }
                again = __any_sync(0xffffffffu, wild);
                if (!again) {
#pragma unroll
                    for (int i = 0; i < kTM; ++i) l[i] += part[i];
                }
            }
            if (again) {
#pragma unroll
                for (int i = 0; i < kTM; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const bool sees = s_on[tx + 16 * j] && t0 + tx + 16 * j < seen[i];
                        s[i][j] = sees ? s[i][j] * sc : -INFINITY;
                        top = fmaxf(top, fmaxf(s[i][j], sees ? kLowest : -INFINITY));
                    }
#pragma unroll
                    for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float nm = fmaxf(m[i], top), base = nm == -INFINITY ? 0.f : nm;
                    const float f = exp2f(m[i] - base);
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        p[i][j] = exp2f(s[i][j] - base);
                        sum += p[i][j];
                        // (on a page that is not there the value is 0, whatever the weight)
                        if (t0 + tx + 16 * j >= seen[i]) p[i][j] = -1.f;
                    }
                    l[i] = l[i] * f + sum;           // (of this thread's tokens: the row's are summed at the end)
                    m[i] = nm;
#pragma unroll
                    for (int k = 0; k < CD; ++k) o[i][k] *= f;
                }
            }
#pragma unroll
            for (int i = 0; i < kTM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) sp[(ty * kTM + i) * LP + tx + 16 * j] = p[i][j];
            __syncwarp();             // a row's weights are written and read by the same half warp
            if (t0 + BN > pc.ctx + pc.tok + 1) {
                add_values<D, true>(o, sp + ty * kTM * LP, sv + tx * 4);
            } else {
                add_values<D, false>(o, sp + ty * kTM * LP, sv + tx * 4);
            }
        }
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        // the unit is done here, or its part goes to the workspace
        float* ws = attn::slot_of(a.workspace, sh, D, pc.slot);
#pragma unroll
        for (int i = 0; i < kTM; ++i) {
            const int r = ty * kTM + i;
            if (r >= rows) continue;
            if (pc.whole()) {
                float* dst = static_cast<float*>(a.out) + ((size_t)(pc.row0 + r / G) * a.heads + pc.hk * G + r % G) * D;
                const float inv = 1.f / l[i], none = m[i] == -INFINITY ? 0.f : NAN;
#pragma unroll
                for (int k = 0; k < CD; k += 4) {
                    const float4 y = make_float4(o[i][k] * inv, o[i][k + 1] * inv, o[i][k + 2] * inv, o[i][k + 3] * inv);
                    *reinterpret_cast<float4*>(dst + tx * 4 + 16 * k) = l[i] == 0.f ? make_float4(none, none, none, none) : y;
                }
            } else {
                if (tx == 0) { ws[r] = m[i]; ws[kBM + r] = l[i]; }
#pragma unroll
                for (int k = 0; k < CD; k += 4)
                    attn::slot_out(ws, kBM)[(size_t)(tx + 4 * k) * kBM + r] = make_float4(o[i][k], o[i][k + 1], o[i][k + 2], o[i][k + 3]);
            }
        }
    }
    if (bad) report_status(a.status, kDevBadSeqlens);
}

template <int D>
constexpr attn::Shape simt_shape() { return {kBM, Tile<D>::BN, 152 * (D == 128 ? 2 : 3), 1}; }

template <int D>
cudaError_t launch_simt(const ChunkAttnArgs& a, cudaStream_t stream)
{
    const attn::Shape sh = simt_shape<D>();
    static KernelSetup setup;
    cudaError_t e = setup(chunk_attn_simt_kernel<D>, Tile<D>::kSmem);
    if (e != cudaSuccess) return e;
    chunk_attn_simt_kernel<D><<<sh.ctas, kThreads, Tile<D>::kSmem, stream>>>(a, sh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return attn::launch_join<float, D>({a.workspace, a.out, a.heads, a.kv_heads}, sh, kBM, stream);
}

attn::Shape shape_of(const ChunkAttnArgs& a) { return a.dim == 128 ? simt_shape<128>() : simt_shape<64>(); }

}  // namespace

bool chunk_attn_fits(const ChunkAttnArgs& a) { return a.bf16 ? chunk_attn_tc_fits(a) : chunk::line_fits(a, shape_of(a)); }

size_t chunk_attn_workspace_bytes(const ChunkAttnArgs& a)
{
    return a.bf16 ? chunk_attn_tc_workspace_bytes(a) : attn::workspace_bytes(shape_of(a), a.dim);
}

cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t stream)
{
    if (a.bf16) return launch_chunk_attn_tc(a, stream);
    return a.dim == 128 ? launch_simt<128>(a, stream) : launch_simt<64>(a, stream);
}

}  // namespace kda
