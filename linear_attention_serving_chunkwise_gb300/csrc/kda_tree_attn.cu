// Softmax attention of a draft tree's tokens over a paged fp32 key/value cache, on the
// CUDA cores (fp32 throughout; bf16 runs in kda_tree_attn_tc.cu): node i of sequence b attends to
// the sequence's context_lens[b] cached tokens and to the nodes on its own path, whose keys and
// values lie in the cache at the logical positions context + j.  One pass over the tokens with the
// running maximum and sum of the softmax; query heads of one group share each loaded tile.
// Bound: for few rows latency (a tile's loads, scores, softmax and values follow one another; where two
// CTAs fit an SM they cover some of it), for many the CUDA cores' fp32 rate.  7 sequences of up to 3001
// tokens, 5 nodes, 6 heads on 2 cache heads, D = 64: 28 us, 0.40 TB/s, join included; 16 with
// 32 nodes: 75 us, 15 TFLOP/s.
//
// A tile's values are zeroed where no row may see the token (past the last node, a page out
// of range): a masked weight is 0, and 0 times whatever lies there must not be NaN.  In the
// tiles that hold draft nodes, where each row sees other nodes, a weight of 0 is skipped.
#include "kda_tree_attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kBN = 64;

// TM rows and 4 tokens (then D / 16 channels) per thread of a 16 x 16 grid
template <int D, int TM>
__global__ void __launch_bounds__(kThreads) tree_attn_simt_kernel(TreeAttnArgs a, attn::Shape sh)
{
    constexpr int BM = 16 * TM, CD = D / 16, LD = D + 4, LP = kBN + 4;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                   // [BM][LD]
    float* sk = sq + BM * LD;         // [BN][LD]
    float* sv = sk + kBN * LD;        // [BN][LD]
    float* sp = sv + kBN * LD;        // [BM][LP]
    __shared__ TreeSmem ts;
    __shared__ unsigned char s_on[kBN];   // the tile's tokens that exist

    const int t = threadIdx.x, lane = t & 31, ty = t >> 4, tx = t & 15;
    const int G = a.heads / a.kv_heads, R = a.nodes * G;
    const float sc = a.scale * 1.4426950408889634f;     // scores in powers of two

    attn::Line line;
    line.begin(a, sh, blockIdx.x, lane);
    attn::Piece pc;
    attn::Recorder rec(a, sh);
    int masks_of = -1;
    bool bad_page = false;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    while (line.next(a, sh, blockIdx.x, pc)) {
        const int b = pc.b, hk = pc.hk, r0 = pc.r0, n = pc.n, ctx = pc.ctx;
        rec.see(line, pc);

        __syncthreads();              // the last unit's reads of shared memory are done
        if (masks_of != b) {
            if (t < 32) tree_masks(ts, a.parents + (size_t)b * a.nodes, a.nodes, lane);
            masks_of = b;
        }
        for (int idx = t; idx < BM * D; idx += kThreads) {
            const int r = idx / D, c = idx - r * D, row = r0 + r;
            sq[r * LD + c] = row < R ? (static_cast<const float*>(a.q)[(((size_t)b * a.nodes + row / G) * a.heads + hk * G + row % G) * D + c]) : 0.f;
        }
        __syncthreads();
        const bool live = pc.seq_ok && ts.ok;
        if (!live && t == 0) report_status(a.status, kDevBadSeqlens);

        float m[TM], l[TM], o[TM][CD];
        uint64_t see[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int row = r0 + ty * TM + i;
            see[i] = live && row < R ? ts.anc[row / G] : 0ull;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int k = 0; k < CD; ++k) o[i][k] = 0.f;
        }
        for (int tile = pc.first; live && tile < pc.last; ++tile) {
            const int t0 = tile * kBN;
            if (tile != pc.first) __syncthreads();
            // a thread has four channels of every (kThreads / (D / 4))-th token; its page ids are read
            // together, then four rows of K and V at a time: two trips to memory instead of two a token
            // (7 sequences of up to 12000 tokens, D = 128: 114 -> 97 us)
            constexpr int kRows = kBN * (D / 4) / kThreads, kStep = kThreads / (D / 4);
            const int j0 = t / (D / 4), c = 4 * (t % (D / 4));
            size_t at[kRows];
            int id[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int pos = t0 + j0 + i * kStep, pg = pos / a.page_size;
                at[i] = ((size_t)(pos - pg * a.page_size) * a.kv_heads + hk) * D + c;
                id[i] = pos < n ? __ldg(a.block_table + (size_t)b * a.table_cols + pg) : -1;
            }
#pragma unroll
            for (int i0 = 0; i0 < kRows; i0 += 4) {
                float4 k4[4], v4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = id[i0 + i];
                    const bool on = p >= 0 && p < a.num_pages;
                    k4[i] = v4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (on) {
                        k4[i] = load4(static_cast<const float*>(a.k_cache) + (size_t)p * a.k_page_stride + at[i0 + i]);
                        v4[i] = load4(static_cast<const float*>(a.v_cache) + (size_t)p * a.v_page_stride + at[i0 + i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + (i0 + i) * kStep, p = id[i0 + i];
                    const bool on = p >= 0 && p < a.num_pages;
                    bad_page |= !on && t0 + j < n;
                    if (c == 0) s_on[j] = on;
                    *reinterpret_cast<float4*>(sk + j * LD + c) = k4[i];
                    *reinterpret_cast<float4*>(sv + j * LD + c) = v4[i];
                }
            }
            __syncthreads();
            float s[TM][4] = {};
            for (int c = 0; c < D; c += 4) {
                float4 k4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + c);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const float4 q4 = *reinterpret_cast<const float4*>(sq + (ty * TM + i) * LD + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(q4.x, k4[j].x, fmaf(q4.y, k4[j].y, fmaf(q4.z, k4[j].z, fmaf(q4.w, k4[j].w, s[i][j]))));
                }
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int pos = t0 + tx + 16 * j, node = pos - ctx;
                    const bool on = s_on[tx + 16 * j] && see[i] != 0 && (node < 0 || (see[i] >> node & 1));
                    s[i][j] = on ? s[i][j] * sc : -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float nm = fmaxf(m[i], top), base = nm == -INFINITY ? 0.f : nm;
                const float f = exp2f(m[i] - base);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(s[i][j] - base);
                    sum += p;
                    sp[(ty * TM + i) * LP + tx + 16 * j] = p;
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[i] = l[i] * f + sum;
                m[i] = nm;
#pragma unroll
                for (int k = 0; k < CD; ++k) o[i][k] *= f;
            }
            __syncwarp();             // a row's weights are written and read by the same half warp
            const bool nodes_here = t0 + kBN > ctx;
            for (int j = 0; j < kBN; ++j) {
                float v[CD];
#pragma unroll
                for (int k = 0; k < CD; k += 4) {
                    const float4 v4 = *reinterpret_cast<const float4*>(sv + j * LD + tx * 4 + 16 * k);
                    v[k] = v4.x; v[k + 1] = v4.y; v[k + 2] = v4.z; v[k + 3] = v4.w;
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const float p = sp[(ty * TM + i) * LP + j];
                    if (nodes_here && p == 0.f) continue;
#pragma unroll
                    for (int k = 0; k < CD; ++k) o[i][k] = fmaf(p, v[k], o[i][k]);
                }
            }
        }
        // the unit is done here, or its part goes to the workspace
        float* ws = attn::slot_of(a.workspace, sh, D, pc.slot);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = ty * TM + i, row = r0 + r;
            if (row >= R) continue;
            if (pc.whole()) {
                float* dst = static_cast<float*>(a.out) + (((size_t)b * a.nodes + row / G) * a.heads + hk * G + row % G) * D;
                const float inv = 1.f / l[i];
#pragma unroll
                for (int k = 0; k < CD; ++k) dst[tx * 4 + 16 * (k & ~3) + (k & 3)] = l[i] == 0.f ? 0.f : o[i][k] * inv;
            } else {
                if (tx == 0) { ws[r] = m[i]; ws[BM + r] = l[i]; }
#pragma unroll
                for (int k = 0; k < CD; k += 4)
                    attn::slot_out(ws, BM)[(size_t)(tx + 4 * k) * BM + r] = make_float4(o[i][k], o[i][k + 1], o[i][k + 2], o[i][k + 3]);
            }
        }
    }
    if (t == 0) rec.leave(a, blockIdx.x);
    if (bad_page) report_status(a.status, kDevBadSeqlens);
}

template <int D, int TM>
constexpr size_t simt_smem() { return (size_t)(16 * TM * (D + 4) + 2 * kBN * (D + 4) + 16 * TM * (kBN + 4)) * 4; }

// As many CTAs as run at once: two to an SM, one where two do not fit its 228 KB (D = 128, 64 rows: 117 KB
// each; with 304 shares there, in two waves, 7 sequences of up to 3001 tokens, 16 nodes, 6 heads on 2
// took 58 us instead of 43, 2 x 20000 tokens, 64 nodes, 8 heads on 2 433 instead of 414).
template <int D, int TM>
constexpr attn::Shape simt_shape() { return {16 * TM, kBN, 152 * (simt_smem<D, TM>() > 112 * 1024 ? 1 : 2), 1}; }

template <int D, int TM>
cudaError_t launch_simt(const TreeAttnArgs& a, cudaStream_t stream)
{
    const attn::Shape sh = simt_shape<D, TM>();
    constexpr size_t smem = simt_smem<D, TM>();
    static KernelSetup setup;
    cudaError_t e = setup(tree_attn_simt_kernel<D, TM>, smem);
    if (e != cudaSuccess) return e;
    tree_attn_simt_kernel<D, TM><<<sh.ctas, kThreads, smem, stream>>>(a, sh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return attn::launch_join<float, D>({a.workspace, a.out, a.heads, a.kv_heads}, sh, a.nodes * (a.heads / a.kv_heads), stream);
}

// rows of a unit: 16 while the whole (sequence, head) fits them (the other rows of a larger
// block would be computed for nothing: 15 rows take 30 us, in a block of 64 40 us), 64 otherwise
// (each loaded tile serves four times the rows: 96 rows take 79 us, in blocks of 16 107 us; all
// four before the page ids were read together)
bool small_rows(int nodes, int group) { return nodes * group <= 16; }

attn::Shape simt_shape_of(int nodes, int group, int dim)
{
    if (dim == 128) return small_rows(nodes, group) ? simt_shape<128, 1>() : simt_shape<128, 4>();
    return small_rows(nodes, group) ? simt_shape<64, 1>() : simt_shape<64, 4>();
}

cudaError_t launch_simt_dim(const TreeAttnArgs& a, cudaStream_t stream)
{
    const bool small = small_rows(a.nodes, a.heads / a.kv_heads);
    if (a.dim == 128) return small ? launch_simt<128, 1>(a, stream) : launch_simt<128, 4>(a, stream);
    return small ? launch_simt<64, 1>(a, stream) : launch_simt<64, 4>(a, stream);
}

}  // namespace

bool tree_attn_fits(const TreeAttnArgs& a)
{
    return a.bf16 ? tree_attn_tc_fits(a) : attn::line_fits(a, simt_shape_of(a.nodes, a.heads / a.kv_heads, a.dim));
}

size_t tree_attn_workspace_bytes(int batch, int nodes, int heads, int kv_heads, int dim, bool bf16)
{
    if (bf16) return tree_attn_tc_workspace_bytes(nodes, heads / kv_heads, dim);
    return attn::workspace_bytes(simt_shape_of(nodes, heads / kv_heads, dim), dim);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t stream)
{
    return a.bf16 ? launch_tree_attn_tc(a, stream) : launch_simt_dim(a, stream);
}

}  // namespace kda
