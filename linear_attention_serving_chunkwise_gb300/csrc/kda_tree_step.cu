// KDA on a draft tree: the outputs of every node from one read of the state (kda_tree_decode),
// and the state moved to the end of an accepted path (kda_tree_commit).  The linear-attention
// counterpart of kda_decode_multi, whose drafts are a chain (llm-atlas "K3_RESEARCH.md", Q28:
// draft tokens; Q07: the O(1) state update).
//
// With S_i = (I - beta_i k_i k_i^T) Diag(e^{g_i}) S_{parent(i)} + beta_i k_i v_i^T, G_i the sum of
// g along the path from the context to node i, and j over the nodes of that path,
//     w_i = beta_i (v_i - (e^{G_i} k_i)^T S - sum_{j above i} <e^{G_i - G_j} k_i, k_j> w_j)
//     o_i = (e^{G_i} q_i)^T S + sum_{j on i's path} <e^{G_i - G_j} q_i, k_j> w_j
// so the state S is read once for all nodes and nothing of the size of a state is kept per
// node.  e^{G_i - G_j} is formed as one exponential of a difference <= 0, for ancestor pairs
// only: no factor of it can overflow, however deep the tree, and a g of -inf is a reset (path_g).  The commit is then
//     S <- Diag(e^{G_n}) S + sum_{j on the path} (e^{G_n - G_j} k_j) w_j^T.
// Here: the step for dk = 64 on the CUDA cores (dk = 128: kda_tree_step_tc.cu), and the commit.
// The step's bound: instruction issue and shared memory, 64 x 96 heads x 16 nodes 205 us, 1.04 TB/s;
// at dk = 128 this form took 666 us where the tensor cores' takes 229.  The commit's: HBM, one read
// and one write of the state; 256 x 96 heads, dk = 128: 466 us, 6.9 TB/s, the rate of a copy (with the prologue 525).  A CTA a
// state in registers has its 64 KB in flight at once, and the path's few vectors are folded
// while the state arrives.
#include "kda_draft_launch.h"
#include "kda_tree.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ the step
// One CTA per (sequence, head), 2 D threads.  Warp w owns state columns [16 w, 16 w + 16); lane
// (rs, cq) holds rows [rs D/8, ...) of the float4 column 4 cq in registers.
template <int D>
struct StepLayout {
    // floats: k, q, G of every node, then X (becoming w) and Y, then A and P
    static __host__ __device__ size_t floats(int K) { return (size_t)K * D * 5 + 2 * (size_t)K * K; }
};

template <typename Tin, int D>
__global__ void __launch_bounds__(2 * D) tree_decode_kernel(TreeDecodeArgs a)
{
    constexpr int kThreads = 2 * D, kWarps = kThreads / 32, R = D / 8, C = D / 32;
    extern __shared__ __align__(16) float sm[];
    __shared__ TreeSmem ts;
    const int K = a.nodes, H = a.num_heads;
    float* sk = sm;
    float* sq = sk + K * D;
    float* sg = sq + K * D;
    float* sx = sg + K * D;
    float* sy = sx + K * D;
    float* sA = sy + K * D;
    float* sP = sA + K * K;

    const int bh = blockIdx.x, b = bh / H, h = bh % H;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int rs = lane >> 2, cq = lane & 3, col = 16 * w + 4 * cq, r0 = rs * R;

    const float* S = a.state + (size_t)bh * D * D + col;
    float4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(r0 + i) * D));

    if (w == 0) tree_masks(ts, a.parents + (size_t)b * K, K, lane);
    for (int idx = t; idx < K * D; idx += kThreads) {
        const int j = idx / D, c = idx - j * D;
        const size_t at = (((size_t)b * K + j) * H + h) * D + c;
        sk[idx] = to_f32(static_cast<const Tin*>(a.k)[at]);
        sq[idx] = to_f32(static_cast<const Tin*>(a.q)[at]);
        sg[idx] = path_g(a.g[at], a.prologue);
    }
    __syncthreads();
    if (!ts.ok) {
        if (t == 0 && h == 0) report_status(a.status, kDevBadSeqlens);
        return;
    }
    if (a.prologue & kProQK) {
        for (int i = w; i < 2 * K; i += kWarps) {
            float* x = (i & 1 ? sq : sk) + (i >> 1) * D;
            float ss = 0.f;
            for (int c = lane; c < D; c += 32) ss += x[c] * x[c];
            const float inv = l2_inv(warp_sum(ss));
            for (int c = lane; c < D; c += 32) x[c] = l2_scale(x[c], inv, Tin{});
        }
        __syncthreads();
    }
    // G: a thread per channel walks the nodes in order (parents come first)
    if (t < D) {
        for (int i = 0; i < K; ++i) {
            const uint64_t above = ts.anc[i] & ~(1ull << i);
            if (above) sg[i * D + t] += sg[(63 - __clzll((long long)above)) * D + t];   // the last one above i is its parent
        }
    }
    __syncthreads();
    // A and P on the pairs of one path, a warp per pair (pairs dealt by node)
    for (int i = 0; i < K; ++i) {
        uint64_t m = ts.anc[i];
        int nth = i;
        while (m) {
            const int j = __ffsll((long long)m) - 1;
            m &= m - 1;
            if ((nth++) % kWarps != w) continue;
            float da = 0.f, dp = 0.f;
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const int c = lane + 32 * e;
                const float x = expf(sg[i * D + c] - sg[j * D + c]) * sk[j * D + c];
                da = fmaf(x, sk[i * D + c], da);
                dp = fmaf(x, sq[i * D + c], dp);
            }
            da = warp_sum(da);
            dp = warp_sum(dp);
            if (lane == 0) { sA[i * K + j] = da; sP[i * K + j] = dp; }
        }
    }
    __syncthreads();
    for (int idx = t; idx < K * D; idx += kThreads) {
        const float e = expf(sg[idx]);
        sk[idx] *= e;
        sq[idx] *= e;
    }
    __syncthreads();
    // X = (e^G k)^T S, Y = (e^G q)^T S
    for (int v = 0; v < 2 * K; ++v) {
        const float* x = (v < K ? sk + v * D : sq + (v - K) * D) + r0;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float e = x[i];
            acc.x = fmaf(e, s[i].x, acc.x);
            acc.y = fmaf(e, s[i].y, acc.y);
            acc.z = fmaf(e, s[i].z, acc.z);
            acc.w = fmaf(e, s[i].w, acc.w);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
        if (rs == 0) *reinterpret_cast<float4*>((v < K ? sx + v * D : sy + (v - K) * D) + col) = acc;
    }
    __syncthreads();
    // the writes and outputs: every value channel is on its own
    if (t < D) {
        for (int i = 0; i < K; ++i) {
            const size_t tok = ((size_t)b * K + i) * H + h;
            uint64_t m = ts.anc[i];
            float wi = 0.f, oi = 0.f;
            if (m) {
                m &= ~(1ull << i);
                float x = sx[i * D + t];
                oi = sy[i * D + t];
                while (m) {
                    const int j = __ffsll((long long)m) - 1;
                    m &= m - 1;
                    const float wj = sx[j * D + t];
                    x = fmaf(sA[i * K + j], wj, x);
                    oi = fmaf(sP[i * K + j], wj, oi);
                }
                wi = beta_of(a.beta[tok], a.prologue) * (to_f32(static_cast<const Tin*>(a.v)[tok * D + t]) - x);
                oi = fmaf(sP[i * K + i], wi, oi);
                if (a.gate) oi = gate1(oi, a.gate[tok * D + t]);
            }
            sx[i * D + t] = wi;
            a.writes[tok * D + t] = wi;
            a.out[tok * D + t] = oi;
        }
    }
}

// ------------------------------------------------------------------ the commit
constexpr int kCommitThreads = 256;
constexpr int kCommitChunk = 8;      // path tokens folded into one update of the state

// One CTA per (sequence, head); a thread holds D / (256 / (D/4)) rows of one float4 column.
// CTAs an SM has room for, which is what keeps HBM busy while each waits for its path's vectors:
// 256 x 96 heads x 8 nodes took 530 us with two of dk = 128, 464 with three; of dk = 64 188 with
// two, 162 with four, 132 with six, 145 with eight (whose 32 registers a thread spill).
template <typename Tin, int D>
__global__ void __launch_bounds__(kCommitThreads, D == 128 ? 3 : 6) tree_commit_kernel(TreeCommitArgs a)
{
    constexpr int C4 = D / 4, RG = kCommitThreads / C4, RP = D / RG, NW = kCommitThreads / 32;
    const int K = a.nodes, H = a.num_heads;
    const int bh = blockIdx.x, b = bh / H, h = bh % H;
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5, cg = t % C4, rg = t / C4;
    __shared__ float sc[kCommitChunk][D], sw[kCommitChunk][D], sdec[D], sinv[kCommitChunk];
    __shared__ int snode[kTreeMaxNodes];
    __shared__ int sbad;

    const int n = a.n_accept[b];
    if (n == 0) return;
    if (t == 0) sbad = n < 0 || n > K;
    __syncthreads();
    if (!sbad && t < n) {
        snode[t] = a.path[(size_t)b * K + t];
        if (snode[t] < 0 || snode[t] >= K) sbad = 1;
    }
    __syncthreads();
    if (sbad) {
        if (t == 0 && h == 0) report_status(a.status, kDevBadSeqlens);
        return;
    }

    float* S = a.state + (size_t)bh * D * D;
    float4 s[RP];
#pragma unroll
    for (int i = 0; i < RP; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)(rg * RP + i) * D) + cg);

    for (int d0 = 0; d0 < n; d0 += kCommitChunk) {
        const int m = min(kCommitChunk, n - d0);
        if (d0) __syncthreads();
        for (int idx = t; idx < m * D; idx += kCommitThreads) {
            const int j = idx / D, c = idx - j * D;
            sw[j][c] = a.writes[(((size_t)b * K + snode[d0 + j]) * H + h) * D + c];
        }
        if (a.prologue & kProQK) {
            for (int j = wp; j < m; j += NW) {
                const Tin* k = static_cast<const Tin*>(a.k) + (((size_t)b * K + snode[d0 + j]) * H + h) * D;
                float ss = 0.f;
                for (int c = lane; c < D; c += 32) { const float x = to_f32(k[c]); ss += x * x; }
                ss = warp_sum(ss);
                if (lane == 0) sinv[j] = l2_inv(ss);
            }
            __syncthreads();
        }
        if (t < D) {                         // from the last token back: the decay after each one's write
            float after = 0.f;
            for (int j = m - 1; j >= 0; --j) {
                const size_t at = (((size_t)b * K + snode[d0 + j]) * H + h) * D + t;
                float k = to_f32(static_cast<const Tin*>(a.k)[at]);
                if (a.prologue & kProQK) k = l2_scale(k, sinv[j], Tin{});
                sc[j][t] = expf(after) * k;
                after += g_of(a.g[at], a.prologue);
            }
            sdec[t] = expf(after);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const float d = sdec[rg * RP + i];
            s[i].x *= d; s[i].y *= d; s[i].z *= d; s[i].w *= d;
        }
        for (int j = 0; j < m; ++j) {
            const float4 w4 = *reinterpret_cast<const float4*>(&sw[j][4 * cg]);
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const float c = sc[j][rg * RP + i];
                s[i].x = fmaf(c, w4.x, s[i].x);
                s[i].y = fmaf(c, w4.y, s[i].y);
                s[i].z = fmaf(c, w4.z, s[i].z);
                s[i].w = fmaf(c, w4.w, s[i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RP; ++i) __stcs(reinterpret_cast<float4*>(S + (size_t)(rg * RP + i) * D) + cg, s[i]);
}

template <typename Tin, int D>
cudaError_t launch_step(const TreeDecodeArgs& a, cudaStream_t stream)
{
    const size_t smem = StepLayout<D>::floats(a.nodes) * sizeof(float);
    static KernelSetup setup;
    const cudaError_t e = setup(tree_decode_kernel<Tin, D>, StepLayout<D>::floats(kTreeMaxNodes) * sizeof(float));
    if (e != cudaSuccess) return e;
    tree_decode_kernel<Tin, D><<<a.batch * a.num_heads, 2 * D, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename Tin, int D>
cudaError_t launch_commit(const TreeCommitArgs& a, cudaStream_t stream)
{
    tree_commit_kernel<Tin, D><<<a.batch * a.num_heads, kCommitThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode(const TreeDecodeArgs& a, cudaStream_t stream)
{
    if (a.dk == 128) return launch_tree_decode_tc(a, stream);
    return a.bf16 ? launch_step<__nv_bfloat16, 64>(a, stream) : launch_step<float, 64>(a, stream);
}

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t stream)
{
    if (a.dk == 128) return a.bf16 ? launch_commit<__nv_bfloat16, 128>(a, stream) : launch_commit<float, 128>(a, stream);
    return a.bf16 ? launch_commit<__nv_bfloat16, 64>(a, stream) : launch_commit<float, 64>(a, stream);
}

}  // namespace kda
