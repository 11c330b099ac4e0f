// Verification of drafted tokens against the target's probabilities, from given random
// numbers: which drafted tokens are kept and which token follows them (llm-atlas
// "K3_RESEARCH.md", Q28: the MTP layer tuned into an EAGLE-3 draft model).
//
// The walk starts at the context (row 0 of the target) and looks at the children of the
// current node in index order; child c with token x and uniform u is kept when
//     draft given:  u * q_c(x) < p(x)          (kept with probability min(1, p / q))
//     no draft:     u * m < p(x), m = 1 - sum of p over the children turned down before it
// and the walk goes on from c.  Where no child is kept, the next token is drawn from what is
// left of the current row: max(p - q, 0) with a draft, p without the turned-down tokens
// otherwise (p itself when nothing is left or nothing was turned down), as the argmax of
// rest(v) / noise(v): with noise ~ Exp(1) that is a draw from rest / sum(rest), so no sum
// over the vocabulary is needed, and every step is one IEEE operation on each element: the
// result does not depend on how the vocabulary is split.
//
// One thread-block cluster per sequence, the vocabulary split over its CTAs; each CTA repeats
// the walk (K gathered probabilities) and scans its slice of the one row that is sampled.
// Bound: HBM, 8 bytes (12 after a turned-down draft) per vocabulary entry.
#include <cooperative_groups.h>

#include "kda_draft_launch.h"
#include "kda_tree.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;      // the portable cluster size

// larger score first, then the lower index; scores are >= 0, whose bits order like integers
__device__ __forceinline__ uint64_t key_of(float score, int idx)
{
    return ((uint64_t)__float_as_uint(score) << 32) | (uint32_t)(0xffffffffu - (uint32_t)idx);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// What is not above zero (a negative zero or NaN too) counts as zero.
__device__ __forceinline__ float above_zero(float x) { return x > 0.f ? x : 0.f; }

struct Walk {
    int kept[kTreeMaxNodes];        // the kept nodes in order
    int tok[kTreeMaxNodes];         // tokens turned down at the last node (no draft)
    int n_kept, n_down, row, first_down, bad;
};

// Warp 0: the walk.  Lanes gather what every node's test needs, then lane 0 walks.
__device__ void walk_tree(const VerifyArgs& a, int b, Walk& wk, float* sp, float* sq, int* stok, int* spar, float* su, int lane)
{
    const int K = a.nodes;
    bool bad = false;
    for (int i = lane; i < K; i += 32) {
        const int p = a.parents[(size_t)b * K + i], x = a.tokens[(size_t)b * K + i];
        bool ok = p >= kTreePad && p < i;
        if (p != kTreePad) ok = ok && x >= 0 && x < a.vocab;
        spar[i] = p;
        stok[i] = x;
        su[i] = a.uniforms[(size_t)b * K + i];
        if (ok && p != kTreePad) {
            sp[i] = a.target[((size_t)b * (K + 1) + p + 1) * a.vocab + x];
            if (a.draft) sq[i] = a.draft[((size_t)b * K + i) * a.vocab + x];
        }
        bad |= !ok;
    }
    __syncwarp();
    if (!__any_sync(0xffffffffu, bad)) {
        for (int i = lane; i < K; i += 32) {
            const int p = spar[i];
            if (p >= 0 && spar[p] == kTreePad) bad = true;                                  // hangs on an absent node
            if (a.draft && p != kTreePad)                                                   // a draft row belongs to one child
                for (int j = 0; j < i; ++j) bad |= spar[j] == p;
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        wk.bad = bad;
        int cur = -1, n = 0, down = 0, first = -1;
        float mass = 1.f;
        if (!bad) {
            for (int c = 0; c < K; ++c) {       // children come after their parents: one pass in index order
                if (spar[c] != cur) continue;
                const float p = sp[c];
                bool keep;
                if (a.draft) {
                    keep = __fmul_rn(su[c], sq[c]) < p;
                } else {
                    bool again = false;          // a token turned down here before has no mass left
                    for (int j = 0; j < down; ++j) again |= wk.tok[j] == stok[c];
                    if (again) continue;
                    keep = __fmul_rn(su[c], mass) < p;
                }
                if (keep) {
                    wk.kept[n++] = c;
                    cur = c;
                    mass = 1.f;
                    down = 0;
                    first = -1;
                } else {
                    wk.tok[down++] = stok[c];
                    if (first < 0) first = c;
                    mass = __fsub_rn(mass, p);
                }
            }
        }
        wk.n_kept = n;
        wk.n_down = down;
        wk.first_down = first;
        wk.row = cur + 1;
    }
}

__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a)
{
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int b = blockIdx.x / C, t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int V = a.vocab;
    __shared__ Walk wk;
    __shared__ float sp[kTreeMaxNodes], sq[kTreeMaxNodes], su[kTreeMaxNodes];
    __shared__ int stok[kTreeMaxNodes], spar[kTreeMaxNodes];
    __shared__ uint64_t red[kThreads / 32];
    __shared__ uint64_t best[2][kMaxCluster];   // by pass; rank 0's copy collects, every rank gets the result

    if (w == 0) walk_tree(a, b, wk, sp, sq, stok, spar, su, lane);
    cl.sync();                                 // every CTA of the cluster runs: its shared memory can be written

    const float* prow = a.target + ((size_t)b * (a.nodes + 1) + wk.row) * V;
    const float* nrow = a.noise + (size_t)b * V;
    const int per = (V + C - 1) / C;
    const int v0 = rank * per, v1 = min(V, v0 + per);
    uint64_t win = 0;
    if (!wk.bad) {
        // pass 0 draws from what is left; pass 1 from the row itself, when nothing is left
        for (int pass = 0; pass < 2; ++pass) {
            const float* qrow = pass == 0 && a.draft && wk.first_down >= 0 ? a.draft + ((size_t)b * a.nodes + wk.first_down) * V : nullptr;
            const int n_down = pass == 0 && !a.draft ? wk.n_down : 0;
            uint64_t mine = 0;
            for (int v = v0 + t; v < v1; v += kThreads) {
                float r = above_zero(prow[v]);
                if (qrow) r = above_zero(__fsub_rn(r, qrow[v]));
                for (int j = 0; j < n_down; ++j) r = wk.tok[j] == v ? 0.f : r;
                mine = max64(mine, key_of(__fdiv_rn(r, nrow[v]), v));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine = max64(mine, __shfl_xor_sync(0xffffffffu, mine, o));
            if (lane == 0) red[w] = mine;
            __syncthreads();
            if (t < C) {                       // thread r hands this CTA's best to rank r
                uint64_t m = 0;
                for (int i = 0; i < kThreads / 32; ++i) m = max64(m, red[i]);
                *cl.map_shared_rank(&best[pass][rank], t) = m;
            }
            cl.sync();
            win = 0;
            for (int i = 0; i < C; ++i) win = max64(win, best[pass][i]);
            if ((win >> 32) != 0) break;       // the same in every CTA of the cluster
        }
    }
    cl.sync();                                 // no CTA leaves while another may still write to it
    if (rank == 0) {
        const int n = wk.bad ? 0 : wk.n_kept;
        for (int i = t; i < a.nodes; i += kThreads) a.path[(size_t)b * a.nodes + i] = i < n ? wk.kept[i] : -1;
        if (t == 0) {
            a.n_accept[b] = n;
            a.next_token[b] = wk.bad ? -1 : (int)(0xffffffffu - (uint32_t)win);
            if (wk.bad) report_status(a.status, kDevBadSeqlens);
        }
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream)
{
    int cluster = kMaxCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a);
}

}  // namespace kda
