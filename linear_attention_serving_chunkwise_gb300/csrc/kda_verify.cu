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
// the walk (K gathered probabilities, one warp) and scans its slice of the one row that is
// sampled.  The quotient is formed only where it can win: rest / noise > best is first tested as
// rest >= best (1 - 2^-21) noise, which no rounding can turn down wrongly, with the best of the
// whole warp, so that after the first batch few elements get as far as a division.
// Bound: HBM, 8 bytes (12 after a turned-down draft) per vocabulary entry, behind the walk's
// latency (about 4 us).  The rows' slices come by bulk copies of 4 KB through a ring of four stages: loads
// into registers, four at a time of 4 bytes a lane (rows need not start on 16 bytes), were
// throttled, 62 us instead of 48 for 256 chains of 4 over 100003 (281 MB with the drafts' rows,
// 5.8 TB/s of the copy's 6.8).  64 trees of 32 nodes over 131072: 21 us (67 MB); one row of 32003: 6.6 us.
// Eight stages of 2 KB: 66 us, two of 8 KB: 47, but one row 7.0.
#include <cooperative_groups.h>

#include "kda_draft_launch.h"
#include "kda_draft_sm100.cuh"
#include "kda_tree.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;         // the portable cluster size
constexpr int kBatch = 4;           // entries of a lane in a chunk
constexpr int kChunk = kThreads * kBatch, kStages = 4;
// a chunk of a row in shared memory, from the 16-byte boundary before it to the one after it
constexpr int kSlot = kChunk * 4 + 32, kRing = kStages * 3 * kSlot;

// larger score first, then the lower index; scores are >= 0, whose bits order like integers
__device__ __forceinline__ uint64_t key_of(uint32_t score, int idx) { return ((uint64_t)score << 32) | (uint32_t)(0xffffffffu - (uint32_t)idx); }
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// What is not above zero (a negative zero or NaN too) counts as zero.
__device__ __forceinline__ float above_zero(float x) { return x > 0.f ? x : 0.f; }

struct Walk {
    int kept[kTreeMaxNodes];        // the kept nodes in order
    int tok[kTreeMaxNodes];         // tokens turned down at the last node (no draft)
    int n_kept, n_down, row, first_down, bad;
};

// One warp: the walk.  A lane holds nodes lane and lane + 32; the children of the current node
// are a ballot away and each test is a few shuffles.
__device__ void walk_tree(const VerifyArgs& a, int b, Walk& wk, int lane)
{
    const int K = a.nodes;
    int par[2], tok[2];
    float p[2] = {}, q[2] = {}, u[2] = {};
    bool bad = false;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int i = lane + 32 * s;
        par[s] = kTreePad;
        tok[s] = -1;
        if (i < K) {
            par[s] = a.parents[(size_t)b * K + i];
            tok[s] = a.tokens[(size_t)b * K + i];
            u[s] = a.uniforms[(size_t)b * K + i];
        }
        const bool there = par[s] != kTreePad, ok = par[s] >= kTreePad && par[s] < i && (!there || (tok[s] >= 0 && tok[s] < a.vocab));
        bad |= !ok;
        if (ok && there) {
            p[s] = a.target[((size_t)b * (K + 1) + par[s] + 1) * a.vocab + tok[s]];
            if (a.draft) q[s] = a.draft[((size_t)b * K + i) * a.vocab + tok[s]];
        }
        if (!there) tok[s] = -1;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (!bad) {
        // a node may not hang on an absent one; a draft row belongs to one child
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int src = max(par[s], 0), lo = __shfl_sync(0xffffffffu, par[0], src & 31), hi = __shfl_sync(0xffffffffu, par[1], src & 31);
            bad |= par[s] >= 0 && (src < 32 ? lo : hi) == kTreePad;
        }
        if (a.draft) {
            for (int x = -1; x < K; ++x)
                bad |= __popc(__ballot_sync(0xffffffffu, par[0] == x)) + __popc(__ballot_sync(0xffffffffu, par[1] == x)) > 1;
        }
        bad = __any_sync(0xffffffffu, bad);
    }
    int cur = -1, n = 0;
    uint64_t down = 0;                                       // children of cur turned down
    if (!bad) {
        for (bool on = true; on;) {
            uint64_t left = (uint64_t)__ballot_sync(0xffffffffu, par[0] == cur) | (uint64_t)__ballot_sync(0xffffffffu, par[1] == cur) << 32;
            float mass = 1.f;
            down = 0;
            on = false;
            for (; left; left &= left - 1) {
                const int c = __ffsll((long long)left) - 1, src = c & 31;
                const bool hi = c >= 32;
                const int x = __shfl_sync(0xffffffffu, hi ? tok[1] : tok[0], src);
                const float pc = __shfl_sync(0xffffffffu, hi ? p[1] : p[0], src), uc = __shfl_sync(0xffffffffu, hi ? u[1] : u[0], src),
                            qc = __shfl_sync(0xffffffffu, hi ? q[1] : q[0], src);
                bool keep;
                if (a.draft) {
                    keep = __fmul_rn(uc, qc) < pc;
                } else {                                     // a token turned down here before has no mass left
                    const uint64_t same = (uint64_t)__ballot_sync(0xffffffffu, tok[0] == x) | (uint64_t)__ballot_sync(0xffffffffu, tok[1] == x) << 32;
                    if (same & down) {
                        down |= 1ull << c;
                        continue;
                    }
                    keep = __fmul_rn(uc, mass) < pc;
                }
                if (keep) {
                    if (lane == 0) wk.kept[n] = c;
                    ++n;
                    cur = c;
                    on = true;
                    break;
                }
                down |= 1ull << c;
                mass = __fsub_rn(mass, pc);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int i = lane + 32 * s;
        if (i < 64 && (down >> i & 1)) wk.tok[__popcll(down & ((1ull << i) - 1))] = tok[s];
    }
    if (lane == 0) {
        wk.bad = bad;
        wk.n_kept = n;
        wk.n_down = __popcll(down);
        wk.first_down = down ? __ffsll((long long)down) - 1 : -1;
        wk.row = cur + 1;
    }
}

// A lane's best so far, and the least score worth a division: the warp's best less 2^-21 of it.
struct Best {
    uint32_t score = 0;
    int idx = 0;
    float worth = 0.f;
};

// One entry that may win: r is what is left of it before the turned-down tokens are taken out.
__device__ __forceinline__ void offer(Best& best, float r, float noise, int v, const Walk& wk, int n_down)
{
    const uint32_t s = __float_as_uint(__fdiv_rn(r, noise));
    if (s < best.score || (s == best.score && v > best.idx)) return;
    for (int j = 0; j < n_down; ++j)
        if (wk.tok[j] == v) return;
    best.score = s;
    best.idx = v;
}

__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// A part of a row on its way to shared memory: 16-byte pieces that cover entries [c0, c1).
struct Span16 {
    const char* src;
    uint32_t bytes, shift;      // entry c0 is `shift` floats behind the copy's start
    __device__ __forceinline__ Span16(const float* row, int c0, int c1)
    {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(row + c0), hi = reinterpret_cast<uintptr_t>(row + c1);
        src = reinterpret_cast<const char*>(lo & ~(uintptr_t)15);
        bytes = (uint32_t)(((hi + 15) & ~(uintptr_t)15) - (lo & ~(uintptr_t)15));
        shift = (uint32_t)(lo & 15) / 4;
    }
};

__global__ void __launch_bounds__(kThreads, 4) verify_kernel(VerifyArgs a)
{
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int b = blockIdx.x / C, t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int V = a.vocab;                      // (at most KDA_VERIFY_MAX_VOCAB: a slice's end and a chunk past it stay in 31 bits)
    extern __shared__ __align__(16) unsigned char ring[];       // [stage][p, noise, q][kSlot]
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ Walk wk;
    __shared__ uint64_t red[kWarps];
    __shared__ uint64_t best[2][kCluster];      // by pass; every rank's copy collects all ranks' bests

    const float* nrow = a.noise + (size_t)b * V;
    const int per = ((V + C - 1) / C + 3) & ~3;
    const int v0 = min(V, rank * per), v1 = min(V, v0 + per);
    // The slice but for four entries at each end comes in chunks (a copy of whole 16 bytes then stays
    // inside the slice, whatever its alignment); thread 32 sends for them: the noise of the first
    // ones before the walk has said which rows it goes with.
    const int in0 = v0 + 4, in1 = v1 - 4, chunks = in1 > in0 ? (in1 - in0 + kChunk - 1) / kChunk : 0;
    Waiter wait{a.status};
    const auto slot = [&](int i, int row) { return ring + ((i % kStages) * 3 + row) * kSlot; };
    const auto send = [&](int i, int row, const float* from) {
        const int c0 = in0 + i * kChunk;
        const Span16 s(from, c0, min(in1, c0 + kChunk));
        expect_tx(&full[i % kStages], s.bytes);
        bulk_load(slot(i, row), s.src, s.bytes, &full[i % kStages]);
    };
    if (t == 32) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        mbar_fence_init();
        for (int i = 0; i < min(chunks, kStages); ++i) send(i, 1, nrow);
    }
    if (w == 0) walk_tree(a, b, wk, lane);
    cl.sync();                                  // every CTA of the cluster runs: its shared memory can be written

    const float* prow = a.target + ((size_t)b * (a.nodes + 1) + wk.row) * V;
    uint64_t win = 0;
    if (wk.bad) {
        if (t == 32)                            // (no copy is in flight when the CTA leaves)
            for (int i = 0; i < min(chunks, kStages); ++i) {
                mbar_arrive(&full[i]);
                wait(&full[i], 0);
            }
    } else {
        // pass 0 draws from what is left; pass 1 from the row itself, when nothing is left
        for (int pass = 0; pass < 2; ++pass) {
            const float* qrow = pass == 0 && a.draft && wk.first_down >= 0 ? a.draft + ((size_t)b * a.nodes + wk.first_down) * V : nullptr;
            const int n_down = pass == 0 && !a.draft ? wk.n_down : 0;
            Best mine;
            const auto one = [&](int v) {
                float r = above_zero(prow[v]);
                if (qrow) r = above_zero(__fsub_rn(r, qrow[v]));
                const float n = nrow[v];
                if (r >= mine.worth * n) offer(mine, r, n, v, wk, n_down);
            };
            if (pass == 0 && chunks) {
                const auto send_rest = [&](int i) {
                    send(i, 0, prow);
                    if (qrow) send(i, 2, qrow);
                    mbar_arrive(&full[i % kStages]);
                };
                if (t == 32)
                    for (int i = 0; i < min(chunks, kStages); ++i) send_rest(i);
                __syncwarp();
                const uint32_t ps = Span16(prow, in0, in1).shift, ns = Span16(nrow, in0, in1).shift, qs = qrow ? Span16(qrow, in0, in1).shift : 0;
                const int e0 = w * 32 * kBatch + lane;
                for (int i = 0; i < chunks; ++i) {
                    const int next = i + kStages - 1;       // into the stage that chunk i - 1 has left
                    if (t == 32 && i > 0 && next < chunks) {
                        wait(&empty[next % kStages], (next / kStages - 1) & 1);
                        send(next, 1, nrow);
                        send_rest(next);
                    }
                    __syncwarp();
                    wait(&full[i % kStages], (i / kStages) & 1);
                    const float *sp = reinterpret_cast<const float*>(slot(i, 0)) + ps + e0, *sn = reinterpret_cast<const float*>(slot(i, 1)) + ns + e0,
                                *sq = reinterpret_cast<const float*>(slot(i, 2)) + qs + e0;
                    const int v = in0 + i * kChunk + e0;
                    float p[kBatch], e[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const bool in = v + 32 * k < in1;
                        p[k] = in ? above_zero(sp[32 * k]) : 0.f;
                        e[k] = in ? sn[32 * k] : 1.f;
                        if (qrow && in) p[k] = above_zero(__fsub_rn(p[k], sq[32 * k]));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[i % kStages]);
                    bool any = false;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) any |= p[k] >= mine.worth * e[k];
                    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        if (p[k] >= mine.worth * e[k]) offer(mine, p[k], e[k], v + 32 * k, wk, n_down);
                    mine.worth = __uint_as_float(__reduce_max_sync(0xffffffffu, mine.score)) * (1.f - 0x1p-21f);
                }
                if (t < 8) one(t < 4 ? v0 + t : v1 - 8 + t);
            } else {
#pragma unroll 4
                for (int v = v0 + t; v < v1; v += kThreads) one(v);
            }
            uint64_t key = key_of(mine.score, mine.idx);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) key = max64(key, __shfl_xor_sync(0xffffffffu, key, o));
            if (lane == 0) red[w] = key;
            __syncthreads();
            if (t < C) {                        // thread r hands this CTA's best to rank r
                uint64_t m = 0;
                for (int i = 0; i < kWarps; ++i) m = max64(m, red[i]);
                *cl.map_shared_rank(&best[pass][rank], t) = m;
            }
            cl.sync();
            win = 0;
            for (int i = 0; i < C; ++i) win = max64(win, best[pass][i]);
            if ((win >> 32) != 0) break;        // the same in every CTA of the cluster
        }
    }
    wait.finish();
    cl.sync();                                  // no CTA leaves while another may still write to it
    if (rank == 0) {
        const int n = wk.bad ? 0 : wk.n_kept;
        for (int i = t; i < a.nodes; i += kThreads) a.path[(size_t)b * a.nodes + i] = i < n ? wk.kept[i] : -1;
        if (t == 0) {
            a.n_accept[b] = n;
            // (a row without any probability: the lowest index, as an argmax over zeros has it)
            a.next_token[b] = wk.bad ? -1 : (win >> 32) ? (int)(0xffffffffu - (uint32_t)win) : 0;
            if (wk.bad) report_status(a.status, kDevBadSeqlens);
        }
    }
}

}  // namespace

// A CTA spends about 4 us on the walk and on meeting its cluster, whatever its slice.  So all CTAs
// should run at once (4 to an SM, by their rings): a cluster is made smaller and its slices longer
// until they do.  256 rows of 100003: 48 us with clusters of 2, 53 of 4, 58 of 1; 100 trees over 131072:
// 28 us with 4, 35 with 8, 39 with 2.
constexpr long long kMostCtas = 4 * 152;

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream)
{
    int cluster = kCluster;
    while (cluster > 1 && (long long)a.batch * cluster > kMostCtas) cluster /= 2;
    static KernelSetup setup;
    const cudaError_t e = setup(verify_kernel, kRing);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRing;
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
