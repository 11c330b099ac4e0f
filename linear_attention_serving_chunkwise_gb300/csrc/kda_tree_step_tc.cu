// KDA on a draft tree, dk = dv = 128, with the state's products on the tensor cores (tcgen05).
// The formulas are those of kda_tree_step.cu; here is how they are spread.
//
// A (sequence, head) is a unit; nodes go in blocks of 16.  Of the two products with the state,
// X = (e^G k)^T S and Y = (e^G q)^T S, one MMA group gives all 32 rows of a block: the state is
// the A operand in tensor memory (lane = value channel, column = key channel), the block's e^G k
// and e^G q are the B operand.  The outputs are fp32, so both operands are split into two tf32
// parts, x = hi + lo to 2^-24: D = S_hi (E_hi | E_lo) + S_lo E_hi, the dropped lo lo product
// being of the size of an fp32 rounding.  A value channel's X and Y then lie in one lane, and the
// forward substitution over the nodes runs there in registers, one thread per channel.
//
// Warp roles of a persistent CTA, each ahead of the next by its buffers:
//     16        copies states (32 KB halves, 2 to 4 in flight: HBM's latency is covered by these)
//     4 - 7     split a state into tensor memory
//     8 - 15    prepare a block: G along the paths, e^G k and e^G q split into the B operand, and
//               A_ij = <e^{G_i - G_j} k_i, k_j>, P_ij = <e^{G_i - G_j} q_i, k_j> on the ancestor pairs
//               alone, each exponential of a difference <= 0 (a factored e^{-G_j} would overflow)
//     17        issues the products
//     0 - 3     substitution and outputs
// Bound: HBM (one read of the state) up to about 16 nodes, then the pairs of the preparation.
// Every wait is bounded (Waiter).
#include "kda_draft_launch.h"
#include "kda_draft_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int D = 128, NB = 16;                     // channels; nodes of a block
constexpr int kPrepThreads = 256, kThreads = 640, kCtas = 152;
// registers a thread: at launch, and after the split (substitution, state, preparation, the rest)
constexpr int kStartRegs = 96, kSolveRegs = 96, kSplitRegs = 104, kPrepRegs = 112, kRestRegs = 40;
static_assert(128 * (kSolveRegs + kSplitRegs + kRestRegs) + kPrepThreads * kPrepRegs <= kThreads * kStartRegs, "register split");
constexpr int kHalf = 64 * D * 4;                   // bytes of half a state
constexpr int kETile = 4 * NB * D * 4;              // k hi, q hi, k lo, q lo rows of a block
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColHi = 0, kColLo = 128, kColD = 256;   // D: two buffers of 64 columns

struct Plan {
    int states, tiles;      // halves of the state ring, B tiles
    int k, g, q, ap, w, shared, bytes;   // offsets
};

struct Shared {
    uint64_t s_full[4], s_empty[4], t_full, t_empty, e_full[2], e_empty[2], d_full[2], d_empty[2], a_full[2], a_empty[2];
    alignas(16) signed char parent[kTreeMaxNodes];   // -1: none
    TreeSmem tree[2];       // of the preparation, of the substitution
    uint32_t tmem;
};

__host__ __device__ constexpr Plan plan_of(int K, int states, int tiles)
{
    Plan p = {};
    p.states = states;
    p.tiles = tiles;
    int at = states * kHalf + tiles * kETile;
    p.k = at; at += K * D * 4;
    p.g = at; at += K * D * 4;
    p.q = at; at += NB * D * 4;
    p.ap = at; at += 2 * NB * ((K + 1) & ~1) * 8;   // two blocks' rows of (A, P), rows of 16-byte multiples
    p.w = at; at += K * D * 4;
    at = (at + 15) & ~15;
    p.shared = at;
    p.bytes = at + (int)sizeof(Shared);
    return p;
}

// x rounded to tf32 (half away from zero), in two integer operations: the conversion
// instruction runs at a quarter of their rate and would be the state split's bound.
__device__ __forceinline__ float to_tf32(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }
// the same for an operand of the tensor core, which drops the low bits itself
__device__ __forceinline__ float as_tf32(float x) { return __uint_as_float(__float_as_uint(x) + 0x1000u); }

struct Units {              // this CTA's, one after the other (a sequence's heads stay together)
    int first, last;
};

// ------------------------------------------------------------------ preparation
// (Loops are unrolled no more than their registers ask for: the five roles run side by side, and
// straight-line code for each would be fetched anew for every block.)
template <typename Tin>
__device__ __forceinline__ void prepare(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t)
{
    const int K = a.nodes, H = a.num_heads, KP = (K + 1) & ~1, lane = t & 31, w = t >> 5, c = t & 127;
    const bool decays = t < D;                      // one half of the threads has the decays, the other k and q
    float* sk = reinterpret_cast<float*>(base + pl.k);
    float* sg = reinterpret_cast<float*>(base + pl.g);
    float* sq = reinterpret_cast<float*>(base + pl.q);
    TreeSmem& tree = sm.tree[0];
    Waiter wait{a.status};
    uint32_t block = 0;
    int tree_of = -1;
    // channel c of a block's nodes, loaded a block ahead and kept as it lies in memory (a conversion
    // would wait for the load); past the last node the last one again
    float rg[NB];
    Tin rk[NB], rq[NB];
    auto load = [&](int u, int i0) {
        u = min(u, un.last - 1);
        const int b = u / H, h = u - b * H;
        const size_t at = ((size_t)b * K * H + h) * D + c;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const size_t o = at + (size_t)(min(i0 + i, K - 1) * H) * D;
            if (decays) {
                rg[i] = a.g[o];
            } else {
                rk[i] = static_cast<const Tin*>(a.k)[o];
                rq[i] = static_cast<const Tin*>(a.q)[o];
            }
        }
    };
    load(un.first, 0);
    for (int u = un.first; u < un.last; ++u) {
        const int b = u / H;
        if (b != tree_of) {
            bar_sync(1, kPrepThreads);              // the last tree has been read
            if (w == 0) {
                tree_masks(tree, a.parents + (size_t)b * K, K, lane);
                for (int i = lane; i < K; i += 32) {
                    const uint64_t above = tree.anc[i] & ~(1ull << i);
                    sm.parent[i] = tree.ok && above ? (signed char)(63 - __clzll((long long)above)) : (signed char)-1;
                }
            }
            tree_of = b;
        }
        for (int i0 = 0; i0 < K; i0 += NB, ++block) {
            const int n = min(NB, K - i0), eb = block % pl.tiles, ab = block & 1;
            bar_sync(1, kPrepThreads);              // the last block's k, q and G have been read; the tree is there
            if (decays) {
                // G in powers of two: a node's is its parent's and its own g; parents come first
                const uint4 up = *reinterpret_cast<const uint4*>(sm.parent + i0);
                const uint32_t ups[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (i >= n) break;
                    const int p = (int)(signed char)(ups[i / 4] >> 8 * (i % 4));
                    const float own = g_of(rg[i], a.prologue) * kLog2e;
                    sg[(i0 + i) * D + c] = p >= 0 ? own + sg[p * D + c] : own;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (i >= n) break;
                    sk[(i0 + i) * D + c] = to_f32(rk[i]);
                    sq[i * D + c] = to_f32(rq[i]);
                }
            }
            if (i0 + NB < K) load(u, i0 + NB);
            else load(u + 1, 0);
            bar_sync(1, kPrepThreads);
            if (a.prologue & kProQK) {
                for (int i = w; i < 2 * n; i += kPrepThreads / 32) {
                    float4* x = reinterpret_cast<float4*>(i & 1 ? sq + (i >> 1) * D : sk + (i0 + (i >> 1)) * D) + lane;
                    float4 v = *x;
                    float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float inv = l2_inv(ss);
                    *x = make_float4(l2_scale(v.x, inv, Tin{}), l2_scale(v.y, inv, Tin{}), l2_scale(v.z, inv, Tin{}), l2_scale(v.w, inv, Tin{}));
                }
                bar_sync(1, kPrepThreads);
            }
            // the B operand
            if (block >= (uint32_t)pl.tiles) wait(&sm.e_empty[eb], (block / pl.tiles - 1) & 1);
            uint8_t* et = base + pl.states * kHalf + eb * kETile;
#pragma unroll 2
            for (int i = t >> 7; i < n; i += 2) {   // (rows of the block beyond its nodes: columns of D that nobody reads)
                const float e = ex2(sg[(i0 + i) * D + c]);
                const float kx = sk[(i0 + i) * D + c] * e, qx = sq[i * D + c] * e, kh = to_tf32(kx), qh = to_tf32(qx);
                *reinterpret_cast<float*>(et + sw128_off_f32(i, c, 4 * NB)) = kh;
                *reinterpret_cast<float*>(et + sw128_off_f32(NB + i, c, 4 * NB)) = qh;
                *reinterpret_cast<float*>(et + sw128_off_f32(2 * NB + i, c, 4 * NB)) = as_tf32(kx - kh);
                *reinterpret_cast<float*>(et + sw128_off_f32(3 * NB + i, c, 4 * NB)) = as_tf32(qx - qh);
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.e_full[eb]);
            // the ancestor pairs: a warp to a node, a lane to four channels; entry e of the node's list is its
            // e-th ancestor from the context on, the last is the node itself
            if (block >= 2) wait(&sm.a_empty[ab], (block / 2 - 1) & 1);
            float2* ap = reinterpret_cast<float2*>(base + pl.ap) + ab * NB * KP;
#pragma unroll 1
            for (int i = w; i < n; i += kPrepThreads / 32) {
                const float4 ki = reinterpret_cast<const float4*>(sk + (i0 + i) * D)[lane], qi = reinterpret_cast<const float4*>(sq + i * D)[lane],
                             gi = reinterpret_cast<const float4*>(sg + (i0 + i) * D)[lane];
                auto dots = [&](int j, float& da, float& dp) {
                    const float4 kj = reinterpret_cast<const float4*>(sk + j * D)[lane], gj = reinterpret_cast<const float4*>(sg + j * D)[lane];
                    const float x = ex2(gi.x - gj.x) * kj.x, y = ex2(gi.y - gj.y) * kj.y, z = ex2(gi.z - gj.z) * kj.z, v = ex2(gi.w - gj.w) * kj.w;
                    da = fmaf(x, ki.x, fmaf(y, ki.y, fmaf(z, ki.z, v * ki.w)));
                    dp = fmaf(x, qi.x, fmaf(y, qi.y, fmaf(z, qi.z, v * qi.w)));
                };
                int e = 0;
#pragma unroll 1
                for (uint64_t m = tree.ok ? tree.anc[i0 + i] : 0ull; m; e += 2) {
                    // two pairs at a time; their four sums end in lanes 0, 8, 16 and 24
                    const int j0 = __ffsll((long long)m) - 1;
                    m &= m - 1;
                    const bool two = m != 0;
                    const int j1 = two ? __ffsll((long long)m) - 1 : j0;
                    m &= m - 1;
                    float a0, p0, a1, p1;
                    dots(j0, a0, p0);
                    dots(j1, a1, p1);
                    const bool up = lane & 16, mid = lane & 8;
                    float x = up ? a1 : a0, y = up ? p1 : p0;
                    x += __shfl_xor_sync(0xffffffffu, up ? a0 : a1, 16);
                    y += __shfl_xor_sync(0xffffffffu, up ? p0 : p1, 16);
                    float z = mid ? y : x;
                    z += __shfl_xor_sync(0xffffffffu, mid ? x : y, 8);
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                    if ((lane & 7) == 0 && (two || !up)) reinterpret_cast<float*>(ap + i * KP + e + (up ? 1 : 0))[mid ? 1 : 0] = z;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.a_full[ab]);
        }
    }
}

// ------------------------------------------------------------------ the state into tensor memory
__device__ __forceinline__ void split(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t)
{
    const int lane = t & 31, dv = t;                // lane of tensor memory = value channel
    const uint32_t quad = 32 * (t >> 5);
    Waiter wait{a.status};
    uint32_t half = 0, unit = 0;
    for (int u = un.first; u < un.last; ++u, ++unit) {
        for (int k = 0; k < 2; ++k, ++half) {
            const uint32_t s = half % pl.states;
            wait(&sm.s_full[s], (half / pl.states) & 1);
            if (k == 0 && unit) {
                wait(&sm.t_empty, (unit - 1) & 1);
                tc_fence_after_sync();
            }
            __syncwarp();
            const float* src = reinterpret_cast<const float*>(base + s * kHalf) + dv;
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
                float hi[32], lo[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = src[(c0 + i) * D];
                    hi[i] = to_tf32(x);
                    lo[i] = as_tf32(x - hi[i]);
                }
                tmem_st32(tmem_addr(sm.tmem, quad, kColHi + 64 * k + c0), hi);
                tmem_st32(tmem_addr(sm.tmem, quad, kColLo + 64 * k + c0), lo);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty[s]);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.t_full);
    }
}

// ------------------------------------------------------------------ the products
__device__ __forceinline__ void multiply(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base)
{
    Waiter wait{a.status};
    const uint32_t tm = sm.tmem, tiles = smem_u32(base) + pl.states * kHalf;
    uint32_t block = 0, unit = 0;
    for (int u = un.first; u < un.last; ++u, ++unit) {
        wait(&sm.t_full, unit & 1);
        for (int i0 = 0; i0 < a.nodes; i0 += NB, ++block) {
            const uint32_t eb = block % pl.tiles, db = block & 1;
            wait(&sm.e_full[eb], (block / pl.tiles) & 1);
            if (block >= 2) wait(&sm.d_empty[db], (block / 2 - 1) & 1);
            tc_fence_after_sync();
            if (elect_one()) {
                if (wait.alive) {
                    const uint64_t ed = kmajor_base(tiles + eb * kETile);
                    const uint32_t d = tm + kColD + 64 * db;
#pragma unroll
                    for (int ks = 0; ks < D / 8; ++ks)
                        umma_tf32_tmem_a(d, tm + kColHi + 8 * ks, desc_off(ed, kmajor_off(4 * NB, ks)), idesc_tf32_f32(128, 4 * NB), ks > 0);
#pragma unroll
                    for (int ks = 0; ks < D / 8; ++ks)
                        umma_tf32_tmem_a(d, tm + kColLo + 8 * ks, desc_off(ed, kmajor_off(4 * NB, ks)), idesc_tf32_f32(128, 2 * NB), 1);
                }
                umma_commit(&sm.e_empty[eb]);
                umma_commit(&sm.d_full[db]);
                if (i0 + NB >= a.nodes) umma_commit(&sm.t_empty);
            }
            __syncwarp();
        }
    }
    if (unit) wait(&sm.t_empty, (unit - 1) & 1);    // no product or commit is in flight after this
}

// ------------------------------------------------------------------ substitution and outputs
template <typename Tin>
__device__ __forceinline__ void solve(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t)
{
    const int K = a.nodes, H = a.num_heads, KP = (K + 1) & ~1, lane = t & 31;
    const uint32_t quad = 32 * (t >> 5);
    float* sw = reinterpret_cast<float*>(base + pl.w) + t;      // this channel's writes
    TreeSmem& tree = sm.tree[1];
    Waiter wait{a.status};
    uint32_t block = 0;
    int tree_of = -1;
    constexpr int Q = 4;                                        // nodes at a time
    Tin rv[Q];                                                  // their v and beta, loaded four nodes ahead
    float rb[Q];
    auto load = [&](int u, int i) {                             // (past the last node the last one again)
        u = min(u, un.last - 1);
        const int b = u / H, h = u - b * H;
#pragma unroll
        for (int k = 0; k < Q; ++k) {
            const size_t tok = ((size_t)b * K + min(i + k, K - 1)) * H + h;
            rv[k] = static_cast<const Tin*>(a.v)[tok * D + t];
            rb[k] = a.beta[tok];
        }
    };
    load(un.first, 0);
    for (int u = un.first; u < un.last; ++u) {
        const int b = u / H, h = u - b * H;
        if (b != tree_of) {
            bar_sync(2, 128);
            if (t < 32) {
                tree_masks(tree, a.parents + (size_t)b * K, K, lane);
                if (lane == 0 && !tree.ok) report_status(a.status, kDevBadSeqlens);
            }
            tree_of = b;
            bar_sync(2, 128);
        }
        for (int i0 = 0; i0 < K; i0 += NB, ++block) {
            const uint32_t db = block & 1;
            wait(&sm.d_full[db], (block / 2) & 1);
            wait(&sm.a_full[db], (block / 2) & 1);
            __syncwarp();
            tc_fence_after_sync();
            const uint32_t td = tmem_addr(sm.tmem, quad, kColD + 64 * db);
            const float2* ap = reinterpret_cast<const float2*>(base + pl.ap) + db * NB * KP;
#pragma unroll 1
            for (int g0 = 0; g0 < min(NB, K - i0); g0 += Q) {
                float x[Q], y[Q], x2[Q], y2[Q];                 // X and Y, and their parts from the low half of E
                tmem_ld4(td + g0, x);
                tmem_ld4(td + NB + g0, y);
                tmem_ld4(td + 2 * NB + g0, x2);
                tmem_ld4(td + 3 * NB + g0, y2);
                float v[Q], beta[Q];
#pragma unroll
                for (int k = 0; k < Q; ++k) { v[k] = to_f32(rv[k]); beta[k] = beta_of(rb[k], a.prologue); }
                if (i0 + g0 + Q < K) load(u, i0 + g0 + Q);
                else load(u + 1, 0);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int i = i0 + g0 + k;
                    if (i >= K || !tree.ok) break;
                    const size_t at = (((size_t)b * K + i) * H + h) * D + t;
                    const float2* row = ap + (g0 + k) * KP;
                    uint64_t m = tree.anc[i];
                    const bool there = m != 0;
                    m &= ~(1ull << i);
                    float xi = x[k] + x2[k], yi = y[k] + y2[k];
                    int e = 0;
#pragma unroll 1
                    while (m) {                                 // ancestors, two at a time
                        const float4 c = *reinterpret_cast<const float4*>(row + e);
                        const int j0 = __ffsll((long long)m) - 1;
                        m &= m - 1;
                        const float w0 = sw[j0 * D];
                        xi = fmaf(c.x, w0, xi);
                        yi = fmaf(c.y, w0, yi);
                        ++e;
                        if (m) {
                            const float w1 = sw[(__ffsll((long long)m) - 1) * D];
                            m &= m - 1;
                            xi = fmaf(c.z, w1, xi);
                            yi = fmaf(c.w, w1, yi);
                            ++e;
                        }
                    }
                    float wi = beta[k] * (v[k] - xi);
                    yi = fmaf(row[e].y, wi, yi);
                    if (!there) wi = yi = 0.f;                  // an absent node
                    if (a.gate) yi = gate1(yi, __ldg(a.gate + at));
                    sw[i * D] = wi;
                    a.writes[at] = wi;
                    a.out[at] = yi;
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.d_empty[db]);
                mbar_arrive(&sm.a_empty[db]);
            }
        }
    }
}

// ------------------------------------------------------------------ the states, by one thread
__device__ __forceinline__ void copy_states(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base)
{
    Waiter wait{a.status};
    const char* src = reinterpret_cast<const char*>(a.state) + (size_t)un.first * 2 * kHalf;
    const uint32_t halves = 2 * (un.last - un.first);
    uint32_t i = 0;
    for (; i < halves; ++i) {
        const uint32_t s = i % pl.states;
        if (i >= (uint32_t)pl.states) wait(&sm.s_empty[s], (i / pl.states - 1) & 1);
        if (!wait.alive) break;
        mbar_arrive_expect_tx(&sm.s_full[s], kHalf);
        bulk_load(base + s * kHalf, src + (size_t)i * kHalf, kHalf, &sm.s_full[s]);
    }
    // no load is in flight when the block ends, whatever became of its reader
    for (uint32_t j = i > (uint32_t)pl.states ? i - pl.states : 0; j < i; ++j)
        mbar_wait_bounded(&sm.s_full[j % pl.states], (j / pl.states) & 1, kDraftWaitNs);
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 1) tree_decode_tc_kernel(TreeDecodeArgs a, Plan pl)
{
    extern __shared__ __align__(1024) uint8_t base[];
    Shared& sm = *reinterpret_cast<Shared*>(base + pl.shared);
    const int t = threadIdx.x, warp = t >> 5, total = a.batch * a.num_heads;
    if (warp == 17) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (t == 0) {
        for (int i = 0; i < 4; ++i) { mbar_init(&sm.s_full[i], 1); mbar_init(&sm.s_empty[i], 4); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.e_full[i], kPrepThreads);
            mbar_init(&sm.e_empty[i], 1);
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_empty[i], 4);
            mbar_init(&sm.a_full[i], kPrepThreads / 32);
            mbar_init(&sm.a_empty[i], 4);
        }
        mbar_init(&sm.t_full, 4);
        mbar_init(&sm.t_empty, 1);
        mbar_fence_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const Units un = {(int)((long long)total * blockIdx.x / gridDim.x), (int)((long long)total * (blockIdx.x + 1) / gridDim.x)};
    if (warp < 4) {
        solve<Tin>(a, pl, un, sm, base, t);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSplitRegs));
        split(a, pl, un, sm, base, t - 128);
    } else if (warp < 16) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrepRegs));
        prepare<Tin>(a, pl, un, sm, base, t - 256);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
        if (warp == 17) multiply(a, pl, un, sm, base);
        if (warp == 16 && elect_one()) copy_states(a, pl, un, sm, base);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 17) tmem_dealloc(sm.tmem, 512);
}

// As many state halves and B tiles as fit: two tiles let the preparation run a block ahead of the
// products, and the states are what keeps HBM busy (three halves cover its latency at its full rate).
Plan choose_plan(int K)
{
    constexpr int options[][2] = {{4, 2}, {3, 2}, {2, 2}, {3, 1}, {2, 1}};
    for (const auto& o : options) {
        const Plan p = plan_of(K, o[0], o[1]);
        if (p.bytes <= 232448) return p;
    }
    return {};
}
static_assert(plan_of(kTreeMaxNodes, 2, 1).bytes <= 232448, "the largest tree fits");

template <typename Tin>
cudaError_t launch(const TreeDecodeArgs& a, cudaStream_t stream)
{
    const Plan p = choose_plan(a.nodes);
    static KernelSetup setup;
    const cudaError_t e = setup(tree_decode_tc_kernel<Tin>, 232448, kStartRegs);   // (the split needs its start)
    if (e != cudaSuccess) return e;
    const int total = a.batch * a.num_heads;
    tree_decode_tc_kernel<Tin><<<total < kCtas ? total : kCtas, kThreads, p.bytes, stream>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode_tc(const TreeDecodeArgs& a, cudaStream_t stream)
{
    return a.bf16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace kda
