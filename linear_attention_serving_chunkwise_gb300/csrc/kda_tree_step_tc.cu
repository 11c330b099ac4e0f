// KDA on a draft tree, dk = dv = 128, with the state's products on the tensor cores (tcgen05).
// The formulas are those of kda_tree_step.cu; here is how they are spread.
//
// A (sequence, head) is a unit; nodes go in blocks of 16.  Of the two products with the state,
// X = (e^G k)^T S and Y = (e^G q)^T S, one MMA group gives all 32 rows of a block: the state is
// the A operand in tensor memory (lane = value channel, column = key channel), the block's e^G k
// and e^G q are the B operand.  The outputs are fp32, so both operands are split into two tf32
// parts, x = hi + lo to 2^-23: D = S_hi (E_hi | E_lo) + S_lo E_hi, the dropped lo lo product
// being of the size of an fp32 rounding.  A value channel's X and Y then lie in one lane, and the
// forward substitution over the nodes runs there in registers, one thread per channel.
//
// Warp roles of a persistent CTA, each ahead of the next by its buffers:
//     16        copies states in quarters of 16 KB (what keeps HBM busy), 18 the nodes' k, q, g and v,
//               rows of 256 or 512 bytes: no other warp loads them, so none waits for memory
//     4 - 7     split a state into tensor memory
//     8 - 15    prepare a block (all eight, or four each in turn: groups_of): G along the paths, e^G k
//               and e^G q split into the B operand, and A_ij = <e^{G_i - G_j} k_i, k_j>, P_ij =
//               <e^{G_i - G_j} q_i, k_j> on the ancestor pairs alone, each
//               exponential of a difference <= 0 (a factored e^{-G_j} would overflow)
//     17        issues the products (an elected thread at a time; one thread throughout was no faster)
//     0 - 3, 20 - 23   substitution and outputs, a chain of short steps: the first four alone, or
//               in turn with the others (groups_of)
// Bound: the warps' instructions (about 21 K a block of 16 nodes, half of the issue slots) and their supply, with
// the roles' code side by side in one instruction cache; HBM's one read of the state would allow
// two and a half times the speed.  64 x 96 heads: 1 node 115 us, 3.6 TB/s; 8 nodes 149 us; 16 nodes 229 us,
// 2.7 TB/s (fp32 rows 374 us; with the input prologue 314, with the output gate too 366); 96 units of 6 nodes
// 9 us.  Every wait is bounded (Waiter).
#include "kda_draft_launch.h"
#include "kda_draft_sm100.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int D = 128, NB = 16;                     // channels; nodes of a block
constexpr int kPrepThreads = 256, kThreads = 768, kCtas = 152;
// registers a thread: at launch, and after the split (substitution, state, preparation, the rest)
constexpr int kStartRegs = 80, kSolveRegs = 88, kSplitRegs = 88, kPrepRegs = 88, kRestRegs = 40;
static_assert(128 * (2 * kSolveRegs + kSplitRegs + kRestRegs) + kPrepThreads * kPrepRegs <= kThreads * kStartRegs, "register split");
constexpr int kQuarter = 32 * D * 4;                // bytes of a quarter of a state
constexpr int kETile = 4 * NB * D * 4;              // k hi, q hi, k lo, q lo rows of a block
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kColHi = 0, kColLo = 128, kColD = 256;   // D: two buffers of 64 columns
constexpr int kMostStates = 8;

// Buffers and where they lie (bytes from the start of shared memory).
struct Plan {
    int tiles, raws, vals, keys, states;   // B tiles; blocks of g and q, and of v; units of k; state quarters
    int raw, v, k, g, ap, w, state, shared, bytes;
};

struct Shared {
    uint64_t s_full[kMostStates], s_empty[kMostStates], r_full[2], r_empty[2], v_full[4], v_empty[4], k_empty[2], t_full[4], t_empty[4], e_full[2], e_empty[2],
        d_full[2], d_empty[2], a_full[2], a_empty[2];
    alignas(16) unsigned char above[kTreeMaxNodes][kTreeMaxNodes];   // a node's ancestors from the context on, without itself
    signed char count[kTreeMaxNodes];                // how many those are; -1 for an absent node
    TreeSmem tree[4];       // of the two preparations, of the two substitutions
    float kn[2 * kTreeMaxNodes], qn[2 * NB];   // reciprocal norms (input prologue)
    uint32_t tmem;
};

// Units handled side by side by the preparation and by the substitution (trees of one block only).  One
// group's code is fetched by more warps at the same time, two shorten the chain of steps that a
// block is.  With one and with two, 64 x 96 heads: 12 nodes 186 and 205 us, 13 nodes 212 both, 14 nodes 221 and 216,
// 16 nodes 237 and 227; 16 x 96 heads: 8 nodes 55 and 52, 16 nodes 78 and 68.  A CTA with one unit has nothing for the
// second: 96 units of 13 nodes 11.1 and 12.0 us, of 16 nodes 12.8 and 14.3.
__host__ __device__ constexpr int groups_of(int K) { return K > 12 && K <= NB ? 2 : 1; }

__host__ __device__ constexpr Plan plan_of(int K, int esz, int tiles, int raws, int vals, int keys)
{
    Plan p = {};
    p.tiles = tiles;
    p.raws = raws;
    p.vals = vals;
    p.keys = keys;
    int at = tiles * kETile;
    p.raw = at; at += raws * NB * D * (esz + 4);    // of each block g, then q
    p.v = at; at += vals * NB * D * esz;
    p.k = at; at += keys * K * D * esz;
    p.g = at; at += groups_of(K) * K * D * 4;
    p.w = at; at += groups_of(K) * K * D * 4;
    p.ap = at; at += 2 * NB * ((K + 1) & ~1) * 8;   // two blocks' rows of (A, P), rows of 16-byte multiples
    p.shared = (at + 15) & ~15;
    p.state = (p.shared + (int)sizeof(Shared) + 127) & ~127;
    const int fit = (232448 - p.state) / kQuarter;
    p.states = fit > kMostStates ? kMostStates : fit;
    p.bytes = p.state + p.states * kQuarter;
    return p;
}

// A value in two tf32 parts, high and low: the high one rounded to nearest (half away from zero) in two
// integer operations (the conversion instruction runs at a quarter of their rate and would be
// the state split's bound), the low one what is left of it, at most 12 significant bits of which the tensor core
// drops the last: x = hi + lo to 2^-23 of x.  (Rounded once more in place of dropped, that bit
// would count one up instead of one down.)  The addition wraps a NaN around: those of the GPU's own
// arithmetic, 0x7fffffff, become a zero.  What is left of a NaN is a NaN, though, so it stays one in
// the low part, which is therefore not touched again.
__device__ __forceinline__ float tf32_high(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

// A CTA's units: runs of `run` consecutive ones (heads of a sequence, which share its tree), dealt to
// the CTAs in turn, since trees differ in depth and so in work (a contiguous share each: the last CTA
// ended 30 % after the middle one).
struct Units {
    int total, run, count;
    __device__ Units(int units, int run_) : total(units), run(run_), count(0)
    {
        const int runs = (total + run - 1) / run, mine = (runs - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
        if (mine > 0) {
            const int last = ((int)blockIdx.x + (mine - 1) * (int)gridDim.x) * run;   // the only run that can be short
            count = (mine - 1) * run + min(run, total - last);
        }
    }
    __device__ __forceinline__ int operator[](int i) const
    {
        const int k = i / run;
        return ((int)blockIdx.x + k * (int)gridDim.x) * run + i - k * run;
    }
};

// ------------------------------------------------------------------ preparation
// four channels as they lie in shared memory
__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16* p)
{
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// (Loops are unrolled little: the roles run side by side, and straight-line code for each would
// be fetched anew for every block.)
// kPro (all of them): the input prologue is compiled in (own instances; the common ones stay small)
template <typename Tin, bool kPro>
__device__ __forceinline__ void prepare(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t)
{
    const int groups = groups_of(a.nodes), group = t / (kPrepThreads / groups);
    t -= group * (kPrepThreads / groups);
    const int K = a.nodes, H = a.num_heads, KP = (K + 1) & ~1, lane = t & 31, w = t >> 5, W = kPrepThreads / 32 / groups;
    const int bar = 4 + group, threads = 32 * W;
    const int pro = kPro ? a.prologue : 0;
    const bool norm = pro & kProQK;
    float* sg = reinterpret_cast<float*>(base + pl.g) + group * K * D;
    float *kn = sm.kn + group * kTreeMaxNodes, *qn = sm.qn + group * NB;
    TreeSmem& tree = sm.tree[group];
    Waiter wait{a.status};
    uint32_t block = group;                         // (with two groups a unit is one block)
    int tree_of = -1;
    for (uint32_t unit = group; unit < (uint32_t)un.count; unit += groups, block += groups - 1) {
        const int b = un[unit] / H;
        if (b != tree_of) {
            bar_sync(bar, threads);              // the last tree has been read
            if (w == 0) tree_masks(tree, a.parents + (size_t)b * K, K, lane);
            tree_of = b;
        }
        const Tin* sk = reinterpret_cast<const Tin*>(base + pl.k) + (unit % pl.keys) * K * D;
        // a row's four channels of this lane, normalised where the prologue says so
        auto row4 = [&](const Tin* p, float inv) {
            float4 x = four(p + 4 * lane);
            if (norm) x = make_float4(l2_scale(x.x, inv, Tin{}), l2_scale(x.y, inv, Tin{}), l2_scale(x.z, inv, Tin{}), l2_scale(x.w, inv, Tin{}));
            return x;
        };
        for (int i0 = 0; i0 < K; i0 += NB, ++block) {
            const int n = min(NB, K - i0), eb = block % pl.tiles, ab = block & 1, rb = block % pl.raws;
            const float* graw = reinterpret_cast<const float*>(base + pl.raw + rb * NB * D * ((int)sizeof(Tin) + 4));
            const Tin* sq = reinterpret_cast<const Tin*>(graw + NB * D);
            wait(&sm.r_full[rb], (block / pl.raws) & 1);
            bar_sync(bar, threads);              // the last block's G has been read; the tree is there
            if (norm) {
                for (int i = w; i < 2 * n; i += W) {
                    const float4 v = four((i & 1 ? sq + (i >> 1) * D : sk + (i0 + (i >> 1)) * D) + 4 * lane);
                    float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (lane == 0) (i & 1 ? qn[i >> 1] : kn[i0 + (i >> 1)]) = l2_inv(ss);
                }
            }
            // G in powers of two: the g of the path's nodes in this block and the G of the node before
            // them; 16 threads to a node, all nodes at once
            for (int i = t >> 4; i < n; i += threads / 16) {
                const uint64_t path = tree.anc[i0 + i], before = path & ((1ull << i0) - 1);
                const float4* g4 = reinterpret_cast<const float4*>(graw) + (t & 15);
                float4* out = reinterpret_cast<float4*>(sg) + (t & 15);
#pragma unroll
                for (int c = 0; c < D / 4; c += 16) {
                    float4 x = before ? out[(63 - __clzll((long long)before)) * (D / 4) + c] : make_float4(0.f, 0.f, 0.f, 0.f);
                    for (uint32_t in = (uint32_t)(path >> i0) & 0xffffu; in; in &= in - 1) {
                        const float4 y = g4[(__ffs(in) - 1) * (D / 4) + c];
                        x = make_float4(fmaf(path_g(y.x, pro), kLog2e, x.x), fmaf(path_g(y.y, pro), kLog2e, x.y),
                                        fmaf(path_g(y.z, pro), kLog2e, x.z), fmaf(path_g(y.w, pro), kLog2e, x.w));
                    }
                    out[(i0 + i) * (D / 4) + c] = x;
                }
            }
            bar_sync(bar, threads);
            // the B operand: a warp to a node's row, a lane to four channels (16 bytes of each of its four rows,
            // 16 rows apart: the swizzle, which goes by the row's last three bits, is theirs in common)
            if (block >= (uint32_t)pl.tiles) wait(&sm.e_empty[eb], (block / pl.tiles - 1) & 1);
            uint8_t* et = base + eb * kETile + (lane >> 3) * (4 * NB * 128);
#pragma unroll 1
            for (int i = w; i < n; i += W) {        // (rows of the block beyond its nodes: columns of D that nobody reads)
                const float4 g = four(sg + (i0 + i) * D + 4 * lane), k = row4(sk + (i0 + i) * D, norm ? kn[i0 + i] : 1.f),
                             q = row4(sq + i * D, norm ? qn[i] : 1.f);
                const float e[4] = {ex2(g.x), ex2(g.y), ex2(g.z), ex2(g.w)}, kk[4] = {k.x, k.y, k.z, k.w}, qq[4] = {q.x, q.y, q.z, q.w};
                float kh[4], kl[4], qh[4], ql[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float kx = kk[s] * e[s], qx = qq[s] * e[s];
                    kh[s] = tf32_high(kx);
                    kl[s] = kx - kh[s];
                    qh[s] = tf32_high(qx);
                    ql[s] = qx - qh[s];
                }
                float4* at = reinterpret_cast<float4*>(et + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
                at[0] = make_float4(kh[0], kh[1], kh[2], kh[3]);
                at[NB * 8] = make_float4(qh[0], qh[1], qh[2], qh[3]);
                at[2 * NB * 8] = make_float4(kl[0], kl[1], kl[2], kl[3]);
                at[3 * NB * 8] = make_float4(ql[0], ql[1], ql[2], ql[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.e_full[eb]);
            // the ancestor pairs: a warp to a node, eight lanes to an ancestor, four ancestors at a time (lane
            // l of the eight has channels 4 l + 32 s); entry e of the node's list is its e-th ancestor from the
            // context on, the last is the node itself
            if (block >= 2) wait(&sm.a_empty[ab], (block / 2 - 1) & 1);
            __syncwarp();
            float2* ap = reinterpret_cast<float2*>(base + pl.ap) + ab * NB * KP;
            const int c0 = 4 * (lane & 7), which = lane >> 3;
            auto at4 = [&](const Tin* p, float inv) {
                float4 x = four(p);
                if (norm) x = make_float4(l2_scale(x.x, inv, Tin{}), l2_scale(x.y, inv, Tin{}), l2_scale(x.z, inv, Tin{}), l2_scale(x.w, inv, Tin{}));
                return x;
            };
#pragma unroll 1
            for (int i = w; i < n; i += W) {
                const uint64_t all = tree.ok ? tree.anc[i0 + i] : 0ull;
                const int cnt = __popcll(all);
                uint64_t m = all;                   // from this lane's next ancestor on
                for (int k = 0; k < which; ++k) m &= m - 1;
#pragma unroll 1
                for (int e = which; e - which < cnt; e += 4) {
                    const int j = m ? __ffsll((long long)m) - 1 : i0 + i;
                    float da = 0.f, dp = 0.f;
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int c = c0 + 32 * s;
                        const float4 gi = four(sg + (i0 + i) * D + c), gj = four(sg + j * D + c), kj = at4(sk + j * D + c, norm ? kn[j] : 1.f),
                                     ki = at4(sk + (i0 + i) * D + c, norm ? kn[i0 + i] : 1.f), qi = at4(sq + i * D + c, norm ? qn[i] : 1.f);
                        const float x = ex2(gi.x - gj.x) * kj.x, y = ex2(gi.y - gj.y) * kj.y, z = ex2(gi.z - gj.z) * kj.z, v = ex2(gi.w - gj.w) * kj.w;
                        da = fmaf(x, ki.x, fmaf(y, ki.y, fmaf(z, ki.z, fmaf(v, ki.w, da))));
                        dp = fmaf(x, qi.x, fmaf(y, qi.y, fmaf(z, qi.z, fmaf(v, qi.w, dp))));
                    }
                    const bool up = lane & 4;       // both sums over the eight lanes: A in the first four, P in the others
                    float z = up ? dp : da;
                    z += __shfl_xor_sync(0xffffffffu, up ? da : dp, 4);
                    z += __shfl_xor_sync(0xffffffffu, z, 2);
                    z += __shfl_xor_sync(0xffffffffu, z, 1);
                    if ((lane & 3) == 0 && e < cnt) reinterpret_cast<float*>(ap + i * KP + e)[up ? 1 : 0] = z;
                    m &= m - 1;
                    m &= m - 1;
                    m &= m - 1;
                    m &= m - 1;
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.a_full[ab]);
                mbar_arrive(&sm.r_empty[rb]);
                if (i0 + NB >= K) mbar_arrive(&sm.k_empty[unit % pl.keys]);
            }
        }
    }
    wait.finish();
}

// ------------------------------------------------------------------ the state into tensor memory
__device__ __forceinline__ void split(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t)
{
    const int lane = t & 31, dv = t;                // lane of tensor memory = value channel
    const uint32_t quad = 32 * (t >> 5);
    Waiter wait{a.status};
    uint32_t s = 0, phase = 0;
    for (uint32_t unit = 0; unit < (uint32_t)un.count; ++unit) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            wait(&sm.s_full[s], phase);
            if (unit) {
                wait(&sm.t_empty[k], (unit - 1) & 1);
                tc_fence_after_sync();
            }
            __syncwarp();
            const float* src = reinterpret_cast<const float*>(base + pl.state + s * kQuarter) + dv;
#pragma unroll
            for (int c = 0; c < 32; c += 16) {      // (16 at a time: the second's loads go out under the first's arithmetic)
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = src[(c + i) * D], h = tf32_high(x);
                    hi[i] = __float_as_uint(h);
                    lo[i] = __float_as_uint(x - h);
                }
                tmem_st16u(tmem_addr(sm.tmem, quad, kColHi + 32 * k + c), hi);
                tmem_st16u(tmem_addr(sm.tmem, quad, kColLo + 32 * k + c), lo);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.s_empty[s]);
                mbar_arrive(&sm.t_full[k]);
            }
            if (++s == (uint32_t)pl.states) { s = 0; phase ^= 1; }
        }
    }
    wait.finish();
}

// ------------------------------------------------------------------ the products
__device__ __forceinline__ void multiply(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base)
{
    Waiter wait{a.status};
    const uint32_t tm = sm.tmem, tiles = smem_u32(base);
    uint32_t block = 0;
    for (uint32_t unit = 0; unit < (uint32_t)un.count; ++unit) {
        for (int i0 = 0; i0 < a.nodes; i0 += NB, ++block) {
            const uint32_t eb = block % pl.tiles, db = block & 1;
            const bool last = i0 + NB >= a.nodes;
            wait(&sm.e_full[eb], (block / pl.tiles) & 1);
            if (block >= 2) wait(&sm.d_empty[db], (block / 2 - 1) & 1);
            const uint64_t ed = kmajor_base(tiles + eb * kETile);
            const uint32_t d = tm + kColD + 64 * db;
            // quarter by quarter of the key channels, so that the next state's split follows close behind
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                if (i0 == 0) wait(&sm.t_full[k], unit & 1);
                tc_fence_after_sync();
                if (elect_one()) {
                    if (wait.alive) {
                        const uint64_t e = desc_off(ed, k * kmajor_off(4 * NB, 4));
                        const uint32_t hi = tm + kColHi + 32 * k;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_tf32_tmem_a(d, hi + 8 * ks, desc_off(e, 32 * ks), idesc_tf32_f32(128, 4 * NB), k > 0 || ks > 0);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_tf32_tmem_a(d, hi + (kColLo - kColHi) + 8 * ks, desc_off(e, 32 * ks), idesc_tf32_f32(128, 2 * NB), 1);
                    }
                    if (last) umma_commit(&sm.t_empty[k]);
                    if (k == 3) {
                        umma_commit(&sm.e_empty[eb]);
                        umma_commit(&sm.d_full[db]);
                    }
                }
                __syncwarp();
            }
        }
    }
    if (block) wait(&sm.d_full[(block - 1) & 1], ((block - 1) / 2) & 1);    // no product or commit is in flight after this
    wait.finish();
}

// ------------------------------------------------------------------ substitution and outputs
template <typename Tin, bool kPro>
__device__ __forceinline__ void solve(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int t, int group)
{
    const int K = a.nodes, H = a.num_heads, KP = (K + 1) & ~1, lane = t & 31;
    const int groups = groups_of(K), blocks = (K + NB - 1) / NB;
    if (group >= groups) return;
    const uint32_t quad = 32 * (t >> 5);
    float* sw = reinterpret_cast<float*>(base + pl.w) + group * K * D + t;   // this channel's writes
    TreeSmem& tree = sm.tree[2 + group];
    unsigned char (*above)[kTreeMaxNodes] = sm.above + group * (kTreeMaxNodes / 2);
    signed char* count = sm.count + group * (kTreeMaxNodes / 2);
    Waiter wait{a.status};
    uint32_t block = group * blocks;
    int tree_of = -1;
    constexpr int Q = 4;                                        // nodes at a time
    const size_t step = (size_t)H * D;                          // from node to node of out, writes and the gate
    // beta of node (lane % 16) of a block, loaded a block ahead (past the last node the last one again)
    auto beta_at = [&](int unit, int i0) {
        const int u = un[min(unit, un.count - 1)], b = u / H, h = u - b * H;
        return a.beta[((size_t)b * K + min(i0 + (lane & 15), K - 1)) * H + h];
    };
    float next_beta = beta_at(group, 0);
    for (int unit = group; unit < un.count; unit += groups, block += (groups - 1) * blocks) {
        const int u = un[unit], b = u / H, h = u - b * H;
        if (b != tree_of) {
            bar_sync(2 + group, 128);
            if (t < 32) {
                tree_masks(tree, a.parents + (size_t)b * K, K, lane);
                if (lane == 0 && !tree.ok) report_status(a.status, kDevBadSeqlens);
            }
            tree_of = b;
            bar_sync(2 + group, 128);
            if (t < K) {
                int e = 0;
                for (uint64_t m = tree.anc[t] & ~(1ull << t); m; m &= m - 1) above[t][e++] = (unsigned char)(__ffsll((long long)m) - 1);
                count[t] = tree.anc[t] ? (signed char)e : (signed char)-1;
            }
            bar_sync(2 + group, 128);
        }
        size_t at = ((size_t)b * K * H + h) * D + t;
        for (int i0 = 0; i0 < K; i0 += NB, ++block) {
            const uint32_t db = block & 1, vb = block % pl.vals;
            const float beta16 = beta_of(next_beta, kPro ? a.prologue : 0);
            next_beta = i0 + NB < K ? beta_at(unit, i0 + NB) : beta_at(unit + groups, 0);
            const Tin* sv = reinterpret_cast<const Tin*>(base + pl.v) + vb * NB * D + t;
            wait(&sm.v_full[vb], (block / pl.vals) & 1);
            wait(&sm.d_full[db], (block / 2) & 1);
            wait(&sm.a_full[db], (block / 2) & 1);
            __syncwarp();
            tc_fence_after_sync();
            const uint32_t td = tmem_addr(sm.tmem, quad, kColD + 64 * db);
            const float2* row = reinterpret_cast<const float2*>(base + pl.ap) + db * NB * KP;
            const int n = min(NB, K - i0);
#pragma unroll 1
            for (int g0 = 0; g0 < n; g0 += Q) {
                float x[Q], y[Q], x2[Q], y2[Q];                 // X and Y, and their parts from the low half of E
                tmem_ld4(td + g0, x);
                tmem_ld4(td + NB + g0, y);
                tmem_ld4(td + 2 * NB + g0, x2);
                tmem_ld4(td + 3 * NB + g0, y2);
                // what the four nodes need besides one another's writes, before the first of them: v, beta,
                // the number of ancestors (-1: an absent node), the first four with their pairs, the own pair
                float v[Q], beta[Q], own[Q];
                int cnt[Q];
                uint32_t js[Q];
                float4 c0[Q], c1[Q];
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int i = min(g0 + k, n - 1);
                    const float2* r = row + i * KP;
                    v[k] = to_f32(sv[i * D]);
                    beta[k] = __shfl_sync(0xffffffffu, beta16, g0 + k);
                    cnt[k] = count[i0 + i];
                    js[k] = *reinterpret_cast<const uint32_t*>(above[i0 + i]) & 0x3f3f3f3fu;
                    c0[k] = *reinterpret_cast<const float4*>(r);
                    c1[k] = *reinterpret_cast<const float4*>(r + 2);
                    own[k] = r[max(cnt[k], 0)].y;
                }
                tmem_wait_ld();
                if (!tree.ok) continue;
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int i = g0 + k;
                    if (i >= n) break;
                    float xi = x[k] + x2[k], yi = y[k] + y2[k];
                    if (cnt[k] > 0) {
                        const float w0 = sw[(js[k] & 63) * D];
                        xi = fmaf(c0[k].x, w0, xi);
                        yi = fmaf(c0[k].y, w0, yi);
                    }
                    if (cnt[k] > 1) {
                        const float w1 = sw[(js[k] >> 8 & 63) * D];
                        xi = fmaf(c0[k].z, w1, xi);
                        yi = fmaf(c0[k].w, w1, yi);
                    }
                    if (cnt[k] > 2) {
                        const float w2 = sw[(js[k] >> 16 & 63) * D];
                        xi = fmaf(c1[k].x, w2, xi);
                        yi = fmaf(c1[k].y, w2, yi);
                    }
                    if (cnt[k] > 3) {
                        const float w3 = sw[(js[k] >> 24) * D];
                        xi = fmaf(c1[k].z, w3, xi);
                        yi = fmaf(c1[k].w, w3, yi);
                    }
#pragma unroll 1
                    for (int e = 4; e < cnt[k]; e += 2) {       // deeper nodes
                        const uint32_t j = *reinterpret_cast<const uint16_t*>(&above[i0 + i][e]);
                        const float4 c = *reinterpret_cast<const float4*>(row + i * KP + e);
                        const float w0 = sw[(j & 63) * D], w1 = e + 1 < cnt[k] ? sw[(j >> 8 & 63) * D] : 0.f;
                        xi = fmaf(c.x, w0, xi);
                        yi = fmaf(c.y, w0, yi);
                        if (e + 1 < cnt[k]) {
                            xi = fmaf(c.z, w1, xi);
                            yi = fmaf(c.w, w1, yi);
                        }
                    }
                    float wi = beta[k] * (v[k] - xi);
                    yi = fmaf(own[k], wi, yi);
                    if (a.gate) yi = gate1(yi, __ldg(a.gate + at));
                    if (cnt[k] < 0) wi = yi = 0.f;              // an absent node, whatever its rows hold (its gate too)
                    sw[(i0 + i) * D] = wi;
                    a.writes[at] = wi;
                    a.out[at] = yi;
                    at += step;
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.d_empty[db]);
                mbar_arrive(&sm.a_empty[db]);
                mbar_arrive(&sm.v_empty[vb]);
            }
        }
    }
    wait.finish();
}

// ------------------------------------------------------------------ copies
// the states, by one thread
__device__ __forceinline__ void copy_states(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base)
{
    Waiter wait{a.status};
    const char* src = reinterpret_cast<const char*>(a.state);
    const uint32_t total = 4 * un.count;
    uint32_t i = 0;
    for (; i < total; ++i) {
        const uint32_t s = i % pl.states;
        if (i >= (uint32_t)pl.states) wait(&sm.s_empty[s], (i / pl.states - 1) & 1);
        if (!wait.alive) break;
        mbar_arrive_expect_tx(&sm.s_full[s], kQuarter);
        bulk_load(base + pl.state + s * kQuarter, src + ((size_t)un[i / 4] * 4 + i % 4) * kQuarter, kQuarter, &sm.s_full[s]);
    }
    // no load is in flight when the block ends, whatever became of its reader
    for (uint32_t j = i > (uint32_t)pl.states ? i - pl.states : 0; j < i; ++j)
        mbar_wait_bounded(&sm.s_full[j % pl.states], (j / pl.states) & 1, kDraftWaitNs);
    wait.finish();
}

// a block's rows of k (into its unit's buffer), g, q and v, by one warp, a lane to a row
template <typename Tin>
__device__ __forceinline__ void copy_nodes(const TreeDecodeArgs& a, const Plan& pl, Units un, Shared& sm, uint8_t* base, int lane)
{
    constexpr int E = (int)sizeof(Tin), kRow = D * E;
    const int K = a.nodes, H = a.num_heads;
    Waiter wait{a.status};
    uint32_t block = 0, unit = 0;
    bool go = true;
    for (; unit < (uint32_t)un.count && go; ++unit) {
        const int u = un[unit], b = u / H, h = u - b * H;
        const uint32_t kb = unit % pl.keys;
        if (unit >= (uint32_t)pl.keys) wait(&sm.k_empty[kb], (unit / pl.keys - 1) & 1);
        for (int i0 = 0; i0 < K && go; i0 += NB) {
            const int n = min(NB, K - i0);
            const uint32_t rb = block % pl.raws, vb = block % pl.vals;
            if (block >= (uint32_t)pl.raws) wait(&sm.r_empty[rb], (block / pl.raws - 1) & 1);
            if (block >= (uint32_t)pl.vals) wait(&sm.v_empty[vb], (block / pl.vals - 1) & 1);
            go = __all_sync(0xffffffffu, wait.alive);
            if (!go) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.r_full[rb], n * (2 * kRow + D * 4));
                mbar_arrive_expect_tx(&sm.v_full[vb], n * kRow);
            }
            __syncwarp();
            uint8_t* raw = base + pl.raw + rb * NB * D * (E + 4);
            for (int x = lane; x < 64; x += 32) {
                const int i = x & 15, what = x >> 4;
                if (i >= n) continue;
                const size_t at = (((size_t)b * K + i0 + i) * H + h) * D;
                if (what == 0) bulk_load(raw + i * D * 4, a.g + at, D * 4, &sm.r_full[rb]);
                else if (what == 1) bulk_load(raw + NB * D * 4 + i * kRow, static_cast<const Tin*>(a.q) + at, kRow, &sm.r_full[rb]);
                else if (what == 2) bulk_load(base + pl.k + (kb * K + i0 + i) * kRow, static_cast<const Tin*>(a.k) + at, kRow, &sm.r_full[rb]);
                else bulk_load(base + pl.v + (vb * NB + i) * kRow, static_cast<const Tin*>(a.v) + at, kRow, &sm.v_full[vb]);
            }
            ++block;
        }
    }
    for (uint32_t j = block > (uint32_t)pl.raws ? block - pl.raws : 0; j < block; ++j)
        mbar_wait_bounded(&sm.r_full[j % pl.raws], (j / pl.raws) & 1, kDraftWaitNs);
    for (uint32_t j = block > (uint32_t)pl.vals ? block - pl.vals : 0; j < block; ++j)
        mbar_wait_bounded(&sm.v_full[j % pl.vals], (j / pl.vals) & 1, kDraftWaitNs);
    wait.finish();
}

template <typename Tin, bool kPro>
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
        for (int i = 0; i < kMostStates; ++i) { mbar_init(&sm.s_full[i], 1); mbar_init(&sm.s_empty[i], 4); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.e_full[i], kPrepThreads / groups_of(a.nodes));
            mbar_init(&sm.e_empty[i], 1);
            mbar_init(&sm.d_full[i], 1);
            mbar_init(&sm.d_empty[i], 4);
            mbar_init(&sm.a_full[i], kPrepThreads / 32 / groups_of(a.nodes));
            mbar_init(&sm.a_empty[i], 4);
            mbar_init(&sm.r_full[i], 1);
            mbar_init(&sm.r_empty[i], kPrepThreads / 32 / groups_of(a.nodes));
            mbar_init(&sm.k_empty[i], kPrepThreads / 32 / groups_of(a.nodes));
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.t_full[i], 4);
            mbar_init(&sm.t_empty[i], 1);
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_empty[i], 4);
        }
        mbar_fence_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // (In runs of one unit and of four, 16 nodes: 64 x 96 heads 230 and 223 us, 51 x 96 187 both, 32 x 96 121 and 130,
    // 16 x 96 66 and 73; one node: 64 x 96 157 and 108, 16 x 96 41 and 35.  The rule goes by the deep trees.)
    const Units un(total, total >= 32 * (int)gridDim.x ? 4 : 1);
    if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSolveRegs));
        solve<Tin, kPro>(a, pl, un, sm, base, t, 0);
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSplitRegs));
        split(a, pl, un, sm, base, t - 128);
    } else if (warp < 16) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrepRegs));
        prepare<Tin, kPro>(a, pl, un, sm, base, t - 256);
    } else if (warp >= 20) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSolveRegs));
        solve<Tin, kPro>(a, pl, un, sm, base, t - 640, 1);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
        if (warp == 17) multiply(a, pl, un, sm, base);
        if (warp == 16 && elect_one()) copy_states(a, pl, un, sm, base);
        if (warp == 18) copy_nodes<Tin>(a, pl, un, sm, base, t & 31);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 17) tmem_dealloc(sm.tmem, 512);
}

// Buffers for K nodes: as much in double (v, which waits for the last of the roles, in fourfold: 154 us
// for 64 x 96 heads x 8 nodes when it was taken, 208 with two of v and one unit's k) as leaves the states three
// quarters or more (48 KB in flight cover HBM's latency).
constexpr Plan choose_plan(int K, int esz)
{
    constexpr int options[6][5] = {{2, 2, 4, 2, 4}, {2, 2, 4, 2, 3}, {2, 2, 2, 1, 3}, {1, 2, 2, 2, 3}, {1, 2, 2, 1, 3}, {1, 1, 1, 1, 3}};
    for (const auto& o : options) {
        const Plan p = plan_of(K, esz, o[0], o[1], o[2], o[3]);
        if (p.states >= o[4]) return p;
    }
    return {};
}
// Two groups take their units in turn, and a wait by parity can be one phase ahead at most: each
// group needs slots of its own in the rings it waits on (k comes with g and q).
constexpr bool plan_ok(int K, int esz)
{
    const Plan p = choose_plan(K, esz);
    const int g = groups_of(K);
    return p.bytes > 0 && p.tiles % g == 0 && p.raws % g == 0 && p.vals % g == 0;
}
constexpr bool all_fit()
{
    for (int K = 1; K <= kTreeMaxNodes; ++K)
        if (!plan_ok(K, 2) || !plan_ok(K, 4)) return false;
    return true;
}
static_assert(all_fit(), "every tree has a plan");

template <typename Tin, bool kPro>
cudaError_t launch(const TreeDecodeArgs& a, cudaStream_t stream)
{
    const Plan p = choose_plan(a.nodes, (int)sizeof(Tin));
    static KernelSetup setup;
    const cudaError_t e = setup(tree_decode_tc_kernel<Tin, kPro>, 232448, kStartRegs);   // (the split needs its start)
    if (e != cudaSuccess) return e;
    const int total = a.batch * a.num_heads;
    tree_decode_tc_kernel<Tin, kPro><<<total < kCtas ? total : kCtas, kThreads, p.bytes, stream>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_decode_tc(const TreeDecodeArgs& a, cudaStream_t stream)
{
    if (a.prologue) return a.bf16 ? launch<__nv_bfloat16, true>(a, stream) : launch<float, true>(a, stream);
    return a.bf16 ? launch<__nv_bfloat16, false>(a, stream) : launch<float, false>(a, stream);
}

}  // namespace kda
