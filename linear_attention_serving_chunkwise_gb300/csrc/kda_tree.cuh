// The draft tree of one sequence, shared by the draft-step kernels: parents[i] = -1 hangs
// node i on the context, 0 <= parents[i] < i on an earlier node, -2 marks an absent node.
#pragma once

#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

constexpr int kTreeMaxNodes = 64;   // KDA_TREE_MAX_NODES: one bit of a 64-bit mask per node
constexpr int kTreePad = -2;        // KDA_TREE_PAD

// g as the tree kernels sum it along a path.  e^g is zero in fp32 below -104, and a g of -inf (the state is
// forgotten there) would make differences of later sums inf - inf.  So g counts as -105 at least: G
// stays finite, and e^{G_i - G_j} is zero where such a node lies between the two and untouched by
// it elsewhere, but for G's rounding (2^-25 of |G|, which each such node makes 105 larger).
// A NaN stays one.  With the prologue g is -5 or more.
constexpr float kGLeast = -105.f;
__device__ __forceinline__ float path_g(float g, int prologue)
{
    if (prologue & kProG) return g_of(g, prologue);
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(g), "f"(kGLeast));
    return y;
}

struct TreeSmem {
    uint64_t anc[kTreeMaxNodes];    // bit j of anc[i]: node j is node i or above it; 0 for an absent node
    int up[kTreeMaxNodes];
    int ok;
};

// One warp builds the ancestor masks by pointer doubling: after round r a node's mask holds
// its 2^r nearest ancestors and `up` is the next one beyond them, so K nodes take
// ceil(log2 K) rounds whatever the tree's shape (a chain of 64 walked node by node would be
// 64 dependent loads).  ts.ok becomes 0 for a tree that breaks the rules above.
// The caller synchronises before other warps read ts.
__device__ __forceinline__ void tree_masks(TreeSmem& ts, const int32_t* parents, int K, int lane)
{
    bool bad = false;
    for (int i = lane; i < K; i += 32) {
        const int p = parents[i];
        bad |= p < kTreePad || p >= i;
        ts.anc[i] = p == kTreePad ? 0ull : 1ull << i;
        ts.up[i] = p;
    }
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    if (!bad) {
        for (int i = lane; i < K; i += 32) bad |= ts.up[i] >= 0 && ts.up[ts.up[i]] == kTreePad;   // hangs on an absent node
        bad = __any_sync(0xffffffffu, bad);
    }
    if (!bad) {
        for (int span = 1; span < K; span <<= 1) {
            uint64_t m[2];
            int u[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int i = lane + 32 * s;
                if (i < K) {
                    const int p = ts.up[i];
                    m[s] = ts.anc[i] | (p >= 0 ? ts.anc[p] : 0ull);
                    u[s] = p >= 0 ? ts.up[p] : p;
                }
            }
            __syncwarp();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int i = lane + 32 * s;
                if (i < K) { ts.anc[i] = m[s]; ts.up[i] = u[s]; }
            }
            __syncwarp();
        }
    }
    if (lane == 0) ts.ok = bad ? 0 : 1;
    __syncwarp();
}

}  // namespace kda
