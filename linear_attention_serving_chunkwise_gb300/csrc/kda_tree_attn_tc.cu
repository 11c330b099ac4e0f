// Attention of draft trees over a paged bf16 cache on the Blackwell tensor cores (tcgen05).
// The mathematics, the cut of the work and the join are those of kda_tree_attn.cuh: one pass
// over the tokens, running maximum and sum per row, parts of split units joined afterwards.
//
// The query rows of a (sequence, cache head) -- K nodes x G heads -- fill the 128 lanes of an
// accumulator: S = Q K^T per tile of 128 tokens, the weights overwrite S in tensor memory as
// the bf16 A operand of O += P V, and O stays in tensor memory for the whole piece.  Two
// streams of S and O share the tensor core, so that one stream's softmax runs under the
// other's products:
//     up to 128 rows   the streams take the tiles in turn over the same rows, and their two
//                      parts are joined in the epilogue;
//     more             they take 128 rows each of a 256-row unit, and every tile serves both.
// O is multiplied only when a row's maximum has grown by more than 2^8 since the last time
// (until then the weights are at most 2^8, which bf16 and the fp32 sums hold as well).
//
// Warps 0-3 and 4-7: softmax and epilogue of stream 0 and 1, a row to a thread.  Warps 8-11:
// the cache rows, gathered page by page with 16-byte asynchronous copies into a ring of K
// and V tiles (any page size: the copies need no box).  Warp 12 issues the products, warp 13 copies Q.
// Every wait is bounded; a thread that gave up goes through the rest of its schedule without
// waiting and without touching the tensor core, and the status word says so.
//
// What no row may see: scores are masked per row; rows past the last token or on a page out
// of range are zero in shared memory.  A draft node's values may be seen by some rows only, so
// non-finite ones are replaced by zero in the tile and added back in the epilogue of the
// rows that see the node (a positive weight times infinity or NaN is itself).
#include "kda_sm100.cuh"
#include "kda_tree_attn.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kBN = 128;
constexpr int kSoftmaxThreads = 256, kProducerThreads = 128, kThreads = kSoftmaxThreads + kProducerThreads + 64;
constexpr int kCtas = 152;                          // one to an SM
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;                        // powers of two a maximum may grow before O is multiplied

struct Shared {
    uint64_t kv_full[10], kv_empty[10], s_full[2], p_full[2], q_full, q_empty, o_done, o_free;
    uint64_t bad_nodes[8];                          // by piece: nodes with non-finite values
    uint32_t missing[8][4];                         // by tile: its tokens without a page (a V tile is freed after its softmax, so the
                                                    // copies are never more than 6 tiles past the one the softmax is at)
    TreeSmem tree;
    uint32_t tmem;
};

template <int D, bool kWide>
struct Layout {
    static constexpr int kTile = kBN * D * 2;                   // bytes of a K or V tile, and of 128 rows of Q
    static constexpr int kQ = kTile * (kWide ? 2 : 1);
    static constexpr int kSlots = D == 128 ? 5 : 10;            // ring: K and V tiles in turn
    static constexpr int kLag = kSlots - 2;                     // copies in flight before the oldest is waited for
    static constexpr int kStats = kQ + kSlots * kTile;          // both streams' maxima and sums (streams in turn)
    static constexpr int kShared = kStats + (kWide ? 0 : 2 * 2 * 128 * 4);
    static constexpr int kBytes = kShared + (int)sizeof(Shared);
    static constexpr uint32_t kColS = 0, kColO = 256;           // stream w: S at 128 w, O at 256 + D w
    static_assert(kBytes <= 232448, "shared memory");
};

struct Waiter {
    int* status;
    bool alive = true;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity)
    {
        if (!alive) return;
        if (mbar_try_wait(bar, parity)) return;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_sleep(bar, parity, 1000)) {
            if (globaltimer_ns() - t0 > kWaitNs) {
                alive = false;
                report_status(status, kDevTimeout);
                return;
            }
        }
    }
};

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there)
{
    const int n = there ? 16 : 0;                   // 0: the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7f80u) != 0x7f80u; }

// ------------------------------------------------------------------ the cache rows
template <int D, bool kWide>
__device__ __forceinline__ void produce(const TreeAttnArgs& a, const attn::Shape& sh, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    constexpr int CH = D / 8;                       // 16-byte chunks of a row
    constexpr int RPI = 32 / CH;                    // rows a warp copies at once
    const int lane = t & 31, w = t >> 5;
    // (a cache without pages may be a null pointer: copies of no bytes then start at q)
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.k_cache : a.q);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.v_cache : a.q);
    const size_t row_stride = (size_t)a.kv_heads * D;
    Waiter wait{a.status};
    attn::Line line;
    line.begin(a, sh, blockIdx.x, lane);
    attn::Piece pc;
    uint32_t fill = 0, sent = 0;                    // ring slots begun, and handed over
    bool bad_page = false;
    const int sub = lane / CH, chunk = lane % CH;

    auto hand_over = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&sm.kv_full[sent % L::kSlots]);
        ++sent;
    };
    // one slot's copies are issued: hand over the one kLag before it
    auto filled = [&]() {
        cp_commit();
        ++fill;
        if (fill - sent > L::kLag) {
            cp_wait<L::kLag>();
            hand_over();
        }
    };

    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        const int32_t* table = a.block_table + (size_t)pc.b * a.table_cols;
        // lane l of warp w looks up token 32 w + l of a tile, one tile ahead
        auto look_up = [&](int tile) {
            const int pos = tile * kBN + 32 * w + lane;
            return tile < pc.last && pos < pc.n ? __ldg(table + pos / a.page_size) : -1;
        };
        int id = look_up(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile) {
            const int t0 = tile * kBN, pos = t0 + 32 * w + lane;
            const bool there = id >= 0 && id < a.num_pages;
            const unsigned lost = __ballot_sync(0xffffffffu, !there && pos < pc.n);
            bad_page |= lost != 0;
            const size_t in_page = (size_t)(pos % a.page_size) * row_stride + (size_t)pc.hk * D;
            const size_t koff = there ? (size_t)id * a.k_page_stride + in_page : 0;
            const size_t voff = there ? (size_t)id * a.v_page_stride + in_page : 0;
            const unsigned exists = __ballot_sync(0xffffffffu, there);
            id = look_up(tile + 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s = fill % L::kSlots;
                if (fill >= (uint32_t)L::kSlots) wait(&sm.kv_empty[s], (fill / L::kSlots - 1) & 1);
                uint8_t* dst = base + L::kQ + s * L::kTile;
                if (kv == 0 && lane == 0) sm.missing[fill / 2 & 7][w] = lost;
                const __nv_bfloat16* src = kv ? vc : kc;
                const size_t off = kv ? voff : koff;
                if (kv == 1 && t0 + kBN > pc.ctx) {
                    // draft nodes in the tile: their values pass through registers
                    uint32_t bad = 0;               // of this warp's 32 tokens
                    for (int i0 = 0; i0 < 32; i0 += 8 * RPI) {
                        uint4 x[8];                 // eight loads in flight
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = i0 + k * RPI + sub;
                            const size_t o = __shfl_sync(0xffffffffu, off, r);
                            x[k] = make_uint4(0, 0, 0, 0);
                            if (exists >> r & 1) x[k] = *(reinterpret_cast<const uint4*>(src + o) + chunk);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = i0 + k * RPI + sub;
                            if (t0 + 32 * w + r >= pc.ctx) {
                                uint32_t h[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const bool lo = finite_bf16(h[e]), hi = finite_bf16(h[e] >> 16);
                                    if (!(lo && hi)) bad |= 1u << r;
                                    h[e] = (lo ? h[e] & 0xffffu : 0u) | (hi ? h[e] & 0xffff0000u : 0u);
                                }
                                x[k] = make_uint4(h[0], h[1], h[2], h[3]);
                            }
                            *reinterpret_cast<uint4*>(dst + sw128_chunk(32 * w + r, chunk, 128)) = x[k];
                        }
                    }
                    bad = __reduce_or_sync(0xffffffffu, bad);
                    if (bad && lane == 0) {
                        for (int r = 0; r < 32; ++r)
                            if (bad >> r & 1)
                                atomicOr(reinterpret_cast<unsigned long long*>(&sm.bad_nodes[piece & 7]), 1ull << (t0 + 32 * w + r - pc.ctx));
                    }
                } else {
#pragma unroll 4
                    for (int i = 0; i < 32; i += RPI) {
                        const int r = i + sub;
                        const size_t o = __shfl_sync(0xffffffffu, off, r);
                        cp16(smem_u32(dst + sw128_chunk(32 * w + r, chunk, 128)), src + o + 8 * chunk, exists >> r & 1);
                    }
                }
                filled();
            }
        }
    }
    cp_wait<0>();
    while (sent != fill) hand_over();
    if (bad_page && lane == 0) report_status(a.status, kDevBadSeqlens);
}

// ------------------------------------------------------------------ the query rows
// One warp, as soon as the last piece's scores are done: rows past the last are zero, and
// scale 0 is a zero Q (every score is then 0).
template <int D, bool kWide>
__device__ __forceinline__ void query(const TreeAttnArgs& a, const attn::Shape& sh, Shared& sm, uint8_t* base, int lane)
{
    using L = Layout<D, kWide>;
    constexpr int CH = D / 8;
    const int G = a.heads / a.kv_heads, R = a.nodes * G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    Waiter wait{a.status};
    attn::Line line;
    line.begin(a, sh, blockIdx.x, lane);
    attn::Piece pc;
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        if (piece) wait(&sm.q_empty, (piece - 1) & 1);
        for (int idx = lane; idx < sh.BM * CH; idx += 32) {
            const int r = idx / CH, c = idx % CH, row = pc.r0 + r;
            const bool there = row < R && a.scale != 0.f;
            const size_t off = there ? (((size_t)pc.b * a.nodes + row / G) * a.heads + pc.hk * G + row % G) * D + 8 * c : 0;
            cp16(smem_u32(base + (r >> 7) * L::kTile + sw128_chunk(r & 127, c, 128)), q + off, there);
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full);
    }
}

// ------------------------------------------------------------------ the products
template <int D, bool kWide>
__device__ __forceinline__ void multiply(const TreeAttnArgs& a, const attn::Shape& sh, Shared& sm, uint8_t* base, int lane)
{
    using L = Layout<D, kWide>;
    Waiter wait{a.status};
    attn::Line line;
    line.begin(a, sh, blockIdx.x, lane);
    if (lane != 0) return;
    attn::Piece pc;
    const uint32_t tm = sm.tmem, q0 = smem_u32(base), ring = q0 + L::kQ;
    const uint32_t id_s = idesc_bf16_f32(128, kBN, 0, 0, a.scale < 0.f), id_o = idesc_bf16_f32(128, D, 0, 1);
    uint32_t kv = 0, used[2] = {0, 0};              // ring position of the piece's first K tile; items of each stream so far
    uint32_t piece = 0;
    for (; line.next(a, sh, blockIdx.x, pc); ++piece) {
        const int tiles = pc.last - pc.first, items = kWide ? 2 * tiles : tiles;
        wait(&sm.q_full, piece & 1);
        // item i: stream i % 2; its tile is i (streams in turn) or i / 2 (each tile for both)
        auto scores = [&](int i) {
            const int w = i & 1, tile = kWide ? i >> 1 : i;
            const uint32_t at = kv + 2 * tile, s = at % L::kSlots;
            if (!kWide || w == 0) wait(&sm.kv_full[s], (at / L::kSlots) & 1);
            tc_fence_after_sync();
            if (wait.alive) {
                const uint64_t qd = kmajor_base(q0 + (kWide ? w * L::kTile : 0)), kd = kmajor_base(ring + s * L::kTile);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_bf16(tm + L::kColS + 128 * w, desc_off(qd, kmajor_off(128, ks)), desc_off(kd, kmajor_off(128, ks)), id_s, ks > 0);
            }
            if (!kWide || w == 1) umma_commit(&sm.kv_empty[s]);
            if (i == items - 1) umma_commit(&sm.q_empty);
            umma_commit(&sm.s_full[w]);
        };
        auto values = [&](int i) {
            const int w = i & 1, tile = kWide ? i >> 1 : i;
            const uint32_t at = kv + 2 * tile + 1, s = at % L::kSlots;
            if (!kWide || w == 0) wait(&sm.kv_full[s], (at / L::kSlots) & 1);
            if (i == 0 && piece) wait(&sm.o_free, (piece - 1) & 1);
            wait(&sm.p_full[w], used[w] & 1);
            ++used[w];
            tc_fence_after_sync();
            if (wait.alive) {
                const uint64_t vd = mnmajor_base(ring + s * L::kTile, kBN);
#pragma unroll
                for (int ks = 0; ks < kBN / 16; ++ks)
                    umma_bf16_tmem_a(tm + L::kColO + D * w, tm + L::kColS + 128 * w + 8 * ks, desc_off(vd, mnmajor_off(ks)), id_o, i > 1 || ks > 0);
            }
            if (!kWide || w == 1) umma_commit(&sm.kv_empty[s]);
            if (i == items - 1) umma_commit(&sm.o_done);
        };
        scores(0);
        if (items > 1) scores(1);
        for (int i = 0; i < items; ++i) {
            values(i);
            if (i + 2 < items) scores(i + 2);
        }
        kv += 2 * tiles;
    }
    if (piece) wait(&sm.o_done, (piece - 1) & 1);   // no product or commit is in flight after this
}

// ------------------------------------------------------------------ softmax and epilogue
// What row sees of the tile at t0: 128 bits, four words.
__device__ __forceinline__ void tile_mask(uint64_t see, int t0, int ctx, const uint32_t* missing, uint32_t (&mw)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = t0 + 32 * k - ctx;           // node of the word's first token
        uint32_t x = 0;
        if (see) {
            if (at <= -32) x = 0xffffffffu;
            else if (at < 0) x = ((1u << -at) - 1u) | (uint32_t)(see << -at);
            else if (at < 64) x = (uint32_t)(see >> at);
        }
        mw[k] = x & ~missing[k];
    }
}

template <int D, bool kWide>
__device__ __forceinline__ void softmax(const TreeAttnArgs& a, const attn::Shape& sh, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    float* stats = reinterpret_cast<float*>(base + L::kStats);        // [stream][m, l][128]
    const int lane = t & 31, warp = t >> 5, w = t >> 7, r = t & 127;   // stream and lane of tensor memory
    const int G = a.heads / a.kv_heads, R = a.nodes * G;
    const uint32_t quad = 32 * (warp & 3);                            // the lanes this warp reaches
    const uint32_t tS = tmem_addr(sm.tmem, quad, L::kColS + 128 * w), tO = tmem_addr(sm.tmem, quad, L::kColO);
    const float sc = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;  // scores in powers of two
    Waiter wait{a.status};
    attn::Line line;
    line.begin(a, sh, blockIdx.x, lane);
    attn::Piece pc;
    uint32_t used = 0, done = 0;                    // items of this stream, and tiles, so far
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        const int tiles = pc.last - pc.first;
        bar_sync(1, kSoftmaxThreads);               // everyone is done with the last piece's tree and statistics
        if (warp == 0) tree_masks(sm.tree, a.parents + (size_t)pc.b * a.nodes, a.nodes, lane);
        bar_sync(1, kSoftmaxThreads);
        if (!(pc.seq_ok && sm.tree.ok) && t == 0) report_status(a.status, kDevBadSeqlens);
        const int row = pc.r0 + (kWide ? 128 * w : 0) + r;
        const uint64_t see = pc.seq_ok && sm.tree.ok && row < R ? sm.tree.anc[row / G] : 0ull;
        const bool busy = __any_sync(0xffffffffu, see != 0);
        float m = -INFINITY, l = 0.f;               // m in score units, before sc
        bool begun = false;

        for (int i = kWide ? 0 : w; i < tiles; i += kWide ? 1 : 2) {
            const int t0 = (pc.first + i) * kBN;
            wait(&sm.s_full[w], used & 1);
            ++used;
            __syncwarp();
            tc_fence_after_sync();
            if (busy) {
                uint32_t mw[4];
                const uint32_t* missing = sm.missing[(done + i) & 7];
                const bool all = t0 + kBN <= pc.ctx && !(missing[0] | missing[1] | missing[2] | missing[3]);
                tile_mask(see, t0, pc.ctx, missing, mw);
                auto load = [&](int c, float (&x)[32]) {
                    tmem_ld32(tS + 32 * c, x);
                    tmem_wait_ld();
                    if (!all) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = mw[c] >> k & 1 ? x[k] : -INFINITY;
                    }
                };
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    load(c, x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) top = fmaxf(top, x[k]);
                }
                const bool grow = (top - m) * sc > kGrow;
                if (__any_sync(0xffffffffu, grow)) {
                    const float nm = grow ? top : m;
                    const float f = grow ? ex2((m - nm) * sc) : 1.f;   // 0 for the first maximum
                    l *= f;
                    m = nm;
                    if (begun) {                    // the products of the stream's last tile are done: S is ready
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_ld32(tO + D * w + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= f;
                            tmem_st32(tO + D * w + c, o);
                        }
                    }
                }
                // (x - m) sc in this order: the difference is exact where it matters, however large the scores
                const float2 off = make_float2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m), sc2 = make_float2(sc, sc);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    load(c, x);
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[2 * k], x[2 * k + 1]), off), sc2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = __fadd2_rn(sum, e);
                        p[k] = pack_bf16x2(e.x, e.y);
                    }
                    tmem_st16u(tS + 16 * c, p);
                }
                l += sum.x + sum.y;
                begun = true;
                tmem_wait_st();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[w]);
        }
        done += tiles;

        // epilogue (a row that may see nothing went unmasked through tiles of context)
        if (!see) {
            m = -INFINITY;
            l = 0.f;
        }
        if (!kWide) {
            stats[256 * w + r] = m;
            stats[256 * w + 128 + r] = l;
        }
        wait(&sm.o_done, piece & 1);
        tc_fence_after_sync();
        bar_sync(1, kSoftmaxThreads);
        const uint64_t bad = *const_cast<volatile uint64_t*>(&sm.bad_nodes[piece & 7]) & see;
        // this thread's columns [c0, c1) of the row: stream 1's part is joined when it has one
        const int c0 = kWide ? 0 : w * (D / 2), c1 = kWide ? D : c0 + D / 2;
        const bool two = !kWide && tiles > 1;
        float f0 = 1.f, f1 = 0.f;
        if (!kWide) {
            const float m0 = stats[r], m1 = two ? stats[256 + r] : -INFINITY, l0 = stats[128 + r], l1 = two ? stats[384 + r] : 0.f;
            m = fmaxf(m0, m1);
            f0 = m0 == -INFINITY ? 0.f : ex2((m0 - m) * sc);
            f1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * sc);
            l = (m0 == -INFINITY ? l0 : l0 * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
        }
        const float norm = pc.whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        float* ws = static_cast<float*>(a.workspace) + attn::slot_floats(sh.BM, D) * (size_t)pc.slot;
        const int rl = row - pc.r0;                 // row of the unit
        if (row < R && !pc.whole && c0 == 0) {
            ws[rl] = m == -INFINITY ? m : m * sc;
            ws[sh.BM + rl] = l;
        }
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (((size_t)pc.b * a.nodes + row / G) * a.heads + pc.hk * G + row % G) * D;
        for (int c = c0; c < c1; c += 32) {
            float o[32];
            if (busy) {
                tmem_ld32(tO + (kWide ? D * w : 0) + c, o);
                tmem_wait_ld();
                if (!kWide) {
                    if (two) {
                        float o1[32];
                        tmem_ld32(tO + D + c, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = o[k] * f0 + o1[k] * f1;
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= f0;
                    }
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = l == 0.f ? 0.f : o[k] * norm;
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0.f;
            }
            for (uint64_t left = bad; left; left &= left - 1) {
                const int pos = pc.ctx + __ffsll((long long)left) - 1;
                const int id = a.block_table[(size_t)pc.b * a.table_cols + pos / a.page_size];
                if (id < 0 || id >= a.num_pages) continue;
                const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + (size_t)id * a.v_page_stride +
                                         ((size_t)(pos % a.page_size) * a.kv_heads + pc.hk) * D + c;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float x = __bfloat162float(v[k]);
                    if (!isfinite(x)) o[k] += x;
                }
            }
            if (row < R && pc.whole) {
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                    *reinterpret_cast<uint4*>(dst + c + k) = make_uint4(pack_bf16x2(o[k], o[k + 1]), pack_bf16x2(o[k + 2], o[k + 3]),
                                                                       pack_bf16x2(o[k + 4], o[k + 5]), pack_bf16x2(o[k + 6], o[k + 7]));
            } else if (row < R) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<float4*>(ws + 2 * sh.BM + (size_t)rl * D + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free);
        bar_sync(1, kSoftmaxThreads);
        if (t == 0) sm.bad_nodes[piece & 7] = 0;
    }
}

template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_tc_kernel(TreeAttnArgs a, attn::Shape sh)
{
    using L = Layout<D, kWide>;
    extern __shared__ __align__(1024) uint8_t base[];   // all of it: the swizzled tiles start at 0
    Shared& sm = *reinterpret_cast<Shared*>(base + L::kShared);
    const int t = threadIdx.x, warp = t >> 5;
    if (warp == 12) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (t == 0) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&sm.kv_full[i], kProducerThreads);
            mbar_init(&sm.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
        }
        mbar_init(&sm.q_full, 32);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.o_done, 1);
        mbar_init(&sm.o_free, kSoftmaxThreads / 32);
        for (int i = 0; i < 8; ++i) sm.bad_nodes[i] = 0;
        mbar_fence_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp < 8) softmax<D, kWide>(a, sh, sm, base, t);
    else if (warp < 12) produce<D, kWide>(a, sh, sm, base, t - kSoftmaxThreads);
    else if (warp == 12) multiply<D, kWide>(a, sh, sm, base, t & 31);
    else query<D, kWide>(a, sh, sm, base, t & 31);
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 12) tmem_dealloc(sm.tmem, 512);
}

bool wide_rows(int nodes, int group) { return nodes * group > 128; }

template <int D, bool kWide>
cudaError_t launch(const TreeAttnArgs& a, cudaStream_t stream)
{
    const attn::Shape sh = {kWide ? 256 : 128, kBN, kCtas};
    cudaError_t e = cudaFuncSetAttribute(tree_attn_tc_kernel<D, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D, kWide>::kBytes);
    if (e != cudaSuccess) return e;
    tree_attn_tc_kernel<D, kWide><<<sh.ctas, kThreads, Layout<D, kWide>::kBytes, stream>>>(a, sh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    attn::join_kernel<__nv_bfloat16, D><<<dim3(sh.ctas - 1, (sh.BM + 7) / 8), 256, 0, stream>>>(a, sh);
    return cudaGetLastError();
}

}  // namespace

size_t tree_attn_tc_workspace_bytes(int nodes, int group, int dim)
{
    return attn::slot_floats(wide_rows(nodes, group) ? 256 : 128, dim) * 2 * kCtas * sizeof(float);
}

cudaError_t launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t stream)
{
    const bool wide = wide_rows(a.nodes, a.heads / a.kv_heads);
    if (a.dim == 128) return wide ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
    return wide ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
}

}  // namespace kda
