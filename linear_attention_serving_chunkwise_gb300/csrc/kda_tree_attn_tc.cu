// Attention of draft trees over a paged bf16 cache on the Blackwell tensor cores (tcgen05).
// The mathematics, the cut of the work and the join are those of kda_tree_attn.cuh: one pass
// over the tokens, running maximum and sum per row, parts of split units joined afterwards.
//
// The query rows of a (sequence, cache head) -- K nodes x G heads -- fill the 128 lanes of an
// accumulator: S = Q K^T per tile of 128 tokens, the weights overwrite half of S in tensor
// memory as the bf16 A operand of O += P V, and O stays in tensor memory for the whole piece.  Two
// streams of S and O share the tensor core, so that one stream's softmax runs under the
// other's products:
//     up to 128 rows   the streams take the tiles in turn over the same rows, and their two
//                      parts are joined in the epilogue;
//     more             they take 128 rows each of a 256-row unit, and every tile serves both.
// O is multiplied only when a row's maximum has grown by more than 2^8 since the last time
// (until then the weights are at most 2^8, which bf16 and the fp32 sums hold as well).
//
// Warps 0-3 and 4-7: softmax and epilogue of stream 0 and 1, a row to a thread.  Warps 8-11:
// the cache rows, into a ring of K and V tiles.  A thread of warp 12 issues the products, warps
// 13-15 copy Q.  The last two groups give registers to the softmax.
//
// Bound: HBM's read of the cache for few rows, the tensor pipe (2048 cycles a tile of 256 rows x 128
// tokens, D = 128) and the chain scores - softmax - values of each stream for many; a tile took
// 3000 cycles when 2700 of them were HBM's.  Join included, of a copy's 6.8 TB/s: 2 sequences
// of 131072 tokens, 8 cache heads, 64 rows a head 171 us, 6.3 TB/s; 256 rows 208 us, 5.2 TB/s and
// 1320 TFLOP/s; 32 trees of 16 nodes, 512 to 16384 tokens, 192 rows 223 us, 5.2 TB/s; one node over
// 1500 tokens 18 us, latency (the first tile's way, the join); 128 sequences of 4096 to 32768 tokens, one node, 4 rows
// a head 1396 us, 7.0 TB/s.  D = 64 (half the bytes and products, the same softmax): the 32 trees 181 us, 2 x 131072
// tokens 170 us.  Times of a short loop in a CUDA graph: a long stream of calls runs at the clock of sustained
// load, 230 us for 2 x 131072 and 244 for the 32 trees (1196 and 894 TFLOP/s).
//
// The cache rows come by TMA where the page size is a multiple of 8: a tile is a stack of boxes
// of 8 to 128 rows (the largest power of two in the page size), and 8 rows are one swizzle
// atom, so boxes of any pages stack into the tile the products read.  Other page sizes are
// gathered with 16-byte asynchronous copies, a row to half a warp (where both can be used: 208 us
// by boxes, 246 gathered for 256 rows; 171 and 207 for 64).
// Every wait is bounded; a thread that gave up goes through the rest of its schedule without
// waiting and without touching the tensor core, and the status word says so.
//
// What no row may see: scores are masked per row; rows past the last token or on a page out
// of range are zero in shared memory.  A draft node's values may be seen by some rows only, so
// non-finite ones are replaced by zero in the tile and added back in the epilogue of the
// rows that see the node (a positive weight times infinity or NaN is itself).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_draft_sm100.cuh"
#include "kda_tree_attn.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kBN = 128;
constexpr int kSoftmaxThreads = 256, kProducerThreads = 128, kThreads = kSoftmaxThreads + kProducerThreads + 128;
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;  // a thread; 512 threads start with 128 each
static_assert(kSoftmaxThreads * kSoftmaxRegs + (kThreads - kSoftmaxThreads) * kOtherRegs <= kThreads * 128, "register split");
constexpr int kCtas = 152;                          // one to an SM
// A unit's fixed cost (Q, first tile, epilogue), in tiles: 32 trees of 16 nodes, 96 heads, took 269 us
// with 0, 246 with 2, 223 with 4 and 229 with 8; units of few tiles lose from 6 on.
constexpr int kHead = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTame = 4096.f;                    // largest m sc of the form with one operation
constexpr float kGrow = 8.f;                        // powers of two a maximum may grow before O is multiplied

struct Shared {
    uint64_t kv_full[10], kv_empty[10], v_raw[10], s_full[2], p_full[2], q_full, q_empty, o_done[2], o_free[2];
    uint64_t bad_nodes[8];                          // by piece: nodes with non-finite values
    alignas(16) uint32_t missing[8][4];             // by tile: its tokens without a page (a V tile is freed after its
                                                    // softmax, so the copies are at most 6 tiles past it)
    TreeSmem tree[2];                               // one for each stream: they may be at different pieces
    uint32_t tmem;
};

template <int D, bool kWide>
struct Layout {
    static constexpr int kTile = kBN * D * 2;                   // bytes of a K or V tile, and of 128 rows of Q
    static constexpr int kQ = kTile * (kWide ? 2 : 1);
    static constexpr int kSlots = D == 128 ? 5 : 10;            // ring: K and V tiles in turn
    static constexpr int kLag = kSlots - 2;                     // gathered: slots in flight before the oldest is waited for
    static constexpr int kStats = kQ + kSlots * kTile;          // streams in turn: their maxima and sums, by piece parity
    static constexpr int kShared = kStats + (kWide ? 0 : 2 * 2 * 2 * 128 * 4);
    static constexpr int kBytes = kShared + (int)sizeof(Shared);
    static constexpr uint32_t kColS = 0, kColO = 256;           // stream w: S at 128 w, O at 256 + D w
    static_assert(kBytes <= 232448, "shared memory");
};

struct Maps {
    CUtensorMap k, v;       // [pages][page_size][kv_heads][D], boxes of box_rows x 64 channels
    int box_rows;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there)
{
    const int n = there ? 16 : 0;                   // 0: the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7f80u) != 0x7f80u; }

// ------------------------------------------------------------------ the cache rows
// Where a tile's tokens lie: lane l of producer warp w has token 32 w + l.
struct Rows {
    size_t koff, voff;      // elements from the caches' starts
    unsigned exists, lost;  // of the warp's 32 tokens: on a page; without one although the sequence has them
};

__device__ __forceinline__ Rows rows_of(const TreeAttnArgs& a, const attn::Piece& pc, int pos, int id, size_t row_stride, int D)
{
    const bool there = id >= 0 && id < a.num_pages;
    const size_t in_page = (size_t)(pos % a.page_size) * row_stride + (size_t)pc.hk * D;
    Rows r;
    r.lost = __ballot_sync(0xffffffffu, !there && pos < pc.n);
    r.exists = __ballot_sync(0xffffffffu, there);
    r.koff = there ? (size_t)id * a.k_page_stride + in_page : 0;
    r.voff = there ? (size_t)id * a.v_page_stride + in_page : 0;
    return r;
}

// The warp's 32 rows of a tile through registers; rows that do not exist become zero.  In the
// rows of draft nodes (node 0 in row `node0`, which may be negative) non-finite values become
// zero too and their nodes are noted.
template <int D>
__device__ __forceinline__ void copy_rows(uint8_t* dst, const __nv_bfloat16* src, size_t off, unsigned exists, int w, int lane,
                                          int node0, uint64_t* bad_nodes)
{
    constexpr int CH = D / 8, RPI = 32 / CH;        // 16-byte chunks of a row; rows a warp copies at once
    const int sub = lane / CH, chunk = lane % CH;
    uint32_t bad = 0;
    for (int i0 = 0; i0 < 32; i0 += 8 * RPI) {
        uint4 x[8];                                 // eight loads in flight
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
            if (32 * w + r >= node0) {
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
            if (bad >> r & 1) atomicOr(reinterpret_cast<unsigned long long*>(bad_nodes), 1ull << (32 * w + r - node0));
    }
}

// The same for a V tile that came by TMA; rows past the last token (from row `rows` on) become zero.
constexpr int kCleanThreads = 96;

template <int D>
__device__ __forceinline__ void clean_rows(uint8_t* tile, int node0, int rows, int t, uint64_t* bad_nodes)
{
    constexpr int CH = D / 8, STEP = kCleanThreads / CH;
    const int chunk = t % CH;
#pragma unroll 4
    for (int r = max(0, node0) + t / CH; r < kBN; r += STEP) {
        uint4* at = reinterpret_cast<uint4*>(tile + sw128_chunk(r, chunk, 128));
        if (r >= rows) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4 x = *at;
        uint32_t h[4] = {x.x, x.y, x.z, x.w};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool lo = finite_bf16(h[e]), hi = finite_bf16(h[e] >> 16);
            bad |= !(lo && hi);
            h[e] = (lo ? h[e] & 0xffffu : 0u) | (hi ? h[e] & 0xffff0000u : 0u);
        }
        if (bad) {
            *at = make_uint4(h[0], h[1], h[2], h[3]);
            atomicOr(reinterpret_cast<unsigned long long*>(bad_nodes), 1ull << (r - node0));
        }
    }
}

// By TMA.  Warp 0 of the four issues the boxes, a lane to a box; a V tile with draft nodes is
// handed over by the other three once they have cleaned it.  A tile with tokens that have no
// page passes through registers, by all four.
template <int D, bool kWide>
__device__ __forceinline__ void produce_boxes(const TreeAttnArgs& a, const attn::Shape& sh, const Maps& maps, attn::Line line, Shared& sm,
                                              uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    const int lane = t & 31, w = t >> 5, box = maps.box_rows;
    Waiter wait{a.status};
    attn::Piece pc;
    uint32_t fill = 0, raw_phase = 0;
    bool bad_page = false;
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        if (t == 0) sm.bad_nodes[piece & 7] = 0;    // (before this warp lets any other see a tile of the piece)
        const int32_t* table = a.block_table + (size_t)pc.b * a.table_cols;
        auto look_up = [&](int tile) {              // box `lane` of the tile
            const int pos = tile * kBN + lane * box;
            return tile < pc.last && lane * box < kBN && pos < pc.n ? __ldg(table + pos / a.page_size) : -1;
        };
        int next = look_up(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile) {
            const int t0 = tile * kBN, pos = t0 + lane * box, id = next;
            const bool wanted = lane * box < kBN && pos < pc.n, there = wanted && id >= 0 && id < a.num_pages;
            const bool lost = __any_sync(0xffffffffu, wanted && !there);
            const int boxes = __popc(__ballot_sync(0xffffffffu, there));
            next = look_up(tile + 1);
            const bool nodes = t0 + kBN > pc.ctx;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++fill) {
                const uint32_t s = fill % L::kSlots;
                uint8_t* dst = base + L::kQ + s * L::kTile;
                if (w == 0 && fill >= (uint32_t)L::kSlots) wait(&sm.kv_empty[s], (fill / L::kSlots - 1) & 1);
                if (lost) {
                    const int p = t0 + 32 * w + lane;
                    const Rows rows = rows_of(a, pc, p, p < pc.n ? __ldg(table + p / a.page_size) : -1, (size_t)a.kv_heads * D, D);
                    bad_page |= rows.lost != 0;
                    bar_sync(10, kProducerThreads); // the slot is free
                    if (kv == 0 && lane == 0) sm.missing[fill / 2 & 7][w] = rows.lost;
                    copy_rows<D>(dst, static_cast<const __nv_bfloat16*>(kv ? a.v_cache : a.k_cache), kv ? rows.voff : rows.koff, rows.exists,
                                 w, lane, kv ? pc.ctx - t0 : kBN, &sm.bad_nodes[piece & 7]);
                    fence_proxy_async_smem();
                    bar_sync(10, kProducerThreads);
                    if (t == 0) mbar_arrive(&sm.kv_full[s]);
                    continue;
                }
                uint64_t* const landed = kv && nodes ? &sm.v_raw[s] : &sm.kv_full[s];
                if (w == 0) {
                    const bool go = __all_sync(0xffffffffu, wait.alive);
                    if (kv == 0 && lane < 4) sm.missing[fill / 2 & 7][lane] = 0;
                    __syncwarp();
                    if (lane == 0) {
                        if (go) mbar_arrive_expect_tx(landed, boxes * box * D * 2);
                        else mbar_arrive(landed);
                    }
                    __syncwarp();
                    if (go && there) {
#pragma unroll
                        for (int c = 0; c < D; c += 64)
                            tma_load_4d(dst + (c / 64) * (kBN * 128) + lane * box * 128, kv ? &maps.v : &maps.k, landed, c, pc.hk,
                                        pos % a.page_size, id);
                    }
                } else if (kv && nodes) {
                    wait(landed, raw_phase >> s & 1);
                    raw_phase ^= 1u << s;
                    clean_rows<D>(dst, pc.ctx - t0, pc.n - t0, t - 32, &sm.bad_nodes[piece & 7]);
                    fence_proxy_async_smem();
                    bar_sync(11, kCleanThreads);
                    if (t == 32) mbar_arrive(&sm.kv_full[s]);
                }
            }
        }
    }
    // no load is in flight when the block ends, whatever became of its reader
    if (w == 0)
        for (uint32_t i = fill > (uint32_t)L::kSlots ? fill - L::kSlots : 0; i < fill; ++i)
            mbar_wait_bounded(&sm.kv_full[i % L::kSlots], (i / L::kSlots) & 1, kDraftWaitNs);
    if (bad_page && lane == 0) report_status(a.status, kDevBadSeqlens);
    wait.finish();
}

// By 16-byte asynchronous copies, all four warps.
template <int D, bool kWide>
__device__ __forceinline__ void produce_gather(const TreeAttnArgs& a, const attn::Shape& sh, attn::Line line, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int lane = t & 31, w = t >> 5;
    // (a cache without pages may be a null pointer: copies of no bytes then start at q)
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.k_cache : a.q);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.v_cache : a.q);
    const size_t row_stride = (size_t)a.kv_heads * D;
    Waiter wait{a.status};
    attn::Piece pc;
    uint32_t fill = 0, sent = 0;                    // ring slots begun, and handed over
    bool bad_page = false;
    const int sub = lane / CH, chunk = lane % CH;

    auto hand_over = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&sm.kv_full[sent % L::kSlots]);
        ++sent;
    };
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        if (t == 0) sm.bad_nodes[piece & 7] = 0;
        bar_sync(10, kProducerThreads);
        const int32_t* table = a.block_table + (size_t)pc.b * a.table_cols;
        auto look_up = [&](int tile) {              // one tile ahead
            const int pos = tile * kBN + 32 * w + lane;
            return tile < pc.last && pos < pc.n ? __ldg(table + pos / a.page_size) : -1;
        };
        int id = look_up(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile) {
            const int t0 = tile * kBN;
            const Rows rows = rows_of(a, pc, t0 + 32 * w + lane, id, row_stride, D);
            bad_page |= rows.lost != 0;
            id = look_up(tile + 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s = fill % L::kSlots;
                if (fill >= (uint32_t)L::kSlots) wait(&sm.kv_empty[s], (fill / L::kSlots - 1) & 1);
                uint8_t* dst = base + L::kQ + s * L::kTile;
                if (kv == 0 && lane == 0) sm.missing[fill / 2 & 7][w] = rows.lost;
                const __nv_bfloat16* src = kv ? vc : kc;
                const size_t off = kv ? rows.voff : rows.koff;
                if (kv == 1 && t0 + kBN > pc.ctx) {
                    copy_rows<D>(dst, src, off, rows.exists, w, lane, pc.ctx - t0, &sm.bad_nodes[piece & 7]);
                } else {
#pragma unroll 4
                    for (int i = 0; i < 32; i += RPI) {
                        const int r = i + sub;
                        const size_t o = __shfl_sync(0xffffffffu, off, r);
                        cp16(smem_u32(dst + sw128_chunk(32 * w + r, chunk, 128)), src + o + 8 * chunk, rows.exists >> r & 1);
                    }
                }
                cp_commit();
                ++fill;
                if (fill - sent > L::kLag) {        // hand over the slot kLag before this one
                    cp_wait<L::kLag>();
                    hand_over();
                }
            }
        }
    }
    cp_wait<0>();
    while (sent != fill) hand_over();
    if (bad_page && lane == 0) report_status(a.status, kDevBadSeqlens);
    wait.finish();
}

// ------------------------------------------------------------------ the query rows
// Three warps, as soon as the last piece's scores are done.  Rows past the unit's last are left as
// they are (no row's result depends on another row); scale 0 is a zero Q (every score is then 0).
constexpr int kQueryThreads = 96;

template <int D, bool kWide>
__device__ __forceinline__ void query(const TreeAttnArgs& a, const attn::Shape& sh, attn::Line line, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    constexpr int CH = D / 8, STEP = kQueryThreads / CH;   // chunks of a row; rows copied at once
    const int G = a.heads / a.kv_heads, R = a.nodes * G, c = t % CH;
    const int step_node = STEP / G, step_head = STEP - step_node * G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    Waiter wait{a.status};
    attn::Piece pc;
    attn::Recorder rec;
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        rec.see(line, pc);
        int r = t / CH, node = (pc.r0 + r) / G, head = pc.r0 + r - node * G;
        const __nv_bfloat16* src = q + ((size_t)pc.b * a.nodes * a.heads + pc.hk * G) * D + 8 * c;
        if (piece) wait(&sm.q_empty, (piece - 1) & 1);
#pragma unroll 4
        for (const int rows = min(sh.BM, R - pc.r0); r < rows; r += STEP) {
            const bool there = a.scale != 0.f;
            cp16(smem_u32(base + (r >> 7) * L::kTile + sw128_chunk(r & 127, c, 128)), there ? src + ((size_t)node * a.heads + head) * D : q, there);
            node += step_node;
            head += step_head;
            if (head >= G) { head -= G; ++node; }
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full);
    }
    if (t == 0) rec.leave(a, blockIdx.x);
    wait.finish();
}

// ------------------------------------------------------------------ the products
template <int D, bool kWide>
__device__ __forceinline__ void multiply(const TreeAttnArgs& a, const attn::Shape& sh, attn::Line line, Shared& sm, uint8_t* base)
{
    using L = Layout<D, kWide>;
    Waiter wait{a.status};
    attn::Piece pc;
    const uint32_t tm = sm.tmem, q0 = smem_u32(base), ring = q0 + L::kQ;
    const uint32_t id_s = idesc_bf16_f32(128, kBN, 0, 0, a.scale < 0.f), id_o = idesc_bf16_f32(128, D, 0, 1);
    // ring slot and phase of the next K and V tile; items of each stream so far
    uint32_t ks_ = 0, kp = 0, vs_ = 1, vp = 0, used[2] = {0, 0}, pieces[2] = {0, 0};   // (and pieces of each stream)
    auto advance = [](uint32_t& s, uint32_t& phase) {
        s += 2;
        if (s >= (uint32_t)L::kSlots) { s -= L::kSlots; phase ^= 1; }
    };
    uint32_t piece = 0;
    for (; line.next(a, sh, blockIdx.x, pc); ++piece) {
        const int tiles = pc.last - pc.first, items = kWide ? 2 * tiles : tiles;
        wait(&sm.q_full, piece & 1);
        // item i: stream i % 2; its tile is i (streams in turn) or i / 2 (each tile for both)
        auto scores = [&](int i, int w) {
            const bool first = !kWide || w == 0, last = !kWide || w == 1;   // to use the tile
            const uint32_t s = ks_;
            if (first) wait(&sm.kv_full[s], kp);
            if (last) advance(ks_, kp);
            tc_fence_after_sync();
            {
                if (wait.alive) {
                    const uint64_t qd = kmajor_base(q0 + (kWide ? w * L::kTile : 0)), kd = kmajor_base(ring + s * L::kTile);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_bf16(tm + L::kColS + 128 * w, desc_off(qd, kmajor_off(128, ks)), desc_off(kd, kmajor_off(128, ks)), id_s, ks > 0);
                }
                umma_commit(&sm.s_full[w]);
                if (last) umma_commit(&sm.kv_empty[s]);
                if (i == items - 1) umma_commit(&sm.q_empty);
            }
        };
        auto values = [&](int i, int w) {
            const bool first = !kWide || w == 0, last = !kWide || w == 1;
            const uint32_t s = vs_;
            if (first) wait(&sm.kv_full[s], vp);
            if (last) advance(vs_, vp);
            if (i == w) {                           // the stream's first products of the piece overwrite O
                if (pieces[w]) wait(&sm.o_free[w], (pieces[w] - 1) & 1);
                ++pieces[w];
            }
            wait(&sm.p_full[w], used[w] & 1);
            ++used[w];
            tc_fence_after_sync();
            {
                if (wait.alive) {
                    const uint64_t vd = mnmajor_base(ring + s * L::kTile, kBN);
#pragma unroll
                    for (int ks = 0; ks < kBN / 16; ++ks)
                        umma_bf16_tmem_a(tm + L::kColO + D * w, tm + L::kColS + 128 * w + 8 * ks, desc_off(vd, mnmajor_off(ks)), id_o, i > 1 || ks > 0);
                }
                if (last) umma_commit(&sm.kv_empty[s]);
                if (i + 2 >= items) umma_commit(&sm.o_done[w]);
            }
        };
        // (one thread for all of it: with the whole warp in the waits and a thread elected for each
        // group of products their issue took 3000 cycles a tile, now 2150 of the pipe's 2048)
        scores(0, 0);
        if (items > 1) scores(1, 1);
        for (int i = 0; i < items; i += 2) {        // both streams in turn
            values(i, 0);
            if (i + 2 < items) scores(i + 2, 0);
            if (i + 1 < items) values(i + 1, 1);
            if (i + 3 < items) scores(i + 3, 1);
        }
    }
    for (int w = 0; w < 2; ++w)                     // no product or commit is in flight after this
        if (pieces[w]) wait(&sm.o_done[w], (pieces[w] - 1) & 1);
    wait.finish();
}

// ------------------------------------------------------------------ softmax and epilogue
// What row sees of the tile at t0: 128 bits, four words.
__device__ __forceinline__ void tile_mask(uint64_t see, int t0, int ctx, uint4 lost, uint32_t (&mw)[4])
{
    const uint32_t missing[4] = {lost.x, lost.y, lost.z, lost.w};
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

__device__ __forceinline__ float max_of(const float (&x)[32])
{
    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        a0 = fmaxf(a0, fmaxf(x[k], x[k + 1]));
        a1 = fmaxf(a1, fmaxf(x[k + 2], x[k + 3]));
    }
    return fmaxf(a0, a1);
}

// One step of the transpose of 4 x 4 pieces over four lanes: lanes that differ in bit `by`
// exchange the later of two pieces for the earlier one.
__device__ __forceinline__ void swap_pieces(uint4& lo, uint4& hi, bool upper, int by)
{
    uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
    uint32_t* h = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? l[e] : h[e], by);
        if (upper) l[e] = got;
        else h[e] = got;
    }
}

template <int D, bool kWide>
__device__ __forceinline__ void softmax(const TreeAttnArgs& a, const attn::Shape& sh, attn::Line line, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D, kWide>;
    float* stats = reinterpret_cast<float*>(base + L::kStats);        // [stream][m, l][128]
    const int lane = t & 31, warp = t >> 5, w = t >> 7, r = t & 127;   // stream and lane of tensor memory
    const int G = a.heads / a.kv_heads, R = a.nodes * G;
    const uint32_t quad = 32 * (warp & 3);                            // the lanes this warp reaches
    const uint32_t tS = tmem_addr(sm.tmem, quad, L::kColS + 128 * w), tO = tmem_addr(sm.tmem, quad, L::kColO);
    const float sc = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;  // scores in powers of two
    Waiter wait{a.status};
    attn::Piece pc;
    uint32_t used = 0, done = 0, pieces[2] = {0, 0};   // items of this stream, tiles, pieces of each stream so far
    int masks_of = -1;
    TreeSmem& tree = sm.tree[w];
    for (uint32_t piece = 0; line.next(a, sh, blockIdx.x, pc); ++piece) {
        const int tiles = pc.last - pc.first;
        if (pc.b != masks_of) {
            bar_sync(2 + w, 128);                   // the stream's warps have read the last tree
            if ((warp & 3) == 0) tree_masks(tree, a.parents + (size_t)pc.b * a.nodes, a.nodes, lane);
            masks_of = pc.b;
            bar_sync(2 + w, 128);
        }
        if (!(pc.seq_ok && tree.ok) && t == 0) report_status(a.status, kDevBadSeqlens);
        const int row = pc.r0 + (kWide ? 128 * w : 0) + r;
        const uint64_t see = pc.seq_ok && tree.ok && row < R ? tree.anc[row / G] : 0ull;
        const bool busy = __any_sync(0xffffffffu, see != 0);
        // m in score units, before sc; a row that may see nothing never asks for another maximum
        float m = see ? -INFINITY : INFINITY, l = 0.f;
        bool begun = false;

        for (int i = kWide ? 0 : w; i < tiles; i += kWide ? 1 : 2) {
            const int t0 = (pc.first + i) * kBN;
            wait(&sm.s_full[w], used & 1);
            ++used;
            __syncwarp();
            tc_fence_after_sync();
            if (busy) {
                const uint4 missing = *reinterpret_cast<const uint4*>(sm.missing[(done + i) & 7]);
                const bool all = t0 + kBN <= pc.ctx && !(missing.x | missing.y | missing.z | missing.w);
                const float2 sc2 = make_float2(sc, sc);
                // (x - m) sc in this order: the difference is exact where it matters, whatever the scores
                auto weigh = [&](const float (&x)[32], float2 off, float2& sum, uint32_t (&p)[16]) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[2 * k], x[2 * k + 1]), off), sc2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = __fadd2_rn(sum, e);
                        p[k] = pack_bf16x2(e.x, e.y);
                    }
                };
                bool stored = false;
                if (all && !begun) {
                    float x[32];
                    tmem_ld32(tS, x);
                    tmem_wait_ld();
                    m = see ? max_of(x) : INFINITY;
                }
                // A tile that every row sees whole: the weights are formed from the last maximum (in
                // a piece's first tile, that of 32 tokens) while the tile's own is still being
                // found, and stored over the scores once it is known that it may stand (nearly always).
                // x sc - m sc in one operation: m sc's rounding is a factor that a row's weights share, and
                // up to kTame it is 2^-13 of a weight, below bf16's rounding, where the maximum changes.
                if (all && !__any_sync(0xffffffffu, see && !(fabsf(m) * sc <= kTame))) {
                    const float2 off = make_float2(-m * sc, -m * sc);
                    auto weigh = [&](const float (&x)[32], float2 off, float2& sum, uint32_t (&p)[16]) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * k], x[2 * k + 1]), sc2, off);
                            const float2 e = make_float2(ex2(y.x), ex2(y.y));
                            sum = __fadd2_rn(sum, e);
                            p[k] = pack_bf16x2(e.x, e.y);
                        }
                    };
                    float2 sum = make_float2(0.f, 0.f);
                    float top = -INFINITY;
                    uint32_t p[4][16];
                    float xa[32], xb[32];
                    tmem_ld32(tS, xa);
                    tmem_wait_ld();
                    tmem_ld32(tS + 32, xb);
                    top = fmaxf(top, max_of(xa));
                    weigh(xa, off, sum, p[0]);
                    tmem_wait_ld();
                    tmem_ld32(tS + 64, xa);
                    top = fmaxf(top, max_of(xb));
                    weigh(xb, off, sum, p[1]);
                    tmem_wait_ld();
                    tmem_ld32(tS + 96, xb);
                    top = fmaxf(top, max_of(xa));
                    weigh(xa, off, sum, p[2]);
                    tmem_wait_ld();
                    top = fmaxf(top, max_of(xb));
                    weigh(xb, off, sum, p[3]);
                    if (!__any_sync(0xffffffffu, (top - m) * sc > kGrow)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_st16u(tS + 16 * c, p[c]);
                        l += sum.x + sum.y;
                        stored = true;
                    }
                }
                if (!stored) {
                    // masks, the first maximum, or one that has grown: the maximum first, then the weights
                    // (word c's go to columns 16 c, over scores that have been read)
                    uint32_t mw[4] = {~0u, ~0u, ~0u, ~0u};
                    if (!all) tile_mask(see, t0, pc.ctx, missing, mw);
                    auto read = [&](int c, float (&x)[32]) {
                        const uint32_t on = c == 0 ? mw[0] : c == 1 ? mw[1] : c == 2 ? mw[2] : mw[3];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = on >> k & 1 ? x[k] : -INFINITY;
                    };
                    float top = -INFINITY, x[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        read(c, x);
                        top = fmaxf(top, max_of(x));
                    }
                    const bool grow = (top - m) * sc > kGrow;
                    const float nm = grow ? top : m;
                    const float f = grow ? ex2((m - nm) * sc) : 1.f;   // 0 for the first maximum
                    l *= f;
                    m = nm;
                    if (begun && __any_sync(0xffffffffu, grow)) {      // (S is ready: the stream's last products into O are done)
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            tmem_ld32(tO + D * w + c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] *= f;
                            tmem_st32(tO + D * w + c, x);
                        }
                    }
                    const float2 off = make_float2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
                        read(c, x);
                        weigh(x, off, sum, p);
                        tmem_st16u(tS + 16 * c, p);
                    }
                    l += sum.x + sum.y;
                }
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
        const bool two = !kWide && tiles > 1;       // stream 1 has a part of the same rows
        float* st = stats + (kWide ? 0 : 512 * (piece & 1));
        if (!kWide) {
            st[256 * w + r] = m;
            st[256 * w + 128 + r] = l;
        }
        for (int k = 0; k < 2; ++k)                 // the streams this thread reads: its own, or both of the piece
            if (kWide ? k == w : k == 0 || two) wait(&sm.o_done[k], pieces[k]++ & 1);
        __syncwarp();
        tc_fence_after_sync();
        if (!kWide) bar_sync(1, kSoftmaxThreads);
        const uint64_t bad = *const_cast<volatile uint64_t*>(&sm.bad_nodes[piece & 7]) & see;
        // this thread's columns [c0, c1) of the row: stream 1's part is joined when it has one
        const int c0 = kWide ? 0 : w * (D / 2), c1 = kWide ? D : c0 + D / 2;
        float f0 = 1.f, f1 = 0.f;
        if (!kWide) {
            const float m0 = st[r], m1 = two ? st[256 + r] : -INFINITY, l0 = st[128 + r], l1 = two ? st[384 + r] : 0.f;
            m = fmaxf(m0, m1);
            f0 = m0 == -INFINITY ? 0.f : ex2((m0 - m) * sc);
            f1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * sc);
            l = (m0 == -INFINITY ? l0 : l0 * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
        }
        const float norm = pc.whole() ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        float* ws = attn::slot_of(a, sh, D, pc.slot);
        const int rl = row - pc.r0;                 // row of the unit
        if (row < R && !pc.whole() && c0 == 0) {
            ws[rl] = m == -INFINITY ? m : m * sc;
            ws[sh.BM + rl] = l;
        }
        // out's row of this thread (in rows of D), and of the four rows of its group of four lanes
        const int orow = row < R ? (int)(((size_t)pc.b * a.nodes + row / G) * a.heads + pc.hk * G + row % G) : -1;
        int orows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) orows[k] = __shfl_sync(0xffffffffu, orow, (lane & ~3) + k);
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
            if (pc.whole()) {
                // Four lanes hold four rows of 32 channels, 16 bytes at a time; after the exchange
                // lane j holds piece j of each row, and a store covers 64 bytes of eight rows
                // instead of 16 bytes of 32.
                uint4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                      pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
                swap_pieces(x[0], x[1], lane & 1, 1);
                swap_pieces(x[2], x[3], lane & 1, 1);
                swap_pieces(x[0], x[2], lane & 2, 2);
                swap_pieces(x[1], x[3], lane & 2, 2);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (orows[k] >= 0)
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (size_t)orows[k] * D + c + 8 * (lane & 3)) = x[k];
            } else if (row < R) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    attn::slot_out(ws, sh.BM)[(size_t)((c + k) / 4) * sh.BM + rl] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            if (kWide || w == 0 || two) mbar_arrive(&sm.o_free[w]);
            if (!kWide && (w == 1 || two)) mbar_arrive(&sm.o_free[w ^ 1]);
        }
    }
    wait.finish();
}

template <int D, bool kWide, bool kBoxes>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_tc_kernel(TreeAttnArgs a, attn::Shape sh, const __grid_constant__ Maps maps)
{
    using L = Layout<D, kWide>;
    extern __shared__ __align__(1024) uint8_t base[];   // all of it: the swizzled tiles start at 0
    Shared& sm = *reinterpret_cast<Shared*>(base + L::kShared);
    const int t = threadIdx.x, warp = t >> 5;
    attn::Line line;
    line.begin(a, sh, blockIdx.x, t & 31);
    if (warp == 12) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    if (t == 0) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&sm.kv_full[i], kBoxes ? 1 : kProducerThreads);
            mbar_init(&sm.kv_empty[i], 1);
            mbar_init(&sm.v_raw[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.o_free[i], kWide ? 4 : 8);
        }
        mbar_init(&sm.q_full, kQueryThreads);
        mbar_init(&sm.q_empty, 1);
        for (int i = 0; i < 8; ++i) sm.bad_nodes[i] = 0;
        mbar_fence_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax<D, kWide>(a, sh, line, sm, base, t);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < 12) {
            if constexpr (kBoxes) produce_boxes<D, kWide>(a, sh, maps, line, sm, base, t - kSoftmaxThreads);
            else produce_gather<D, kWide>(a, sh, line, sm, base, t - kSoftmaxThreads);
        } else if (warp == 12) {
            if (elect_one()) multiply<D, kWide>(a, sh, line, sm, base);
        } else {
            query<D, kWide>(a, sh, line, sm, base, t - 13 * 32);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 12) tmem_dealloc(sm.tmem, 512);
}

// 256-row units where 128 would not hold all rows of a (sequence, head): every tile is then read and
// turned into operands once.  256 rows, 2 x 131072 tokens: 208 us wide, 324 in two units of 128;
// 128 rows: 190 wide (half of it empty), 178 with both streams on them.
bool wide_rows(int nodes, int group) { return nodes * group > 128; }
attn::Shape shape_of(bool wide) { return {wide ? 256 : 128, kBN, kCtas, kHead}; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Whether the cache can be read in boxes: see the top; a map holds strides below 2^40 bytes.
bool in_boxes(const TreeAttnArgs& a)
{
    const size_t most = ((size_t)1 << 40) / 2 - 1;
    return a.page_size % 8 == 0 && a.num_pages > 0 && a.k_page_stride <= most && a.v_page_stride <= most;
}

bool make_map(CUtensorMap* m, const void* cache, size_t page_stride, const TreeAttnArgs& a, int rows)
{
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t D = (cuuint64_t)a.dim, H = (cuuint64_t)a.kv_heads;
    const cuuint64_t dims[4] = {D, H, (cuuint64_t)a.page_size, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {D * 2, H * D * 2, (cuuint64_t)page_stride * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, a.dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kWide, bool kBoxes>
cudaError_t launch(const TreeAttnArgs& a, cudaStream_t stream)
{
    using L = Layout<D, kWide>;
    const auto kernel = tree_attn_tc_kernel<D, kWide, kBoxes>;
    const attn::Shape sh = shape_of(kWide);
    Maps maps = {};
    if (kBoxes) {
        maps.box_rows = min(a.page_size & -a.page_size, kBN);
        if (!make_map(&maps.k, a.k_cache, a.k_page_stride, a, maps.box_rows) || !make_map(&maps.v, a.v_cache, a.v_page_stride, a, maps.box_rows))
            return cudaErrorInvalidValue;
    }
    // (the register split needs the block to start with all 128 registers a thread)
    static KernelSetup setup;
    cudaError_t e = setup(kernel, L::kBytes, 128);
    if (e != cudaSuccess) return e;
    kernel<<<sh.ctas, kThreads, L::kBytes, stream>>>(a, sh, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return attn::launch_join<__nv_bfloat16, D>(a, sh, stream);
}

template <int D>
cudaError_t launch_dim(const TreeAttnArgs& a, cudaStream_t stream)
{
    const bool wide = wide_rows(a.nodes, a.heads / a.kv_heads);
    if (in_boxes(a)) return wide ? launch<D, true, true>(a, stream) : launch<D, false, true>(a, stream);
    return wide ? launch<D, true, false>(a, stream) : launch<D, false, false>(a, stream);
}

}  // namespace

size_t tree_attn_tc_workspace_bytes(int nodes, int group, int dim)
{
    return attn::workspace_bytes(shape_of(wide_rows(nodes, group)), dim);
}

bool tree_attn_tc_fits(const TreeAttnArgs& a) { return attn::line_fits(a, shape_of(wide_rows(a.nodes, a.heads / a.kv_heads))); }

cudaError_t launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t stream)
{
    return a.dim == 128 ? launch_dim<128>(a, stream) : launch_dim<64>(a, stream);
}

}  // namespace kda
