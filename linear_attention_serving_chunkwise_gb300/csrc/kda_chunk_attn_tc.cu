// Softmax attention of chunks of new tokens over a paged bf16 key/value cache, on the Blackwell tensor cores (tcgen05).
// The cut of the work and the join are those of kda_chunk_attn.cuh: one pass over the tokens, running maximum and sum per
// row, parts of split units joined afterwards.
//
// The query rows of a block of tokens -- tokens x the G heads of a cache head -- fill the 128 lanes of an
// accumulator: S = Q K^T per tile of 128 tokens, the weights overwrite half of S in tensor
// memory as the bf16 A operand of O += P V, and O stays in tensor memory for the whole piece.  Two
// streams of S and O, of 128 rows each, share the tensor core and every tile, so that one stream's softmax runs under the
// other's products.  (Units of 128 rows, whose tiles the streams take in turn, lose where there is work: 32 single tokens after 8192 252 us
// instead of 214, 40 tokens 537 instead of 236; for 129 tokens after none they win, 17.7 us instead of 20.5.)
// A row's maximum is set anew, and O multiplied, only when its weights of a tile sum to more than 2^15 (until then no
// weight is more, which bf16 and the fp32 sums hold as well).  That takes up to 15 bits of the range that O has for values: 2^24 tiles
// of 2^15 make a row's sum 2^39 at most, so with values up to 2^82, the fp32 kernel's bound, nothing overflows.  A limit of 2^8
// leaves seven bits more and costs four times sharper scores than a standard normal's 37 % (a prompt of 8192 400 -> 545 us).
// The weights are rounded to bf16 because the tensor core takes both operands of a product in one 16-bit type, and the values
// are bf16; their sum is that of the unrounded ones.
//
// Warps 0-3 and 4-7: softmax and epilogue of stream 0 and 1, a row to a thread.  Warps 8-11:
// the cache rows, into a ring of K and V tiles.  A thread of warp 12 issues the products, warps
// 13-15 copy Q.  The last two groups give registers to the softmax.
//
// Bound, for many rows: not the tensor pipe alone (69 % busy: 2048 of some 2960 cycles a tile of 256 rows x 128 tokens,
// D = 128) but each stream's chain scores - softmax - values, which the other one's products cover only in part.  The softmax's way
// from scores to weights takes 1200 cycles, of which 750 form 128 weights a thread, and the products' thread adds waits and commits.
// 2048 tokens after 131072, 32 heads on 8: 2.90 to 2.95 ms, 1500 to 1530 TFLOP/s (0.79 of cuBLAS's burst); 12 sequences of 1 to 2048 tokens
// after up to 16384, 96 heads on 8: 4.05 to 4.10 ms, 1420 to 1440; a prompt of 8192: 399 us, 1380; 512 after 131072: 735 us, 1500; 16
// prompts of 512: 99 us, 350 (a unit of three tiles costs 11 us: its first tile, masks and epilogue); 64 tokens after 4096 to 32768
// each: 790 to 810 us, 6.2 TB/s; D = 64: 2048 after 131072 2.2 ms, 1000 (the same
// softmax for half the products).  In one wave instead of eight the first two took 3.52 and 4.83 ms instead of 3.03 and 4.27;
// with the weights handed over in two parts 2.99 and 4.37 instead of 3.00 and 4.20.
//
// The cache rows come by TMA where the page size is a multiple of 8: a tile is a stack of boxes
// of 8 to 128 rows (the largest power of two in the page size), and 8 rows are one swizzle
// atom, so boxes of any pages stack into the tile the products read.  Other page sizes are
// gathered with 16-byte asynchronous copies, a row to half a warp (2.95 ms by boxes, 4.30 gathered for 2048 after 131072).
// Every wait is bounded; a thread that gave up goes through the rest of its schedule without
// waiting and without touching the tensor core, and the status word says so.
//
// What no row may see: scores are masked per row; rows past the block's last token or on a page out
// of range are zero in shared memory.  The values of the block's own tokens may be seen by some rows only, so
// non-finite ones are replaced by zero in the tile and added back in the epilogue of the
// rows that see the token (a positive weight times infinity or NaN is itself).
#include <float.h>

#include "kda_attn_tc.cuh"
#include "kda_chunk_attn.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kBN = kTileTokens, kBM = 256;
constexpr int kSoftmaxThreads = 256, kProducerThreads = 128, kThreads = kSoftmaxThreads + kProducerThreads + 128;
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;  // a thread; 512 threads start with 128 each
static_assert(kSoftmaxThreads * kSoftmaxRegs + (kThreads - kSoftmaxThreads) * kOtherRegs <= kThreads * 128, "register split");
constexpr int kCtas = 152;                          // one to an SM
// A unit's fixed cost (Q, first tile, epilogue), in tiles: with 1, 2, 4 and 6 a prompt of 8192 took 477, 443, 399 and 405 us.
constexpr int kHead = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTame = 4096.f;                     // largest m sc of the form with one operation
constexpr float kMostSum = 32768.f;                 // most that a row's weights of a tile may sum to before its maximum is set anew
// The maximum of a row that sees tokens whose scores are all -inf: its weights are 0 over 0, as by the definition, where a row that sees
// no token (maximum -inf) becomes zero.
constexpr float kLowest = -FLT_MAX;

struct Shared {
    uint64_t kv_full[10], kv_empty[10], v_raw[10], s_full[2], p_full[2], q_full, q_empty, o_done[2], o_free[2];
    alignas(16) uint32_t missing[8][4];             // by tile: its tokens without a page (a V tile is freed after its
                                                    // softmax, so the copies are at most 6 tiles past it)
    alignas(16) uint32_t bad[8][8];                 // by piece: the block's own tokens with non-finite values
    chunk::Line lines[chunk::kMaxWaves];
    uint32_t tmem;
};

// A CTA's ranges one after another.
struct Walk {
    const Shared& sm;
    int waves, w = 0;
    chunk::Line line;
    __device__ __forceinline__ Walk(const Shared& s, int n) : sm(s), waves(n), line(s.lines[0]) {}
    __device__ __forceinline__ bool next(const ChunkAttnArgs& a, const Shape& sh, chunk::Piece& p)
    {
        while (!line.next(a, sh, p)) {
            if (++w >= waves) return false;
            line = sm.lines[w];
        }
        return true;
    }
};

template <int D>
struct Layout {
    static constexpr int kTile = kBN * D * 2;                   // bytes of a K or V tile, and of 128 rows of Q
    static constexpr int kQ = 2 * kTile;
    static constexpr int kSlots = D == 128 ? 5 : 10;            // ring: K and V tiles in turn
    static constexpr int kLag = kSlots - 2;                     // gathered: slots in flight before the oldest is waited for
    static constexpr int kShared = kQ + kSlots * kTile;
    static constexpr int kBytes = kShared + (int)sizeof(Shared);
    static constexpr uint32_t kColS = 0, kColO = 256;           // stream w: S at 128 w, O at 256 + D w
    static_assert(kBytes <= 232448, "shared memory");
};

// ------------------------------------------------------------------ the cache rows
// By TMA.  Warp 0 of the four issues the boxes, a lane to a box; a V tile with tokens that not
// all rows see is handed over by the other three once they have cleaned it.  A tile with tokens that have no
// page passes through registers, by all four.
template <int D>
__device__ __forceinline__ void produce_boxes(const ChunkAttnArgs& a, const Shape& sh, const Maps& maps, int waves, Shared& sm,
                                              uint8_t* base, int t)
{
    using L = Layout<D>;
    const int lane = t & 31, w = t >> 5, box = maps.box_rows;
    Waiter wait{a.status};
    Walk walk(sm, waves);
    chunk::Piece pc;
    uint32_t fill = 0, raw_phase = 0;
    bool bad_page = false;
    for (uint32_t piece = 0; walk.next(a, sh, pc); ++piece) {
        if (t < 8) sm.bad[piece & 7][t] = 0;        // (before this warp lets any other see a tile of the piece)
        const int32_t* table = a.block_table + (size_t)pc.b * a.table_cols;
        auto look_up = [&](int tile) {              // box `lane` of the tile
            const int pos = tile * kBN + lane * box;
            return tile < pc.last && lane * box < kBN && pos < pc.seen ? __ldg(table + pos / a.page_size) : -1;
        };
        int next = look_up(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile) {
            const int t0 = tile * kBN, pos = t0 + lane * box, id = next;
            const bool wanted = lane * box < kBN && pos < pc.seen, there = wanted && id >= 0 && id < a.num_pages;
            const bool lost = __any_sync(0xffffffffu, wanted && !there);
            const int boxes = __popc(__ballot_sync(0xffffffffu, there));
            next = look_up(tile + 1);
            const bool partly = t0 + kBN > pc.common;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++fill) {
                const uint32_t s = fill % L::kSlots;
                uint8_t* dst = base + L::kQ + s * L::kTile;
                if (w == 0 && fill >= (uint32_t)L::kSlots) wait(&sm.kv_empty[s], (fill / L::kSlots - 1) & 1);
                if (lost) {
                    const int p = t0 + 32 * w + lane;
                    const Rows rows = rows_of(a, pc.hk, p, pc.seen, p < pc.seen ? __ldg(table + p / a.page_size) : -1, (size_t)a.kv_heads * D, D);
                    bad_page |= rows.lost != 0;
                    bar_sync(10, kProducerThreads); // the slot is free
                    if (kv == 0 && lane == 0) sm.missing[fill / 2 & 7][w] = rows.lost;
                    copy_rows<D>(dst, static_cast<const __nv_bfloat16*>(kv ? a.v_cache : a.k_cache), kv ? rows.voff : rows.koff, rows.exists,
                                 w, lane, kv ? pc.common - t0 : kBN, sm.bad[piece & 7]);
                    fence_proxy_async_smem();
                    bar_sync(10, kProducerThreads);
                    if (t == 0) mbar_arrive(&sm.kv_full[s]);
                    continue;
                }
                uint64_t* const landed = kv && partly ? &sm.v_raw[s] : &sm.kv_full[s];
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
                } else if (kv && partly) {
                    wait(landed, raw_phase >> s & 1);
                    raw_phase ^= 1u << s;
                    clean_rows<D>(dst, pc.common - t0, pc.seen - t0, t - 32, sm.bad[piece & 7]);
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
template <int D>
__device__ __forceinline__ void produce_gather(const ChunkAttnArgs& a, const Shape& sh, int waves, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D>;
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int lane = t & 31, w = t >> 5;
    // (a cache without pages may be a null pointer: copies of no bytes then start at q)
    const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.k_cache : a.q);
    const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.num_pages ? a.v_cache : a.q);
    const size_t row_stride = (size_t)a.kv_heads * D;
    Waiter wait{a.status};
    Walk walk(sm, waves);
    chunk::Piece pc;
    uint32_t fill = 0, sent = 0;                    // ring slots begun, and handed over
    bool bad_page = false;
    const int sub = lane / CH, chunk = lane % CH;

    auto hand_over = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&sm.kv_full[sent % L::kSlots]);
        ++sent;
    };
    for (uint32_t piece = 0; walk.next(a, sh, pc); ++piece) {
        if (t < 8) sm.bad[piece & 7][t] = 0;
        bar_sync(10, kProducerThreads);
        const int32_t* table = a.block_table + (size_t)pc.b * a.table_cols;
        auto look_up = [&](int tile) {              // one tile ahead
            const int pos = tile * kBN + 32 * w + lane;
            return tile < pc.last && pos < pc.seen ? __ldg(table + pos / a.page_size) : -1;
        };
        int id = look_up(pc.first);
        for (int tile = pc.first; tile < pc.last; ++tile) {
            const int t0 = tile * kBN;
            const Rows rows = rows_of(a, pc.hk, t0 + 32 * w + lane, pc.seen, id, row_stride, D);
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
                if (kv == 1 && t0 + kBN > pc.common) {
                    copy_rows<D>(dst, src, off, rows.exists, w, lane, pc.common - t0, sm.bad[piece & 7]);
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

template <int D>
__device__ __forceinline__ void query(const ChunkAttnArgs& a, const Shape& sh, int waves, Shared& sm, uint8_t* base, int t)
{
    using L = Layout<D>;
    constexpr int CH = D / 8, STEP = kQueryThreads / CH;   // chunks of a row; rows copied at once
    const int G = a.heads / a.kv_heads, c = t % CH;
    const int step_token = STEP / G, step_head = STEP - step_token * G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    Waiter wait{a.status};
    Walk walk(sm, waves);
    chunk::Piece pc;
    if (t == 0) chunk::clear_records(a, sh, gridDim.x, blockIdx.x);
    for (uint32_t piece = 0; walk.next(a, sh, pc); ++piece) {
        if (t == 0) chunk::record(a, sh, walk.line, pc);
        int r = t / CH, token = r / G, head = r - token * G;
        const __nv_bfloat16* src = q + ((size_t)pc.row0 * a.heads + pc.hk * G) * D + 8 * c;
        if (piece) wait(&sm.q_empty, (piece - 1) & 1);
#pragma unroll 4
        for (const int rows = pc.tokens * G; r < rows; r += STEP) {
            const bool there = a.scale != 0.f;
            cp16(smem_u32(base + (r >> 7) * L::kTile + sw128_chunk(r & 127, c, 128)), there ? src + ((size_t)token * a.heads + head) * D : q, there);
            token += step_token;
            head += step_head;
            if (head >= G) { head -= G; ++token; }
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full);
    }
    wait.finish();
}

// ------------------------------------------------------------------ the products
template <int D>
__device__ __forceinline__ void multiply(const ChunkAttnArgs& a, const Shape& sh, int waves, Shared& sm, uint8_t* base)
{
    using L = Layout<D>;
    Waiter wait{a.status};
    Walk walk(sm, waves);
    chunk::Piece pc;
    const uint32_t tm = sm.tmem, q0 = smem_u32(base), ring = q0 + L::kQ;
    const uint32_t id_s = idesc_bf16_f32(128, kBN, 0, 0, a.scale < 0.f), id_o = idesc_bf16_f32(128, D, 0, 1);
    // ring slot and phase of the next K and V tile; items of each stream so far
    uint32_t ks_ = 0, kp = 0, vs_ = 1, vp = 0, used[2] = {0, 0}, pieces[2] = {0, 0};   // (and pieces of each stream)
    auto advance = [](uint32_t& s, uint32_t& phase) {
        s += 2;
        if (s >= (uint32_t)L::kSlots) { s -= L::kSlots; phase ^= 1; }
    };
    uint32_t piece = 0;
    for (; walk.next(a, sh, pc); ++piece) {
        const int tiles = pc.last - pc.first, items = 2 * tiles;
        wait(&sm.q_full, piece & 1);
        // item i: stream i % 2, tile i / 2
        auto next_k = [&](int w) {                  // the slot of the item's keys, once they are there
            const uint32_t s = ks_;
            if (w == 0) wait(&sm.kv_full[s], kp);
            else advance(ks_, kp);
            return s;
        };
        auto scores = [&](int w, uint32_t s) {
            const uint64_t qd = kmajor_base(q0 + w * L::kTile), kd = kmajor_base(ring + s * L::kTile);
            if (wait.alive) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_bf16(tm + L::kColS + 128 * w, desc_off(qd, kmajor_off(128, ks)), desc_off(kd, kmajor_off(128, ks)), id_s, ks > 0);
            }
            umma_commit(&sm.s_full[w]);
        };
        auto scored = [&](int i, int w, uint32_t s) {
            if (w == 1) umma_commit(&sm.kv_empty[s]);
            if (i == items - 1) umma_commit(&sm.q_empty);
        };
        // The values of item i, and the stream's next scores right behind them: all that they need is waited for before the
        // weights are, and slots are given back after both.
        auto step = [&](int i, int w) {
            const bool more = i + 2 < items;
            const uint32_t s = vs_;
            if (w == 0) wait(&sm.kv_full[s], vp);
            else advance(vs_, vp);
            if (i == w) {                           // the stream's first products of the piece overwrite O
                if (pieces[w]) wait(&sm.o_free[w], (pieces[w] - 1) & 1);
                ++pieces[w];
            }
            const uint32_t k = more ? next_k(w) : 0;
            const uint64_t vd = mnmajor_base(ring + s * L::kTile, kBN);
            wait(&sm.p_full[w], used[w] & 1);
            ++used[w];
            tc_fence_after_sync();
            if (wait.alive) {
#pragma unroll
                for (int ks = 0; ks < kBN / 16; ++ks)
                    umma_bf16_tmem_a(tm + L::kColO + D * w, tm + L::kColS + 128 * w + 8 * ks, desc_off(vd, mnmajor_off(ks)), id_o, i > 1 || ks > 0);
            }
            if (more) scores(w, k);
            else umma_commit(&sm.o_done[w]);
            if (w == 1) umma_commit(&sm.kv_empty[s]);
            if (more) scored(i + 2, w, k);
        };
        // (one thread for all of it: with the whole warp in the waits and a thread elected for each
        // group of products their issue took 3000 cycles a tile; with a thread to each stream the streams' products mix, and each
        // waits longer for its own: 0.42 -> 0.50 ms for 2048 tokens after 16384)
        for (int w = 0; w < 2; ++w) {
            const uint32_t k = next_k(w);
            tc_fence_after_sync();
            scores(w, k);
            scored(w, w, k);
        }
        for (int i = 0; i < items; i += 2) {
            step(i, 0);
            step(i + 1, 1);
        }
    }
    for (int w = 0; w < 2; ++w)                     // no product or commit is in flight after this
        if (pieces[w]) wait(&sm.o_done[w], (pieces[w] - 1) & 1);
    wait.finish();
}

// ------------------------------------------------------------------ softmax and epilogue
// What a row that sees `sees` tokens has of the tile at t0: 128 bits, four words.
__device__ __forceinline__ void tile_mask(int sees, int t0, uint4 lost, uint32_t (&mw)[4])
{
    const uint32_t missing[4] = {lost.x, lost.y, lost.z, lost.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = sees - t0 - 32 * k;
        mw[k] = (n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u) & ~missing[k];
    }
}

template <int D>
__device__ __forceinline__ void softmax(const ChunkAttnArgs& a, const Shape& sh, int waves, Shared& sm, int t)
{
    using L = Layout<D>;
    const int lane = t & 31, warp = t >> 5, w = t >> 7, r = t & 127;   // stream and lane of tensor memory
    const int G = a.heads / a.kv_heads;
    const uint32_t quad = 32 * (warp & 3);                            // the lanes this warp reaches
    const uint32_t tS = tmem_addr(sm.tmem, quad, L::kColS + 128 * w), tO = tmem_addr(sm.tmem, quad, L::kColO + D * w);
    const float sc = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;  // scores in powers of two
    const float2 sc2 = make_float2(sc, sc);
    Waiter wait{a.status};
    Walk walk(sm, waves);
    chunk::Piece pc;
    uint32_t used = 0, done = 0;                       // items of this stream, tiles so far
    for (uint32_t piece = 0; walk.next(a, sh, pc); ++piece) {
        const int tiles = pc.last - pc.first;
        if (!pc.ok && t == 0) report_status(a.status, kDevBadSeqlens);
        // this thread's row of the unit, its token of the block, and how many tokens it sees
        const int rl = 128 * w + r, token = rl / G;
        const bool mine = token < pc.tokens;
        const int see = mine && pc.ok ? pc.common + token : 0;
        const bool busy = __any_sync(0xffffffffu, see != 0);
        // m in score units, before sc; a row that may see nothing never asks for another maximum
        float m = see ? -INFINITY : INFINITY, l = 0.f;
        bool begun = false;

        for (int i = 0; i < tiles; ++i) {
            const int t0 = (pc.first + i) * kBN;
            wait(&sm.s_full[w], used & 1);
            ++used;
            __syncwarp();
            tc_fence_after_sync();
            if (busy) {
                float xa[32], xb[32];
                tmem_ld32(tS, xa);
                const uint4 missing = *reinterpret_cast<const uint4*>(sm.missing[(done + i) & 7]);
                const bool all = t0 + kBN <= pc.common && !(missing.x | missing.y | missing.z | missing.w);
                tmem_wait_ld();
                // The quick form wants a maximum to begin with, in kTame's range, and no masks: a second form with masks costs the
                // loop more than it gives (0.412 -> 0.424 ms for 2048 tokens after 16384).
                bool again = !all || !begun || __any_sync(0xffffffffu, see && !(fabsf(m) * sc <= kTame));
                if (!again) {
                    // The weights are formed from the last maximum and stored over the scores unless one is past what
                    // may stand, which their sum tells: no maximum is looked for.
                    // x sc - m sc in one operation: m sc's rounding is a factor that a row's weights share, and
                    // up to kTame it is 2^-13 of a weight, below bf16's rounding, where the maximum changes.
                    const float2 off = make_float2(-m * sc, -m * sc);
                    auto weigh = [&](const float (&x)[32], float2& sum, uint32_t (&p)[16]) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 y = __ffma2_rn(make_float2(x[2 * k], x[2 * k + 1]), sc2, off);
                            const float2 e = make_float2(ex2(y.x), ex2(y.y));
                            sum = __fadd2_rn(sum, e);
                            p[k] = pack_bf16x2(e.x, e.y);
                        }
                    };
                    float2 sum = make_float2(0.f, 0.f);
                    uint32_t p[4][16];
                    tmem_ld32(tS + 32, xb);
                    weigh(xa, sum, p[0]);
                    tmem_wait_ld();
                    tmem_ld32(tS + 64, xa);
                    weigh(xb, sum, p[1]);
                    tmem_wait_ld();
                    tmem_ld32(tS + 96, xb);
                    weigh(xa, sum, p[2]);
                    tmem_wait_ld();
                    weigh(xb, sum, p[3]);
                    again = __any_sync(0xffffffffu, sum.x + sum.y > kMostSum);
                    if (!again) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_st16u(tS + 16 * c, p[c]);
                        l += sum.x + sum.y;
                    }
                }
                if (again) {
                    // masks, a first maximum, or one that has grown or is out of kTame's range: the maximum first, then the weights
                    // (word c's go to columns 16 c, over scores that have been read)
                    uint32_t mw[4];                 // which of the tokens the row sees
                    tile_mask(see, t0, missing, mw);
                    auto read = [&](int c, float (&x)[32]) {
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait_ld();
                        const uint32_t on = c == 0 ? mw[0] : c == 1 ? mw[1] : c == 2 ? mw[2] : mw[3];
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = on >> k & 1 ? x[k] : -INFINITY;
                    };
                    float top = -INFINITY, x[32];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        read(c, x);
                        top = fmaxf(top, max_of(x));
                    }
                    if (top == -INFINITY && (mw[0] | mw[1] | mw[2] | mw[3])) top = kLowest;
                    const bool grow = top > m;
                    const float f = grow ? ex2((m - top) * sc) : 1.f;  // 0 for the first maximum
                    l *= f;
                    if (begun && __any_sync(0xffffffffu, grow)) {      // (S is ready: the stream's last products into O are done)
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            tmem_ld32(tO + c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] *= f;
                            tmem_st32(tO + c, x);
                        }
                    }
                    if (grow) m = top;
                    // (x - m) sc in this order: the difference is exact where it matters, whatever the scores
                    const float2 off = make_float2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t p[16];
                        read(c, x);
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
        wait(&sm.o_done[w], piece & 1);
        __syncwarp();
        tc_fence_after_sync();
        bool bad = false;                           // non-finite values among the block's own tokens
        if (pc.last * kBN > pc.common) {
#pragma unroll
            for (int k = 0; k < 8; ++k) bad |= *const_cast<volatile uint32_t*>(&sm.bad[piece & 7][k]) != 0;
        }
        const float norm = pc.whole() ? (l == 0.f ? 0.f : 1.f / l) : 1.f, none = pc.whole() && m != -INFINITY ? NAN : 0.f;
        float* ws = attn::slot_of(a.workspace, sh, D, pc.slot);
        if (mine && !pc.whole()) {
            ws[rl] = m == -INFINITY ? m : fmaxf(m * sc, kLowest);
            ws[sh.BM + rl] = l;
        }
        // out's row of this thread (in rows of D), and of the four rows of its group of four lanes
        const int orow = mine ? (pc.row0 + token) * a.heads + pc.hk * G + rl - token * G : -1;
        int orows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) orows[k] = __shfl_sync(0xffffffffu, orow, (lane & ~3) + k);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float o[32];
            if (busy) {
                tmem_ld32(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = l == 0.f ? none : o[k] * norm;
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0.f;
            }
            if (bad && see) {                       // (token i of the block is bit i - 1: the first one is seen by all)
                for (int i = 0; i < token; ++i) {
                    if (!(sm.bad[piece & 7][i >> 5] >> (i & 31) & 1)) continue;
                    const int pos = pc.common + i, id = a.block_table[(size_t)pc.b * a.table_cols + pos / a.page_size];
                    if (id < 0 || id >= a.num_pages) continue;
                    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + (size_t)id * a.v_page_stride +
                                             ((size_t)(pos % a.page_size) * a.kv_heads + pc.hk) * D + c;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float x = __bfloat162float(v[k]);
                        if (!isfinite(x)) o[k] += x;
                    }
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
            } else if (mine) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    attn::slot_out(ws, sh.BM)[(size_t)((c + k) / 4) * sh.BM + rl] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free[w]);
    }
    wait.finish();
}

template <int D, bool kBoxes>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_tc_kernel(ChunkAttnArgs a, Shape sh, const __grid_constant__ Maps maps)
{
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t base[];   // all of it: the swizzled tiles start at 0
    Shared& sm = *reinterpret_cast<Shared*>(base + L::kShared);
    const int t = threadIdx.x, warp = t >> 5;
    const int waves = sh.ctas / (int)gridDim.x;
    if (warp < waves) {
        chunk::Line line;
        const bool good = line.begin(a, sh, gridDim.x, warp * gridDim.x + blockIdx.x, t & 31);
        if ((t & 31) == 0) sm.lines[warp] = line;
        if (!good && blockIdx.x == 0 && t == 0) report_status(a.status, kDevBadSeqlens);
    }
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
            mbar_init(&sm.o_free[i], 4);
        }
        mbar_init(&sm.q_full, kQueryThreads);
        mbar_init(&sm.q_empty, 1);
        mbar_fence_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax<D>(a, sh, waves, sm, t);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < 12) {
            if constexpr (kBoxes) produce_boxes<D>(a, sh, maps, waves, sm, base, t - kSoftmaxThreads);
            else produce_gather<D>(a, sh, waves, sm, base, t - kSoftmaxThreads);
        } else if (warp == 12) {
            if (elect_one()) multiply<D>(a, sh, waves, sm, base);
        } else {
            query<D>(a, sh, waves, sm, base, t - 13 * 32);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 12) tmem_dealloc(sm.tmem, 512);
}

// Several waves (see kda_chunk_attn.cuh) where the cache is larger than what they keep together, and blocks enough
// for it: a unit is cut in 16 parts at most.
Shape shape_of(const ChunkAttnArgs& a)
{
    const int TB = kBM / (a.heads / a.kv_heads);
    const double cache = 4. * a.num_pages * a.page_size * a.kv_heads * a.dim, units = ((double)a.tokens / TB + a.batch) * a.kv_heads;
    int waves = 1;
    while (waves < chunk::kMaxWaves && waves * chunk::kResident < cache && 2 * waves * kCtas <= 16 * units) waves *= 2;
    return {kBM, kBN, kCtas * waves, kHead};
}

template <int D, bool kBoxes>
cudaError_t launch(const ChunkAttnArgs& a, cudaStream_t stream)
{
    using L = Layout<D>;
    const auto kernel = chunk_attn_tc_kernel<D, kBoxes>;
    const Shape sh = shape_of(a);
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
    kernel<<<kCtas, kThreads, L::kBytes, stream>>>(a, sh, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return attn::launch_join<__nv_bfloat16, D>({a.workspace, a.out, a.heads, a.kv_heads}, sh, kBM, stream);
}

template <int D>
cudaError_t launch_dim(const ChunkAttnArgs& a, cudaStream_t stream)
{
    return in_boxes(a) ? launch<D, true>(a, stream) : launch<D, false>(a, stream);
}

}  // namespace

size_t chunk_attn_tc_workspace_bytes(const ChunkAttnArgs& a) { return attn::workspace_bytes(shape_of(a), a.dim); }

bool chunk_attn_tc_fits(const ChunkAttnArgs& a) { return chunk::line_fits(a, shape_of(a)); }

cudaError_t launch_chunk_attn_tc(const ChunkAttnArgs& a, cudaStream_t stream)
{
    return a.dim == 128 ? launch_dim<128>(a, stream) : launch_dim<64>(a, stream);
}

}  // namespace kda
