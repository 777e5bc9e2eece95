// spv_tiles.cuh -- attention over the paged cache in tiles of query rows: whole
// prompts, and drafted chains and trees of many rows a key head with scores and
// masks (spv_scores).  5th-generation tensor cores.
//
// Mathematics: as in spv_attention_warps.cuh.  The rows of an item -- a
// sequence, a tile of new tokens x query heads of a key head's group, a key head
// -- see slots of an interval each, so the item has the tiles of keys between
// the lowest and the highest slot that any of its rows sees, and masks are
// looked at only in tiles that some row does not see whole.
//
// What bounds it are the products, 4 D operations for a row and a key, and the
// exponentials beside them (a prompt reads its keys from the L2 after the first
// time).  One block an SM with an equal range of all tiles of all items, found
// from the lengths on the device; in it
//   * PAIR: 256 rows as two tiles of 128.  Four warps hold the first's rows, a
//     row a thread, four the second's.  Tiles of keys are 64 long, so that beside
//     the outputs of both (2 x 128 columns of tensor memory) two tiles of scores
//     of each fit: the next one's products are there when a thread has made its
//     weights, which go where their scores were, and their way through the tensor
//     cores is behind the exponentials.  (With tiles of 128 the warps waited for
//     them: 609 us for the first prompt below.)
//   * else 128 rows, of which two warps share each row's keys (few rows; and D =
//     256, whose outputs take half of tensor memory).  Scores stand in two
//     places in turn.  64 rows or fewer stand in tensor memory twice, 32 or fewer
//     four times, each copy with half or a quarter of a tile's keys (its weights
//     are zero elsewhere): all warps work whatever the number of rows, and the
//     copies are put together at the item's end;
//   * one warp works out the items, one issues the products, two ask for q, four K
//     and V in turn into one ring, a box a page by the copy engine, or row by row
//     (small pages; a sequence's last tile of V, whose slots past the end become
//     zero).  e4m3 lands as it is and is widened to f16 by the warp that asked for
//     it.
// Measured: a prompt of 8,192 tokens, 32 heads on 8 of 128, bf16, pages of 16: 538
// us, 1.0 PFLOP/s of the 1.9 that the products alone could have: for a tile of 64
// keys a thread's scores take 1,500 cycles (loads 240, maximum 400, exponentials
// and weights 450, waits for products 470).  Capped scores, bound by the
// polynomials: 883 us.  Distance biases 586, documents of 1,000 tokens 156, a
// window of 1,024 182, heads of 64 474, 16 heads of 256 536 us.  e4m3 772 us (heads
// of 64 640): widening K and V, four warps.  An item's beginning and end take some
// 12,000 cycles: the outputs 4,600, agreeing on the end 2,000, the next rows'
// intervals and q.
//
// O is only rescaled when a maximum has grown by more than 2^8 (2^7 for f16).
// The blocks' pieces of an item that they share are joined by a dependent
// launch, in their order.
//
// A weight of 0 and an infinity in V make NaN, which a row must not get from a
// slot that it does not see: rows whose result is not finite are computed again
// at the end of a block's range, key by key over what they see.
//
// Every wait is bounded; one that gives up records SPV_ERR_TIMEOUT in the
// workspace, ends the block in order and leaves NaN in all that it still had to
// write.
#pragma once

#include "spv_scored.cuh"
#include "spv_tcgen.cuh"
#include "spv_tma.cuh"

namespace spv {

constexpr int TILES_THREADS = 512;
constexpr int TILES_WARPS = TILES_THREADS / 32;
constexpr int TILES_PREPARE = 64;  // threads that bring q

struct TilesParams : ScoredParams {
    int32_t *timeouts;  // row_status, for waits that gave up
    int q_bf16;
};

// COPIES 0: PAIR.
template <typename C, int D, int COPIES> struct TilesShape {
    static constexpr bool PAIR = COPIES == 0;
    static constexpr bool WIDEN = sizeof(C) == 1;
    static constexpr bool ROWS_WIDEN = WIDEN && PAIR;            // the rows' threads bring q into f16's range, each its row
    static constexpr int PLACE = PAIR ? 64 : 128;                // columns from one place of scores to the next
    static constexpr int SUBS = PAIR ? 2 : 1, ROWS = PAIR ? 256 : 128 / (PAIR ? 1 : COPIES);
    static constexpr int KEYS = PAIR || D == 256 ? 64 : 128;     // of a tile
    static constexpr int OVERHEAD = PAIR ? 6 : 2;                // tiles that an item's beginning and end take as long as
    static constexpr int OF_COPY = KEYS / (PAIR ? 1 : COPIES);   // of them a copy's
    static constexpr int MINE = PAIR ? KEYS : OF_COPY / 2;       // and a thread's
    static constexpr int TILE = KEYS * D * 2, RAW = KEYS * D;    // bytes of K or V as multiplied, and of e4m3
    static constexpr int Q_SUB = 128 * D * 2, Q = SUBS * Q_SUB;
    static constexpr int Q_PLACES = !WIDEN && 2 * Q <= 64 * 1024 ? 2 : 1;
    static constexpr int ROOM = 224 * 1024 - Q_PLACES * Q;
    static constexpr int RAW_STAGES = !WIDEN ? 0 : (PAIR || D == 256 ? 32 : 48) * 1024 / RAW;
    static constexpr int FIT = (ROOM - RAW_STAGES * RAW) / TILE, MOST = WIDEN ? 8 : 10, STAGES = FIT < MOST ? FIT : MOST;
    static constexpr int K_AT = Q_PLACES * Q, RAW_AT = K_AT + STAGES * TILE, CTL_AT = RAW_AT + RAW_STAGES * RAW;
    static constexpr int ITEMS = (STAGES + RAW_STAGES) / 2 + 3;  // whose flags can be in use at once: an item has two tiles at least
    static constexpr int GROUP = PAIR ? 128 : 256;               // threads that belong to the same rows
};

// An item's tiles of keys: [from, to), and of each tile of rows; `seen`: the
// first slot that any of its rows sees.
struct TileLens : SeqLens {
    int from, to, lo[2], hi[2], seen;
};
using TileCursor = CursorOf<TileLens>;

// What the block has of an item, as one warp works it out and passes it to the others.
struct alignas(16) TileItem {
    int b, row_tile, h, flags;
    int ctx, fresh, total, t0;
    int t1, lo0, hi0, lo1;
    int hi1, pad[3];
};
enum TileFlags { ITEM_BAD = 1, ITEM_WHOLE = 2, ITEM_SECOND = 4, ITEM_END = 8 };  // ITEM_SECOND: a piece goes to the block's second place

template <typename S> struct TilesCtl {
    TileItem items[2];
    uint64_t item_full[2], item_empty[2];
    uint64_t full[S::STAGES], empty[S::STAGES], s_full[4], p_full[4], o_done[4], q_full[2], q_empty[2], spare;
    uint64_t q_raw[S::Q_PLACES];
    uint64_t raw_full[S::WIDEN ? 4 : 1][S::WIDEN ? S::RAW_STAGES : 1];  // of each loader warp's rows
    // what makes a missing page of an item matter, of items in turn (they are worked out two ahead): the first slot that any of
    // its rows sees, and the tiles that each tile of rows sees
    int seen[4], spans[S::PAIR ? 4 : 1][4];
    char bad[2][S::ITEMS];                                       // a page id outside the pool, for each group of row warps
    int stop[2], lost[2];
    uint32_t tmem;
    int dead;
    union {
        struct {
            TileCursor start;
            long long sums[TILES_WARPS];
        } find;                                                  // before the roles begin
        struct {
            union {
                alignas(16) int positions[S::SUBS][S::KEYS];     // of moved slots: of a tile's keys, for each group of row warps
                signed char depth[S::Q_PLACES][S::SUBS == 1 ? 64 : 1];  // else, of trees: per place of q the depth of each new token
            };
            float top[2][S::SUBS == 1 ? 256 : 1];                // maxima of the two halves, of a tile and the next; sums
            signed char q_power[S::WIDEN && !S::ROWS_WIDEN ? S::Q_PLACES * S::ROWS : 1];  // e4m3: the rows of q are stored times 2^q_power
        } at;
    };
};

template <typename Ctl> __device__ __forceinline__ bool tiles_wait(Ctl *ctl, uint64_t *bar, uint32_t parity, unsigned *err)
{
    bool ok = false;
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        if (mbar_try_wait(bar, parity)) {
            ok = true;
            break;
        }
        if ((i & 63) == 63 && *reinterpret_cast<volatile int *>(&ctl->dead)) break;
    }
    if (!ok && !*reinterpret_cast<volatile int *>(&ctl->dead)) {
        *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
        atomicExch(err, static_cast<unsigned>(STATUS_TIMEOUT));
    }
    return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ the cut of the work
__device__ __forceinline__ SeqLens tiles_lens(const TilesParams &p, int b)
{
    SeqLens s = seq_lens(p.w.ctx_lens, p.w.new_lens, b, p.w.T, p.c);
    if (p.sc.slot_pos && !s.bad && s.ctx + s.fresh > p.sc.pos_stride) {
        s.bad = true;
        s.total = 0;
    }
    return s;
}

// Slots [lo, hi) that new token t sees (not of a tree).
struct Interval {
    int lo, hi;
};
__device__ __forceinline__ Interval token_interval(const TilesParams &p, const SeqLens &s, int b, int t)
{
    Interval r{0, s.ctx + t + 1};
    if (p.sc.window > 0 && !p.sc.slot_pos) r.lo = max(0, s.ctx + t - p.sc.window + 1);
    const int64_t at = static_cast<int64_t>(b) * p.w.T + t;
    if (p.sc.first) r.lo = max(r.lo, __ldg(p.sc.first + at));
    if (p.sc.last) r.hi = max(r.hi, min(s.total, __ldg(p.sc.last + at)));
    return r;
}

// Tiles of the item's rows.  Where tokens have documents or prefixes a warp
// looks at them together, all lanes for the same item; else each lane may ask
// for an item of its own.
template <typename S> __device__ __forceinline__ TileLens item_tiles(const TilesParams &p, const SeqLens &s, int b, int row_tile, int lane)
{
    TileLens r;
    static_cast<SeqLens &>(r) = s;
    r.from = r.seen = 0x7fffffff;
    r.to = 0;
    const bool sliding = p.sc.window > 0 && !p.sc.slot_pos;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        r.lo[k] = r.hi[k] = 0;
        if (k >= S::SUBS) continue;
        const int r0 = row_tile * S::ROWS + 128 * k, r1 = min(r0 + 128, p.rows);
        if (r0 >= r1 || s.total == 0) continue;
        const int ta = r0 / p.group, tb = min((r1 - 1) / p.group, s.fresh - 1);
        if (ta > tb) continue;
        int lo, hi;
        if (!p.sc.first && !p.sc.last) {
            lo = sliding ? max(0, s.ctx + (p.parent ? 0 : ta) - p.sc.window + 1) : 0;
            hi = p.parent ? s.total : s.ctx + tb + 1;
        } else {
            lo = 0x7fffffff;
            hi = 0;
            for (int t = ta + lane; t <= tb; t += 32) {
                Interval x = token_interval(p, s, b, t);
                if (p.parent) {  // a node's depth is not known here: at least 0
                    x.lo = max(__ldg(p.sc.first + static_cast<int64_t>(b) * p.w.T + t), sliding ? max(0, s.ctx - p.sc.window + 1) : 0);
                    x.hi = s.total;
                }
                if (x.lo < x.hi) {
                    lo = min(lo, x.lo);
                    hi = max(hi, x.hi);
                }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            lo = max(lo, 0);
        }
        if (lo >= hi) continue;
        r.lo[k] = lo / S::KEYS;
        r.hi[k] = (hi + S::KEYS - 1) / S::KEYS;
        r.from = min(r.from, r.lo[k]);
        r.seen = min(r.seen, lo);
        r.to = max(r.to, r.hi[k]);
    }
    if (r.to == 0) r.from = 0;
    return r;
}
__device__ __forceinline__ int count_of(const TileLens &s) { return max(1, s.to - s.from); }
// An item's beginning and end -- its q, the first scores, writing the rows -- take about as long as OVERHEAD tiles, and the
// ranges are cut as if it had so many more, before the first.

// The block's range, by all its threads; `c` is the same for all.
template <typename S> __device__ TileCursor tiles_find(const TilesParams &p, TilesCtl<S> *ctl, int tid)
{
    const int lane = tid & 31, warp = tid >> 5, entries = p.w.B * p.w.row_tiles;
    const int each = (entries + TILES_WARPS - 1) / TILES_WARPS, e0 = warp * each, e1 = min(entries, e0 + each);
    const bool together = p.sc.first || p.sc.last;
    auto count32 = [&](int e) {  // tiles of a head of entry e + lane
        int mine = 0;
        if (!together) {
            if (e + lane < e1) {
                const int b = (e + lane) / p.w.row_tiles;
                mine = count_of(item_tiles<S>(p, tiles_lens(p, b), b, e + lane - b * p.w.row_tiles, lane));
            }
        } else {
            for (int i = 0; i < 32 && e + i < e1; ++i) {
                const int b = (e + i) / p.w.row_tiles;
                const int n = count_of(item_tiles<S>(p, tiles_lens(p, b), b, e + i - b * p.w.row_tiles, lane));
                if (i == lane) mine = n;
            }
        }
        return mine;
    };
    long long sum = 0;
    for (int e = e0; e < e1; e += 32) sum += count32(e) + (e + lane < e1 ? S::OVERHEAD : 0);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) ctl->find.sums[warp] = sum * p.c.kv_heads;
    __syncthreads();
    TileCursor c{};
    long long before = 0, mine = ctl->find.sums[warp];
    for (int i = 0; i < TILES_WARPS; ++i) {
        if (i < warp) before += ctl->find.sums[i];
        c.all += ctl->find.sums[i];
    }
    c.blocks = c.all < gridDim.x ? static_cast<int>(c.all) : static_cast<int>(gridDim.x);
    const int block = blockIdx.x;
    if (block < c.blocks) {
        c.part = quotient(c.all, c.blocks);
        c.more = static_cast<int>(c.all - c.part * c.blocks);
        c.at = range_begin(c, block);
        c.end = range_begin(c, block + 1);
        if (c.at >= before && c.at < before + mine) {
            for (int e = e0; e < e1; e += 32) {
                const int n = count32(e), units = n + (e + lane < e1 ? S::OVERHEAD : 0);
                int upto = units;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const unsigned here = __ballot_sync(0xffffffffu, before + static_cast<long long>(upto) * p.c.kv_heads > c.at);
                if (here) {
                    const int l = __ffs(here) - 1;
                    const int tiles = __shfl_sync(0xffffffffu, n, l);
                    before += static_cast<long long>(__shfl_sync(0xffffffffu, upto - units, l)) * p.c.kv_heads;
                    c.tiles = tiles;
                    c.b = (e + l) / p.w.row_tiles;
                    c.row_tile = e + l - c.b * p.w.row_tiles;
                    c.h = static_cast<int>(quotient(c.at - before, tiles + S::OVERHEAD));
                    c.first = before + static_cast<long long>(c.h) * (tiles + S::OVERHEAD) + S::OVERHEAD;
                    if (c.at < c.first) c.at = c.first < c.end ? c.first : c.end;
                    if (lane == 0) ctl->find.start = c;
                    break;
                }
                before += static_cast<long long>(__shfl_sync(0xffffffffu, upto, 31)) * p.c.kv_heads;
            }
        }
    }
    __syncthreads();
    if (block < c.blocks) {
        c = ctl->find.start;
        c.s = item_tiles<S>(p, tiles_lens(p, c.b), c.b, c.row_tile, lane);
    }
    __syncthreads();  // this place is free
    return c;
}
// The same by one warp, slowly, for what is seldom done at a range's end.
template <typename S> __device__ __noinline__ TileCursor tiles_find_again(const TilesParams &p, int lane)
{
    TileCursor c{};
    long long before = 0;
    const int entries = p.w.B * p.w.row_tiles;
    for (int pass = 0; pass < 2; ++pass) {
        before = 0;
        for (int e = 0; e < entries; ++e) {
            c.b = e / p.w.row_tiles;
            c.row_tile = e - c.b * p.w.row_tiles;
            c.s = item_tiles<S>(p, tiles_lens(p, c.b), c.b, c.row_tile, lane);
            c.tiles = count_of(c.s);
            const long long units = static_cast<long long>(c.tiles + S::OVERHEAD) * p.c.kv_heads;
            if (pass == 1 && before + units > c.at) break;
            before += units;
        }
        if (pass == 0) {
            c.all = before;
            c.blocks = c.all < gridDim.x ? static_cast<int>(c.all) : static_cast<int>(gridDim.x);
            c.part = quotient(c.all, c.blocks);
            c.more = static_cast<int>(c.all - c.part * c.blocks);
            c.at = range_begin(c, blockIdx.x);
            c.end = range_begin(c, blockIdx.x + 1);
        }
    }
    c.h = static_cast<int>(quotient(c.at - before, c.tiles + S::OVERHEAD));
    c.first = before + static_cast<long long>(c.h) * (c.tiles + S::OVERHEAD) + S::OVERHEAD;
    if (c.at < c.first) c.at = c.first < c.end ? c.first : c.end;
    return c;
}
// To the next item; a whole warp.
template <typename S> __device__ __forceinline__ void tiles_next(TileCursor &c, const TilesParams &p, int lane)
{
    c.first += c.tiles + S::OVERHEAD;
    c.at = c.first;
    if (++c.h < p.c.kv_heads) return;
    c.h = 0;
    if (++c.row_tile == p.w.row_tiles) {
        c.row_tile = 0;
        if (++c.b == p.w.B) return;  // the end of everything
    }
    c.s = item_tiles<S>(p, tiles_lens(p, c.b), c.b, c.row_tile, lane);
    c.tiles = count_of(c.s);
}
// The block's tiles of the cursor's item: [first, last), none for an item without keys.
__device__ __forceinline__ int tiles_first(const TileCursor &c) { return c.s.from + static_cast<int>(c.at - c.first); }
__device__ __forceinline__ int tiles_last(const TileCursor &c)
{
    if (c.s.to == 0) return tiles_first(c);
    const long long e = c.first + c.tiles;
    return c.s.from + static_cast<int>((c.end < e ? c.end : e) - c.first);
}
__device__ __forceinline__ bool item_whole(const TileCursor &c) { return c.s.to == 0 || (c.at == c.first && c.end >= c.first + c.tiles); }

// 16-byte chunk `chunk` of row `row` in an operand of ROWS rows.
template <int ROWS> __device__ __forceinline__ uint32_t tile_at(int row, int chunk)
{
    return (chunk >> 3) * (ROWS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// ------------------------------------------------------------------ items
// One warp works out the block's items, two ahead of the others, and notes the
// shared ones.  (Each role by itself, the next item's lengths, spans and
// divisions took all of them thousands of cycles, much of it fetching the code.)
template <typename S> __device__ void tiles_items(const TilesParams &p, TileCursor c, TilesCtl<S> *ctl, unsigned *err, int lane)
{
    const long long begin = c.at;
    int k = 0;
    for (;; tiles_next<S>(c, p, lane), ++k) {
        const bool end = c.at >= c.end;
        if (k >= 2 && !tiles_wait(ctl, &ctl->item_empty[k & 1], (k / 2 - 1) & 1, err)) return;
        if (lane == 0) {
            TileItem &it = ctl->items[k & 1];
            it.b = c.b, it.row_tile = c.row_tile, it.h = c.h;
            it.flags = end ? ITEM_END : (c.s.bad ? ITEM_BAD : 0) | (item_whole(c) ? ITEM_WHOLE : 0) | (c.first < begin ? 0 : ITEM_SECOND);
            it.ctx = c.s.ctx, it.fresh = c.s.fresh, it.total = c.s.total;
            it.t0 = tiles_first(c), it.t1 = tiles_last(c);
            it.lo0 = c.s.lo[0], it.hi0 = c.s.hi[0], it.lo1 = c.s.lo[1], it.hi1 = c.s.hi[1];
            ctl->seen[k & 3] = c.s.seen;
            if (S::PAIR) {
                int(&span)[4] = ctl->spans[S::PAIR ? k & 3 : 0];
                span[0] = c.s.lo[0], span[1] = c.s.hi[0], span[2] = c.s.lo[1], span[3] = c.s.hi[1];
            }
            mbar_arrive(&ctl->item_full[k & 1]);
            if (!end && !item_whole(c))
                note_split(p, c, AttRows{c.b, c.h, c.row_tile * S::ROWS, min(S::ROWS, p.rows - c.row_tile * S::ROWS)}, begin, 0);
        }
        __syncwarp();
        if (end) return;
    }
}
// Whether the phase of `parity` is complete, without a wait.
__device__ __forceinline__ bool mbar_done(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}
// The block's item k, for a whole warp; false at the end, or after a wait gave up.
constexpr int TILES_TAKERS = 8 + 1 + 2 + 4;  // warps that take every item
template <typename Ctl> __device__ __forceinline__ bool take_item(Ctl *ctl, int k, TileItem *it, unsigned *err, int lane)
{
    if (!tiles_wait(ctl, &ctl->item_full[k & 1], (k >> 1) & 1, err)) return false;
    const int4 *from = reinterpret_cast<const int4 *>(&ctl->items[k & 1]);
    const int4 x = from[0], y = from[1], z = from[2];
    // the same in all lanes, and the compiler is told so: what depends on them is then decided once for the warp
    it->b = same_in_warp(x.x), it->row_tile = same_in_warp(x.y), it->h = same_in_warp(x.z), it->flags = same_in_warp(x.w);
    it->ctx = same_in_warp(y.x), it->fresh = same_in_warp(y.y), it->total = same_in_warp(y.z), it->t0 = same_in_warp(y.w);
    it->t1 = same_in_warp(z.x), it->lo0 = same_in_warp(z.y), it->hi0 = same_in_warp(z.z), it->lo1 = same_in_warp(z.w);
    it->hi1 = same_in_warp(from[3].x);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->item_empty[k & 1]);
    return !(it->flags & ITEM_END);
}

// ------------------------------------------------------------------ K and V
// Four warps: tiles of K and V in turn, each warp a quarter of their slots.
template <typename C, int D, int COPIES, typename S = TilesShape<C, D, COPIES>>
__device__ void tiles_load(const TilesParams &p, char *smem, TilesCtl<S> *ctl, unsigned *err, int lt,
                           const CUtensorMap *map_k, const CUtensorMap *map_v)
{
    constexpr int CH = D * static_cast<int>(sizeof(C)) / 16, RPI = 32 / CH, NST = S::STAGES, KEYS = S::KEYS, WARP_ROWS = KEYS / 4;
    constexpr int RST = S::WIDEN ? S::RAW_STAGES : 1;
    const int lane = lt & 31, w = lt >> 5, chunk = lane % CH, sub = lane / CH;
    const uint32_t base = smem_u32(smem);
    const int mask = (1 << p.c.page_shift) - 1;
    int st = 0, pass = 1, filled = 0;  // the ring's place of the next tile, and the parity of its being free (at first it is); places filled
    int raw = 0, waiting = 0;          // e4m3: the place of the next raw tile; raw tiles not widened yet
    int rows[RST];          // e4m3: slots of this warp that exist, of the raw tiles in turn
    bool ok = true;
    auto free_place = [&]() { return tiles_wait(ctl, &ctl->empty[st], pass, err); };
    auto step = [&]() {
        if (++st == NST) st = 0, pass ^= 1;
        if (filled < NST) ++filled;
    };

    // e4m3: widens the oldest raw tile, each warp the rows that it brought; `place` of raw ones, passing parity.
    int oldest = 0, oldest_pass = 0;
    auto widen = [&]() -> bool {
        if (map_k) {
            if (!tiles_wait(ctl, &ctl->raw_full[S::WIDEN ? w : 0][oldest], oldest_pass, err)) return false;
        } else {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        }
        if (!free_place()) return false;
        const char *from = smem + S::RAW_AT + oldest * S::RAW;
        char *to = smem + S::K_AT + st * S::TILE;
        const int there = rows[0];
#pragma unroll 4
        for (int i = 0; i < WARP_ROWS / RPI; ++i) {
            const int r = i * RPI + sub, row = WARP_ROWS * w + r;
            uint4 x = *reinterpret_cast<const uint4 *>(from + row * D + chunk * 16);
            if (r >= there) x = make_uint4(0, 0, 0, 0);  // behind the sequence's end: anything
            const uint32_t b[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = e4m3x2_to_f16x2(b[k] & 0xffffu);
                y[2 * k + 1] = e4m3x2_to_f16x2(b[k] >> 16);
            }
            const bool swap = (chunk >> 2) & 1;  // lanes of two panels store their halves in opposite order
            const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
            *reinterpret_cast<uint4 *>(to + tile_at<KEYS>(row, 2 * chunk + swap)) = swap ? hi : lo;
            *reinterpret_cast<uint4 *>(to + tile_at<KEYS>(row, 2 * chunk + !swap)) = swap ? lo : hi;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->full[st]);
        step();
        if (++oldest == RST) oldest = 0, oldest_pass ^= 1;
        --waiting;
#pragma unroll
        for (int i = 0; i + 1 < RST; ++i) rows[i] = rows[i + 1];
        return true;
    };

    TileItem it;
    int item = 0;
    for (int k = 0; ok; ++k) {
        // The next item may come only when the rows have ended one whose tiles are still raw here: these go first.
        if (S::WIDEN)
            while (ok && waiting > 0 && !__all_sync(0xffffffffu, mbar_done(&ctl->item_full[k & 1], (k >> 1) & 1))) ok = widen();
        if (!ok || !take_item(ctl, k, &it, err, lane)) break;
        const int t0 = it.t0, t1 = it.t1;
        if (t0 == t1) continue;
        const int32_t *table = p.c.table + static_cast<int64_t>(it.b) * p.c.max_pages;
        const int flags = item;
        if (++item == S::ITEMS) item = 0;
        // The page of this slot, in this tile, is outside the pool: that matters from the first slot that is seen on, and to the
        // groups of row warps that see the tile.  (One that does not may be done with the item, and its flag another item's.)
        auto flag = [&](int slot, int tile) {
            if (slot >> p.c.page_shift < ctl->seen[k & 3] >> p.c.page_shift) return;
            const int(&span)[4] = ctl->spans[S::PAIR ? k & 3 : 0];
            if (!S::PAIR || (tile >= span[0] && tile < span[1])) *reinterpret_cast<volatile char *>(&ctl->bad[0][flags]) = 1;
            if (S::PAIR && tile >= span[2] && tile < span[3]) *reinterpret_cast<volatile char *>(&ctl->bad[1][flags]) = 1;
        };
        // With maps each warp asks the copy engine for its slots: a box a page (or what the warp has of a larger one), of 64
        // elements, or e4m3's whole rows; a lane each.  (A lane's takes 80 to 100 cycles: from one warp, 16 of a tile of K
        // and 16 of V took longer than the tile's products.)
        constexpr int PANELS = S::WIDEN ? 1 : D / 64;
        const int box_slots = min(mask + 1, S::WIDEN ? WARP_ROWS : KEYS);
        const int boxes = S::WIDEN ? WARP_ROWS / box_slots : KEYS / box_slots * PANELS;
        const int quarter = S::WIDEN ? boxes : max(1, boxes >> 2), box = S::WIDEN ? lane : w * quarter + lane;
        const int boxes_here = max(0, min(quarter, S::WIDEN ? boxes : boxes - w * quarter));
        const bool asks = map_k && lane < boxes_here;
        const int box_slot = (S::WIDEN ? WARP_ROWS * w : 0) + box / PANELS * box_slots;
        auto lookup = [&](int tile) {  // the page id of this lane's box or row of a tile, unchecked; -1: no such row
            const int j = tile * KEYS + (map_k ? box_slot : WARP_ROWS * w + lane);
            return (map_k ? asks : lane < WARP_ROWS) && tile >= t0 && j < it.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
        };
        int next = lookup(t1 - 1);
        for (int tile = t1 - 1; ok && tile >= t0; --tile) {
            const int j0 = tile * KEYS, page = next;
            next = lookup(tile - 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const PoolView &pool = kv ? p.c.v : p.c.k;
                if (S::WIDEN && waiting == RST && !(ok = widen())) break;
                if (map_k && (S::WIDEN || !kv || j0 + KEYS <= it.total)) {
                    const int slot = j0 + box_slot;
                    if (asks && slot < it.total && static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages)) flag(slot, tile);
                    uint64_t *bar;
                    uint32_t to;
                    if constexpr (S::WIDEN) {
                        bar = &ctl->raw_full[w][raw];
                        to = base + S::RAW_AT + raw * S::RAW + box_slot * D;
                        fence_async_shared();  // its last bytes have been read
                        __syncwarp();
                    } else {
                        if (!(ok = free_place())) break;
                        bar = &ctl->full[st];
                        to = base + S::K_AT + st * S::TILE + (box % PANELS) * (KEYS * 128) + box / PANELS * box_slots * 128;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar, boxes_here * box_slots * (S::WIDEN ? D : 128));
                    __syncwarp();
                    if (asks) tma_box(to, kv ? map_v : map_k, S::WIDEN ? 0 : (box % PANELS) * 64, slot & mask, it.h, page, bar);
                    __syncwarp();
                } else {
                    int pg = page;
                    if (map_k) {  // the last tile of V by rows: slots behind the end become zero
                        const int j = j0 + WARP_ROWS * w + lane;
                        pg = lane < WARP_ROWS && j < it.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
                    }
                    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.c.num_pages)) {
                        if (lane < WARP_ROWS && j0 + WARP_ROWS * w + lane < it.total) flag(j0 + WARP_ROWS * w + lane, tile);
                        pg = -1;
                    }
                    const int64_t mine = pg < 0 ? -1 : pg * pool.page_stride + ((j0 + WARP_ROWS * w + lane) & mask) * pool.slot_stride;
                    const char *from = pool.base + it.h * pool.head_stride + chunk * 16;
                    if (!S::WIDEN && !(ok = free_place())) break;
                    const uint32_t to = base + (S::WIDEN ? S::RAW_AT + raw * S::RAW : S::K_AT + st * S::TILE);
#pragma unroll 2
                    for (int i = 0; i < WARP_ROWS / RPI; ++i) {
                        const int row = WARP_ROWS * w + i * RPI + sub;
                        const int64_t at = __shfl_sync(0xffffffffu, mine, i * RPI + sub);
                        cp_async16_zfill(to + (S::WIDEN ? row * D + chunk * 16 : tile_at<KEYS>(row, chunk)), at < 0 ? pool.base : from + at,
                                         at < 0 ? 0 : 16);
                    }
                    if (!S::WIDEN) {  // the fence for the tensor cores is the writers'
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->full[st]);
                    }
                }
                if constexpr (S::WIDEN) {
                    rows[0] = waiting == 0 ? it.total - j0 - WARP_ROWS * w : rows[0];
#pragma unroll
                    for (int i = 1; i < RST; ++i) rows[i] = waiting == i ? it.total - j0 - WARP_ROWS * w : rows[i];
                    ++waiting;
                    if (++raw == RST) raw = 0;
                } else {
                    step();
                }
            }
        }
    }
    if (S::WIDEN)  // the tiles still on their way
        while (ok && waiting > 0) ok = widen();
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the copy engine's, before the block may end: nobody else may have waited for them
    if (map_k && S::WIDEN) {
        for (; waiting > 0; --waiting) {
            mbar_drain(&ctl->raw_full[S::WIDEN ? w : 0][oldest], oldest_pass);
            if (++oldest == RST) oldest = 0, oldest_pass ^= 1;
        }
    } else if (map_k) {
        for (; filled > 0; --filled) {
            if (--st < 0) st = NST - 1, pass ^= 1;
            mbar_drain(&ctl->full[st], pass ^ 1);
        }
    }
}

// ------------------------------------------------------------------ products
// One warp.
template <typename C, int D, int COPIES, typename S = TilesShape<C, D, COPIES>>
__device__ void tiles_multiply(char *smem, TilesCtl<S> *ctl, unsigned *err, int lane)
{
    constexpr bool BF16 = std::is_same<C, __nv_bfloat16>::value, PAIR = S::PAIR;
    constexpr uint32_t QK = mma_shape(BF16, false, S::KEYS), PV = mma_shape(BF16, true, D);
    constexpr int NST = S::STAGES, KEYS = S::KEYS;
    // all values here are the same in all lanes, and the compiler is told so
    const uint32_t base = smem_u32(smem), tmem = same_in_warp(ctl->tmem);
    int st = 0, phase = 0;             // the ring's place and pass of the next tile of K; V's is the one behind it
    int item = 0, turn0 = 0, turn1 = 0, out0 = 0, out1 = 0;  // which place is next, for scores and for outputs
    uint32_t passes = 0;               // bit i: parity of the weights' barrier of place i
    auto after = [&](int x) { return x + 1 == NST ? 0 : x + 1; };
    TileItem it;
    for (int k = 0; take_item(ctl, k, &it, err, lane); ++k) {
        const int t0 = same_in_warp(it.t0), tiles = same_in_warp(it.t1) - t0;
        if (tiles == 0) continue;
        const int place = S::Q_PLACES == 1 ? 0 : item & 1;
        if (!tiles_wait(ctl, &ctl->q_full[place], (item / S::Q_PLACES) & 1, err)) return;
        ++item;
        const uint32_t q0 = desc_low(base + place * S::Q, 16);
        // s: the tile of rows (PAIR; else 0).  Its tiles of keys have two places of scores in turn.
        auto scores = [&](int s, int k_st) {
            tc_fence_after();
            const int place = s * 2 + (PAIR && s ? turn1 : turn0);
            const uint32_t q = q0 + s * (S::Q_SUB >> 4), k = desc_low(base + S::K_AT + k_st * S::TILE, 16), to = tmem + place * S::PLACE;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                warp_mma<QK>(to, q + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4), k + (((ks >> 2) * (KEYS * 128) + (ks & 3) * 32) >> 4), ks > 0);
            warp_commit(&ctl->s_full[place]);
            (PAIR && s ? turn1 : turn0) ^= 1;
        };
        auto outputs = [&](int s, int v_st, bool add) {
            const int place = s * 2 + (PAIR && s ? out1 : out0);
            const uint32_t o = tmem + 256 + s * 128, w = tmem + place * S::PLACE, v = desc_low(base + S::K_AT + v_st * S::TILE, KEYS * 128);
            if (!tiles_wait(ctl, &ctl->p_full[place], passes >> place & 1, err)) return false;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < KEYS / 16; ++ks)
                warp_mma_ta<PV>(o, w + 16 * ks / S::MINE * S::MINE + 16 * ks % S::MINE / 2, v + ks * (2048 >> 4), add || ks > 0);
            passes ^= 1u << place;
            warp_commit(&ctl->o_done[place]);
            (PAIR && s ? out1 : out0) ^= 1;
            return true;
        };
        auto full = [&](int place, int pass) { return tiles_wait(ctl, &ctl->full[place], pass, err); };
        const int lo0 = PAIR ? it.lo0 : t0, hi0 = PAIR ? it.hi0 : t0 + tiles, lo1 = it.lo1, hi1 = it.hi1;
        bool begun0 = false, begun1 = false, pending0 = false, pending1 = false;
        int v_st = 0, v_pass = 0;
        for (int i = 0; i <= tiles; ++i) {  // the scores of a tile, and the outputs of the one before
            const bool keys = i < tiles;
            const int tile = t0 + tiles - 1 - i;  // from the last: a bias that falls with the distance has its largest scores there
            const bool here0 = keys && tile >= lo0 && tile < hi0, here1 = PAIR && keys && tile >= lo1 && tile < hi1;
            if (keys) {
                if (!full(st, phase)) return;
                if (here0) scores(0, st);
                if (here1) scores(1, st);
                warp_commit(&ctl->empty[st]);
                if (i == tiles - 1) warp_commit(&ctl->q_empty[place]);
            }
            if (i > 0) {
                if (!full(v_st, v_pass)) return;
                if (pending0) {
                    if (!outputs(0, v_st, begun0)) return;
                    begun0 = true;
                }
                if (pending1) {
                    if (!outputs(1, v_st, begun1)) return;
                    begun1 = true;
                }
                warp_commit(&ctl->empty[v_st]);
            }
            pending0 = here0;
            pending1 = here1;
            st = after(st);
            if (st == 0) phase ^= 1;
            v_st = st, v_pass = phase;
            st = after(st);
            if (st == 0) phase ^= 1;
        }
        // one turn more than tiles
        if (st == 0) phase ^= 1;
        st = st == 0 ? NST - 1 : st - 1;
        if (st == 0) phase ^= 1;
        st = st == 0 ? NST - 1 : st - 1;
    }
}

// ------------------------------------------------------------------ q
// Two warps, an item ahead of the others where there is room: q, and of trees
// the depths of the new tokens.  The copy engine brings it where a tile's rows
// are whole tokens (the threads, some 20 instructions for 16 bytes, took 18,000
// cycles for 256 rows); e4m3 caches: it is then multiplied into f16's range where
// it lies, in pairs of tiles by the rows' threads, a row each (889 us for 8,192
// tokens when these two warps did it, 769 since).
template <typename C, int D, int COPIES, typename S = TilesShape<C, D, COPIES>>
__device__ void tiles_prepare(const TilesParams &p, char *smem, TilesCtl<S> *ctl, unsigned *err, int lt, const CUtensorMap *map_q)
{
    const int lane = lt & 31;
    const uint32_t base = smem_u32(smem);
    constexpr int CH = D / 8, STEP = TILES_PREPARE / CH, TIMES = S::PAIR ? 1 : COPIES;  // rows at a time, places of each row
    const int ch = lt % CH, first = lt / CH;
    const int step_t = STEP / p.group, step_g = STEP - step_t * p.group;
    const int64_t token = static_cast<int64_t>(p.q_heads) * D * 2;
    TileItem it;
    int item = 0;
    for (int k = 0; take_item(ctl, k, &it, err, lane); ++k) {
        if (it.t0 == it.t1) continue;
        if (item == p.give_up.item && static_cast<int>(blockIdx.x) == p.give_up.block) {  // the self-test
            *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
            atomicExch(err, static_cast<unsigned>(STATUS_TIMEOUT));
            break;
        }
        const int place = item % S::Q_PLACES, row0 = it.row_tile * S::ROWS, live = min(S::ROWS, p.rows - row0);
        if (item >= S::Q_PLACES && !tiles_wait(ctl, &ctl->q_empty[place], (item / S::Q_PLACES - 1) & 1, err)) break;
        if constexpr (!S::PAIR) {
            if (p.parent && p.sc.slopes && !p.sc.slot_pos)
                for (int t = lt; t < it.fresh; t += TILES_PREPARE) {
                    SeqLens s{it.ctx, it.fresh, it.total, false};
                    ctl->at.depth[place][t] =
                        static_cast<signed char>(token_view(p.sc, p.parent + static_cast<int64_t>(it.b) * p.w.T, s, it.b, p.w.T, t).depth);
                }
        }
        char *to = smem + place * S::Q;
        const uint32_t to32 = base + place * S::Q;
        if (map_q) {
            constexpr int PANELS = D / 64, PARTS = S::PAIR ? 2 : COPIES;  // a box each: 64 elements of 128 rows, or of a copy's
            uint64_t *bar = S::WIDEN ? &ctl->q_raw[place] : &ctl->q_full[place];
            if (lt == 0) mbar_arrive_expect_tx(bar, S::Q);
            __syncwarp();
            if (lt < PANELS * PARTS) {
                const int panel = lt % PANELS, part = lt / PANELS;
                tma_box(to32 + (S::PAIR ? part * S::Q_SUB : part * S::ROWS * 128) + panel * (128 * 128), map_q, panel * 64, it.h * p.group,
                        (row0 + (S::PAIR ? part * 128 : 0)) / p.group, it.b, bar);
            }
            __syncwarp();
            if (S::ROWS_WIDEN) {  // the rows wait for it
                ++item;
                continue;
            }
            if (S::WIDEN) {
                if (!tiles_wait(ctl, bar, (item / S::Q_PLACES) & 1, err)) break;
            } else if (lt != 0) {
                mbar_arrive(bar);
            }
        } else {
            // rows first, first + STEP, ...: their tokens and heads, without a division each
            int t = (row0 + first) / p.group, g = row0 + first - t * p.group;
            const char *row = static_cast<const char *>(p.q) + (static_cast<int64_t>(it.b) * p.w.T * p.q_heads + it.h * p.group) * (D * 2) + ch * 16;
#pragma unroll 4
            for (int r = first; r < S::ROWS; r += STEP) {
                const bool there = r < live && t < it.fresh;
                const char *from = there ? row + t * token + g * (D * 2) : static_cast<const char *>(p.q);
                t += step_t, g += step_g;
                if (g >= p.group) g -= p.group, ++t;
#pragma unroll
                for (int i = 0; i < TIMES; ++i)
                    cp_async16_zfill(to32 + (r >> 7) * S::Q_SUB + tile_at<128>((r & 127) + i * S::ROWS, ch), from, there ? 16 : 0);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        if constexpr (S::ROWS_WIDEN) {
            mbar_arrive(&ctl->q_raw[place]);
            ++item;
            continue;
        }
        if constexpr (S::WIDEN && !S::ROWS_WIDEN) {
#pragma unroll 2
            for (int r = first; r < S::ROWS; r += STEP) {  // every thread the same number of times
                char *at = to + (r >> 7) * S::Q_SUB;
                const uint4 in = *reinterpret_cast<const uint4 *>(at + tile_at<128>(r & 127, ch));
                float x[8], top = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = p.q_bf16 ? Num<__nv_bfloat16>::up(reinterpret_cast<const __nv_bfloat16 *>(&in)[e])
                                    : Num<__half>::up(reinterpret_cast<const __half *>(&in)[e]);
                    top = fabsf(x[e]) < CUDART_INF_F ? fmaxf(top, fabsf(x[e])) : top;
                }
#pragma unroll
                for (int o = CH / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // the largest below 2^15 (the exponent of a number that is not normal counts as the smallest's)
                const int e2 = top > 0.0f ? max(-120, min(120, 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127))) : 0;
                const float up = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
                if (ch == 0) ctl->at.q_power[place * S::ROWS + r] = static_cast<signed char>(e2);
                const uint4 y = make_uint4(pack_mma<__half>(x[0] * up, x[1] * up), pack_mma<__half>(x[2] * up, x[3] * up),
                                           pack_mma<__half>(x[4] * up, x[5] * up), pack_mma<__half>(x[6] * up, x[7] * up));
#pragma unroll
                for (int i = 0; i < TIMES; ++i) *reinterpret_cast<uint4 *>(at + tile_at<128>((r & 127) + i * S::ROWS, ch)) = y;
            }
        }
        if (S::WIDEN || !map_q) {
            fence_async_shared();
            mbar_arrive(&ctl->q_full[place]);
        }
        ++item;
    }
    // the copy engine's, before the block may end: nobody else may have waited for it
    if (map_q && *reinterpret_cast<volatile int *>(&ctl->dead))
        for (int i = max(0, item - S::Q_PLACES); i <= item; ++i) {
            uint64_t *bar = S::WIDEN ? &ctl->q_raw[i % S::Q_PLACES] : &ctl->q_full[i % S::Q_PLACES];
            mbar_drain(bar, (i / S::Q_PLACES) & 1);
        }
}

// ------------------------------------------------------------------ rows
// Multiplies row r of q, where it lies, into f16's range by a power of two, and returns that power's inverse.
template <typename T, int D> __device__ __forceinline__ float widen_row(char *rows, int r)
{
    constexpr uint32_t INF = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    uint32_t top = 0;  // of two columns of elements, as bits: finite ones are ordered as their bits
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(rows + tile_at<128>(r, c));
        const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & __vcmpltu2(w[i], INF));
    }
    const uint16_t most = static_cast<uint16_t>(max(top & 0xffffu, top >> 16));
    const float largest = Num<T>::up(*reinterpret_cast<const T *>(&most));
    // the largest below 2^15 (the exponent of a number that is not normal counts as the smallest's)
    const int e2 = largest > 0.0f ? max(-120, min(120, 14 - (static_cast<int>(__float_as_uint(largest) >> 23) - 127))) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
#pragma unroll 2
    for (int c = 0; c < D / 8; ++c) {
        uint4 *at = reinterpret_cast<uint4 *>(rows + tile_at<128>(r, c));
        const uint4 x = *at;
        const T *y = reinterpret_cast<const T *>(&x);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_mma<__half>(Num<T>::up(y[2 * i]) * up, Num<T>::up(y[2 * i + 1]) * up);
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
}
// All threads that have rows of the same tile of rows.
template <int N> __device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(N) : "memory"); }
// The two warps that share rows.
__device__ __forceinline__ void halves_sync(int w) { asm volatile("bar.sync %0, 64;" ::"r"(3 + w) : "memory"); }

__device__ __forceinline__ void store_32bytes(void *at, const uint32_t (&y)[8])
{
    if ((reinterpret_cast<uintptr_t>(at) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
                     "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(at)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4 *>(at)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

// Rows [r_from, r_from + r_count) of the cursor's item (or of the block's piece
// of it) whose result is not finite, again: a warp a row, key by key over what
// the row sees, in 32 bits.  Rows whose scores are NaN, or that have a bad page,
// stay as they are.
template <typename C, int D, int COPIES>
__device__ void tiles_again(const TilesParams &p, const TileCursor &c, long long begin, int r_from, int r_count, int warp, int warps, int lane)
{
    using S = TilesShape<C, D, COPIES>;
    constexpr int PER = D / 32;  // columns of a lane, next to one another
    const int row0 = c.row_tile * S::ROWS, live = min(S::ROWS, p.rows - row0), t0 = tiles_first(c), t1 = tiles_last(c);
    if (t0 == t1) return;
    const bool whole = item_whole(c);
    float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * (S::ROWS * (D + 2));
    const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
    const float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
    const int32_t *pos = p.sc.slot_pos ? p.sc.slot_pos + (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.sc.pos_stride : nullptr;
    auto up = [&](const void *x, int64_t i) {
        return p.q_bf16 ? Num<__nv_bfloat16>::up(static_cast<const __nv_bfloat16 *>(x)[i]) : Num<__half>::up(static_cast<const __half *>(x)[i]);
    };
#pragma unroll 1
    for (int r = r_from + warp; r < min(r_from + r_count, live); r += warps) {
        const int t = (row0 + r) / p.group, g = row0 + r - t * p.group;
        if (t >= c.s.fresh) continue;
        const int64_t at = ((static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g) * D + PER * lane;
        float *piece = part + 2 * S::ROWS + r * D + PER * lane;
        bool redo = false;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float y = whole ? up(p.out, at + e) : piece[e];
            redo |= !(fabsf(y) < CUDART_INF_F);
        }
        if (!__any_sync(0xffffffffu, redo)) continue;
        Interval see = token_interval(p, c.s, c.b, t);
        TokenView view{};
        if (p.parent) {
            view = token_view(p.sc, p.parent + static_cast<int64_t>(c.b) * p.w.T, c.s, c.b, p.w.T, t);
            see.lo = view.bits ? view.lo : c.s.total;
            see.hi = c.s.total;
        }
        const int own = pos ? __ldg(pos + c.s.ctx + t) : c.s.ctx + (p.parent ? view.depth : t);
        const float slope = p.sc.slopes ? __ldg(p.sc.slopes + c.h * p.group + g) * LOG2E : 0.0f;
        float m = -CUDART_INF_F, l = 0.0f, q[PER], x[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            q[e] = up(p.q, at + e);
            x[e] = 0.0f;
        }
        bool fine = true;
#pragma unroll 1
        for (int j = max(see.lo, t0 * S::KEYS); fine && j < min(see.hi, t1 * S::KEYS); ++j) {
            if (p.parent && j >= c.s.ctx && !(view.bits >> (j - c.s.ctx) & 1)) continue;
            int there = pos ? __ldg(pos + j) : j;
            if (!pos && p.parent && j >= c.s.ctx && p.sc.slopes)
                there = c.s.ctx + token_view(p.sc, p.parent + static_cast<int64_t>(c.b) * p.w.T, c.s, c.b, p.w.T, j - c.s.ctx).depth;
            if (pos && p.sc.window > 0 && own - there >= p.sc.window) continue;
            const int page = page_of(p.c, table, j);
            fine = page >= 0;
            if (!fine) continue;
            const C *k = reinterpret_cast<const C *>(row_ptr(p.c, p.c.k, page, j, c.h)) + PER * lane;
            const C *v = reinterpret_cast<const C *>(row_ptr(p.c, p.c.v, page, j, c.h)) + PER * lane;
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < PER; ++e) s += q[e] * Num<C>::up(k[e]);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= factor;
            fine = s == s;
            if (p.sc.cap2 != 0.0f) {
                float y[1] = {s};
                cap_all(p.sc, y);
                s = y[0];
            }
            if (p.sc.slopes) s = fmaf(-slope, fabsf(static_cast<float>(own - there)), s);
            if (!fine || s == -CUDART_INF_F) continue;
            if (s > m) {
                const float a = fast_exp2(m - s);
                m = s;
                l *= a;
#pragma unroll
                for (int e = 0; e < PER; ++e) x[e] *= a;
            }
            const float w = fast_exp2(s - m);
            l += w;
#pragma unroll
            for (int e = 0; e < PER; ++e) x[e] += w * Num<C>::up(v[e]);
        }
        if (!fine || l == 0.0f) continue;
        const float unit = whole ? (p.c.v_scale ? __ldg(p.c.v_scale + c.h) : 1.0f) / l : fast_exp2(m - part[r]);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (!whole)
                piece[e] = x[e] * unit;
            else if (p.q_bf16)
                static_cast<__nv_bfloat16 *>(p.out)[at + e] = __float2bfloat16_rn(x[e] * unit);
            else
                static_cast<__half *>(p.out)[at + e] = __float2half_rn(x[e] * unit);
        }
    }
}

// NaN for these rows of the cursor's item, after a wait gave up.  Items without
// keys have what they always have.
template <int D, typename S> __device__ void tiles_lost(const TilesParams &p, const TileCursor &c, long long begin, int r_from, int r_count, int tid, int threads)
{
    const AttRows rows{c.b, c.h, c.row_tile * S::ROWS, min(S::ROWS, p.rows - c.row_tile * S::ROWS)};
    const int to = min(r_from + r_count, rows.live);
    const bool empty = c.s.to == 0 && !c.s.bad;
    if (item_whole(c)) {
        const float m = empty ? -CUDART_INF_F : CUDART_NAN_F;
        for (int i = r_from * (D / 4) + tid; i < to * (D / 4); i += threads) {
            const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p.q_bf16)
                write_row<__nv_bfloat16, D>(p, rows, i / (D / 4), i % (D / 4) * 4, zero, m, 0.0f, 1.0f);
            else
                write_row<__half, D>(p, rows, i / (D / 4), i % (D / 4) * 4, zero, m, 0.0f, 1.0f);
        }
    } else {  // a piece: its maximum is enough
        float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * (S::ROWS * (D + 2));
        for (int r = r_from + tid; r < to; r += threads) {
            part[r] = CUDART_NAN_F;
            part[S::ROWS + r] = 0.0f;
        }
        if (r_from == 0) note_split(p, c, rows, begin, tid);
    }
    if (!empty && !c.s.bad && tid == 0 && p.timeouts) p.timeouts[c.b] = STATUS_TIMEOUT;
}

// What is left to do for a group's rows at the end of its range, out of line:
// rows that were not finite, of the first `done` items, and NaN from there on
// where a wait gave up.
template <typename C, int D, int COPIES>
__device__ __noinline__ void tiles_finish(const TilesParams &p, bool again, int done, int group, int tid)
{
    using S = TilesShape<C, D, COPIES>;
    const int lane = tid & 31;
    TileCursor c = tiles_find_again<S>(p, lane);
    const long long begin = c.at;
    const int r_from = 128 * group, r_count = S::PAIR ? 128 : S::ROWS;
    for (int k = 0; c.at < c.end; tiles_next<S>(c, p, lane), ++k) {
        if (k >= done)
            tiles_lost<D, S>(p, c, begin, r_from, r_count, tid, S::GROUP);
        else if (again)
            tiles_again<C, D, COPIES>(p, c, begin, r_from, r_count, tid >> 5, S::GROUP / 32, lane);
    }
}

// Whether a row's products become scores before the bias is taken off them: where the largest product is not the largest
// score (no factor above 0), and where the bias, times 31 bits of distance, would not be finite in units of the products.
__device__ __forceinline__ bool products_first(float factor, float slope) { return !(fabsf(slope) < factor * 0x1p90f); }

// Cap, bias and a window over moved slots of a row's MINE scores of a tile whose
// first key is jb: the true scores are then x f - off.  products: some row of the
// warp has products_first, so all do; slope_in: the slope in units of x.
template <int MINE, bool PAIR, typename Ctl>
__device__ __forceinline__ void tile_shape(const TilesParams &p, unsigned long long (&x)[MINE / 2], float *f, float *off, int ctx, int total,
                                           Ctl *ctl, int place, int jb, int own, int all_own, bool products, float slope, float slope_in, int origin, const int *positions)
{
    const ScoresView &v = p.sc;
    if (v.cap2 != 0.0f) {
        cap_pairs(v, x, *f);
        *f = 1.0f;
    } else if (products) {
        const unsigned long long f2 = pack2(*f, *f);
#pragma unroll
        for (int i = 0; i < MINE / 2; ++i) x[i] = mul2(x[i], f2);
        *f = 1.0f;
    }
    if (moved_slots(v)) {
        const float s = -slope_in;
        if (v.window > 0) {
            const int2 *at = reinterpret_cast<const int2 *>(positions);
#pragma unroll
            for (int i = 0; i < MINE / 2; ++i) {
                const int2 there = at[i];
                const int a = own - there.x, b = own - there.y;
                const float2 y = unpair(x[i]);
                x[i] = pack2(a >= v.window ? -CUDART_INF_F : fmaf(s, fabsf(static_cast<float>(a)), y.x),
                             b >= v.window ? -CUDART_INF_F : fmaf(s, fabsf(static_cast<float>(b)), y.y));
            }
        } else {
            const ulonglong2 *at = reinterpret_cast<const ulonglong2 *>(positions);
            const float mine = static_cast<float>(own - origin);
            const unsigned long long mine2 = pack2(mine, mine);
#pragma unroll
            for (int i = 0; i < MINE / 2; i += 2) {
                const ulonglong2 there = at[i / 2];
                const float2 a = unpair(fadd2(mine2, there.x)), b = unpair(fadd2(mine2, there.y)), y = unpair(x[i]), z = unpair(x[i + 1]);
                x[i] = pack2(fmaf(s, fabsf(a.x), y.x), fmaf(s, fabsf(a.y), y.y));
                x[i + 1] = pack2(fmaf(s, fabsf(b.x), z.x), fmaf(s, fabsf(b.y), z.y));
            }
        }
    } else if (v.slopes) {
        const float s = slope_in;
        if (!PAIR && p.parent && jb + MINE > ctx) {  // a node's position is its depth's
#pragma unroll
            for (int i = 0; i < MINE / 2; ++i) {
                const float2 y = unpair(x[i]);
                float z[2] = {y.x, y.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = jb + 2 * i + k, there = j >= ctx && j < total ? ctx + ctl->at.depth[place][j - ctx] : j;
                    z[k] = fmaf(-s, fabsf(static_cast<float>(own - there)), z[k]);
                }
                x[i] = pack2(z[0], z[1]);
            }
        } else if (all_own >= jb + MINE - 1) {
            // no key is ahead: the distance is that of the place behind the last key and the places before it (the nearest keys,
            // which count most, so have the smallest terms and roundings)
            *off = slope * static_cast<float>(own - (jb + MINE));
#pragma unroll
            for (int i = 0; i < MINE / 2; ++i) {
                const float2 y = unpair(x[i]);
                x[i] = pack2(fmaf(-s, static_cast<float>(MINE - 2 * i), y.x), fmaf(-s, static_cast<float>(MINE - 1 - 2 * i), y.y));
            }
        } else {
            const float far = static_cast<float>(own - jb);
#pragma unroll
            for (int i = 0; i < MINE / 2; ++i) {
                const float2 y = unpair(x[i]);
                x[i] = pack2(fmaf(-s, fabsf(far - static_cast<float>(2 * i)), y.x), fmaf(-s, fabsf(far - static_cast<float>(2 * i + 1)), y.y));
            }
        }
    }
}

// A row a thread (PAIR), or half of its keys.  tid: 0 .. 255.
template <typename C, int D, int COPIES, typename S = TilesShape<C, D, COPIES>>
__device__ void tiles_rows(const TilesParams &p, char *smem, TilesCtl<S> *ctl, unsigned *err, int tid)
{
    using M = typename MmaOf<C, C>::type;  // e4m3: f16
    constexpr float UP = Weights<M>::UP;
    constexpr int KEYS = S::KEYS, MINE = S::MINE, GROUP = S::GROUP, PART = S::ROWS * (D + 2);
    constexpr bool PAIR = S::PAIR;
    constexpr int HALVES = PAIR ? 1 : 2, OF_ROW = PAIR ? 1 : COPIES;
    const int lane = tid & 31, quad = same_in_warp(tid >> 7), half = PAIR ? 0 : quad, group = PAIR ? quad : 0, lane_row = tid & 127;
    const int copy = PAIR ? 0 : lane_row / S::ROWS;
    const int r = PAIR ? 128 * group + lane_row : lane_row % S::ROWS, group_tid = tid - 128 * group;  // row of the item; place in the group
    const uint32_t quarter = static_cast<uint32_t>(lane_row & ~31) << 16;
    const uint32_t tm_o = ctl->tmem + quarter + 256 + group * 128;
    const ScoresView &v = p.sc;
    const bool moved = moved_slots(v);
    const bool by_depth = !PAIR && p.parent && v.slopes && !v.slot_pos;  // the depths beside q are read in every tile
    int n = 0, item = 0;  // tiles of this group; items with tiles
    TileItem it;
    int k = 0;
    bool ok = true;
    it.flags = 0;
    for (;; ++k) {
        // The next item, for the whole group: a warp that a wait has given up stops all.
        const bool some = take_item(ctl, k, &it, err, lane);
        if (!some) {
            if (!(it.flags & ITEM_END) && lane == 0) *reinterpret_cast<volatile int *>(&ctl->stop[group]) = 1;
            group_sync<GROUP>(group);
            break;
        }
        const int t0 = it.t0, t1 = it.t1, row0 = it.row_tile * S::ROWS, live = min(S::ROWS, p.rows - row0);
        const int s0 = PAIR ? max(t0, group ? it.lo1 : it.lo0) : t0, s1 = max(s0, PAIR ? min(t1, group ? it.hi1 : it.hi0) : t1);
        const float v_scale = p.c.v_scale ? __ldg(p.c.v_scale + it.h) : 1.0f;
        const bool mine = r < live;
        const int token = (row0 + r) / p.group;
        const int64_t row_at = (static_cast<int64_t>(it.b) * p.w.T + token) * p.q_heads + it.h * p.group + (row0 + r) - token * p.group;
        float m = -CUDART_INF_F, l = 0.0f;  // a maximum so far less UP: what l and O are sums against
        bool any_bad = it.flags & ITEM_BAD;
        const int place = item % S::Q_PLACES;
        // What the row sees, asked for before the others are waited for: the last warp then finds it in the L1.
        const bool there = mine && token < it.fresh && t0 < t1;
        const SeqLens lens{it.ctx, it.fresh, it.total, false};
        Interval see{0, 0};
        unsigned long long bits = 0;
        int own = 0;
        const int32_t *pos = v.slot_pos ? v.slot_pos + (static_cast<int64_t>(it.b) * p.c.kv_heads + it.h) * v.pos_stride : nullptr;
        if (there && !p.parent) {
            see = token_interval(p, lens, it.b, token);
            own = moved ? __ldg(pos + it.ctx + token) : it.ctx + token;
        }
        if constexpr (!PAIR) {
            if (there && p.parent) {
                const TokenView view = token_view(v, p.parent + static_cast<int64_t>(it.b) * p.w.T, lens, it.b, p.w.T, token);
                bits = view.bits;
                own = moved ? __ldg(pos + it.ctx + token) : it.ctx + view.depth;
                see.hi = bits ? it.ctx : 0;
                see.lo = view.lo;
            }
        }
        const int origin = moved && t0 < t1 ? __ldg(pos + it.ctx) : 0;  // the first new token's position
        const float slope = there && v.slopes ? __ldg(v.slopes + it.h * p.group + (row0 + r) - token * p.group) * LOG2E : 0.0f;
        float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + it.h) : 1.0f);
        group_sync<GROUP>(group);  // all have read the last item's sums and flags
        if (*reinterpret_cast<volatile int *>(&ctl->stop[group])) break;
        if (t0 < t1) {
            if constexpr (S::ROWS_WIDEN) {
                ok = tiles_wait(ctl, &ctl->q_raw[place], (item / S::Q_PLACES) & 1, err);
                if (ok) {
                    char *row = smem + place * S::Q + group * S::Q_SUB;
                    factor *= p.q_bf16 ? widen_row<__nv_bfloat16, D>(row, lane_row) : widen_row<__half, D>(row, lane_row);
                }
                fence_async_shared();
                mbar_arrive(&ctl->q_full[place]);
            } else {
                ok = tiles_wait(ctl, &ctl->q_full[place], (item / S::Q_PLACES) & 1, err);
                if (S::WIDEN) factor *= exp2f(-static_cast<float>(ctl->at.q_power[place * S::ROWS + r]));
            }
            if (OF_ROW == 1 && !by_depth) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->q_empty[place]);
            }
            const bool products = __any_sync(0xffffffffu, products_first(factor, slope)), shaped = v.cap2 != 0.0f || v.slopes || moved || products;
            const float slope_in = v.cap2 != 0.0f || products ? slope : slope / factor;
            const bool works = __any_sync(0xffffffffu, there);
            // the slots that all rows of the warp see (votes of each tile took hundreds of cycles)
            const int all_lo = __reduce_max_sync(0xffffffffu, see.lo), all_hi = __reduce_min_sync(0xffffffffu, see.hi);
            const int all_own = __reduce_min_sync(0xffffffffu, there ? own : 0x7fffffff);
            bool huge = false;  // scores beyond what a fused difference allows
            auto position = [&](int tile) {
                const int j = tile * KEYS + group_tid;
                return moved && group_tid < KEYS && tile >= s0 && j < it.total ? __ldg(pos + j) : 0;
            };
            int next_at = position(s1 - 1);
#pragma unroll 1
            for (int tile = s1 - 1; tile >= s0; --tile, ++n) {  // to its end even after a wait gave up: the halves meet at each tile
                const int buf = group * 2 + (n & 1);
                const int of_tile = copy * S::OF_COPY + half * MINE;  // this thread's keys
                const uint32_t tm_s = ctl->tmem + quarter + buf * S::PLACE + of_tile;
                const int jb = tile * KEYS + of_tile;
                if (moved) {  // positions of the tile's keys, asked for a tile ahead
                    group_sync<GROUP>(group);  // the last tile's have been read
                    // as distances to the item's first token where no window has to be exact: 32 bits hold those below 2^24
                    if (group_tid < KEYS)
                        ctl->at.positions[group][group_tid] = v.window > 0 ? next_at : __float_as_int(static_cast<float>(origin - next_at));
                    group_sync<GROUP>(group);
                    next_at = position(tile - 1);
                }
                ok = ok && tiles_wait(ctl, &ctl->s_full[buf], (n >> 1) & 1, err);
                tc_fence_after();
                __syncwarp();
                if (works) {
                    // Pairs of scores, so that one instruction works on two.
                    unsigned long long x[MINE / 2];
                    constexpr int LOAD = MINE < 64 ? MINE : 64;
#pragma unroll
                    for (int i = 0; i < MINE; i += LOAD) {
                        uint32_t y[LOAD];
                        if constexpr (LOAD == 64)
                            tc_ld64(y, tm_s + i);
                        else if constexpr (LOAD == 32)
                            tc_ld32(y, tm_s + i);
                        else
                            tc_ld16(y, tm_s + i);
#pragma unroll
                        for (int e = 0; e < LOAD; e += 2) x[(i + e) / 2] = pack2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                    }
                    // The true scores are x f - off.
                    float f = factor, off = 0.0f;
                    if (shaped) tile_shape<MINE, PAIR>(p, x, &f, &off, it.ctx, it.total, ctl, place, jb, own, all_own, products, slope, slope_in, origin, ctl->at.positions[group] + of_tile);
                    if (all_lo > jb || all_hi < jb + MINE) {
#pragma unroll
                        for (int i = 0; i < MINE; i += 32) {
                            constexpr int AT_A_TIME = MINE < 32 ? MINE : 32;
                            const int lo = min(max(see.lo - jb - i, 0), 32), hi = min(max(see.hi - jb - i, 0), 32);
                            unsigned mask = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
                            if (!PAIR && p.parent) {
                                const int o = it.ctx - (jb + i);  // the first new token's column, from here
                                if (o < 32 && o > -64) mask |= static_cast<unsigned>(o >= 0 ? bits << o : bits >> -o);
                            }
                            mask = lo == 32 ? 0u : mask & ~((1u << lo) - 1u);
#pragma unroll
                            for (int k = 0; k < AT_A_TIME; k += 2) {
                                const float2 y = unpair(x[(i + k) / 2]);
                                x[(i + k) / 2] = pack2(mask >> k & 1 ? y.x : -CUDART_INF_F, mask >> (k + 1) & 1 ? y.y : -CUDART_INF_F);
                            }
                        }
                    }
                    float tops[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 y = unpair(x[i]);
                        tops[i] = fmaxf(y.x, y.y);
                    }
#pragma unroll
                    for (int i = 4; i < MINE / 2; ++i) {
                        const float2 y = unpair(x[i]);
                        tops[i & 3] = fmax3(tops[i & 3], y.x, y.y);
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * f - off;
                    if (HALVES == 2) {  // the maximum of both halves, by the two warps that have these rows
                        ctl->at.top[n & 1][tid] = top;
                        halves_sync(lane_row / 32);  // (the places of two tiles: the one before has been read when both are here)
                        top = fmaxf(top, ctl->at.top[n & 1][tid ^ 128]);
                    }
                    if (tile == s1 - 1) {
                        m = top - UP;
                        huge = __any_sync(0xffffffffu, fabsf(m) > 0x1p20f && m != -CUDART_INF_F);
                    } else if (__any_sync(0xffffffffu, top - m > UP + Weights<M>::LAG)) {  // as a difference: a sum may round up to a score 16 above
                        const float grown = fmaxf(m, top - UP), a = grown == -CUDART_INF_F ? 0.0f : fast_exp2(m - grown);
                        m = grown;
                        huge |= __any_sync(0xffffffffu, fabsf(m) > 0x1p20f && m != -CUDART_INF_F);
                        l *= a;
                        // (those of the tile before that were done before this tile's scores)
                        ok = ok && tiles_wait(ctl, &ctl->o_done[buf ^ 1], ((n - 1) >> 1) & 1, err);
                        tc_fence_after();
#pragma unroll 1
                        for (int i = half * (D / HALVES); i < (half + 1) * (D / HALVES); i += 16) {
                            uint32_t y[16];
                            tc_ld16(y, tm_o + i);
#pragma unroll
                            for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * a);
                            tc_st16(tm_o + i, y);
                        }
                    }
                    float base = m == -CUDART_INF_F ? 0.0f : m + off;
                    if (huge) {
                        // the score is rounded as m was, not fused with the difference: of scores this large the largest would
                        // else miss m by more than a weight can hold
                        const unsigned long long f2 = pack2(f, f), none = pack2(-off, -off);
#pragma unroll
                        for (int i = 0; i < MINE / 2; ++i) x[i] = fadd2(mul2(x[i], f2), none);
                        f = 1.0f;
                        base = m == -CUDART_INF_F ? 0.0f : m;
                    }
                    const unsigned long long f2 = pack2(f, f), base2 = pack2(-base, -base);
                    unsigned long long sum[2] = {0, 0};
                    constexpr int AT_ONCE = MINE < 64 ? MINE : 64;
#pragma unroll
                    for (int i0 = 0; i0 < MINE; i0 += AT_ONCE) {
                        uint32_t pk[AT_ONCE / 2];
#pragma unroll
                        for (int i = 0; i < AT_ONCE; i += 2) {
                            const float2 y = unpair(ffma2(x[(i0 + i) / 2], f2, base2));
                            const float a = fast_exp2(y.x), b = fast_exp2(y.y);
                            sum[i / 2 & 1] = fadd2(sum[i / 2 & 1], pack2(a, b));
                            // rounded to 16 bits for the product (half a step of the type each); l keeps 32 bits
                            pk[i / 2] = pack_mma<M>(a, b);
                        }
                        if constexpr (AT_ONCE == 64)
                            tc_st32(tm_s + i0 / 2, pk);
                        else if constexpr (AT_ONCE == 32)
                            tc_st16(tm_s + i0 / 2, pk);
                        else
                            tc_st8(tm_s + i0 / 2, pk);
                    }
                    if (OF_ROW > 1) {  // no weights for the keys of the row's other copies
                        uint32_t none[MINE / 2];
#pragma unroll
                        for (int i = 0; i < MINE / 2; ++i) none[i] = 0;
#pragma unroll
                        for (int i = 1; i < OF_ROW; ++i) {
                            const uint32_t to = ctl->tmem + quarter + buf * S::PLACE + (copy + i) % OF_ROW * S::OF_COPY + half * MINE;
                            if constexpr (MINE == 32)
                                tc_st16(to, none);
                            else if constexpr (MINE == 16)
                                tc_st8(to, none);
                        }
                    }
                    const float2 all = unpair(fadd2(sum[0], sum[1]));
                    l += all.x + all.y;
                    tc_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&ctl->p_full[buf]);
            }
            if (s0 < s1) ok = ok && tiles_wait(ctl, &ctl->o_done[group * 2 + ((n - 1) & 1)], ((n - 1) >> 1) & 1, err);
            tc_fence_after();
            if (OF_ROW == 1 && by_depth) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->q_empty[place]);
            }
            any_bad |= *reinterpret_cast<volatile char *>(&ctl->bad[group][item % S::ITEMS]) != 0;
            ++item;
        }
        const bool tiles = s0 < s1;
        group_sync<GROUP>(group);  // all have read the item's flag, and the last tile's maxima
        if (group_tid == 0) {
            if (*reinterpret_cast<volatile int *>(&ctl->dead)) ctl->stop[group] = 1;
            if (t0 < t1) ctl->bad[group][(item - 1) % S::ITEMS] = 0;
        }
        if (HALVES == 2) ctl->at.top[0][tid] = l, ctl->at.top[1][tid] = m;
        group_sync<GROUP>(group);
        if (*reinterpret_cast<volatile int *>(&ctl->stop[group])) break;  // a wait gave up: this item is among what is lost
        if (HALVES == 2) l += ctl->at.top[0][tid ^ 128];
        float part_of = 1.0f;  // what this copy's sums are multiplied by
        if (OF_ROW > 1) {
            float of_all = -CUDART_INF_F, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < OF_ROW; ++i) of_all = fmaxf(of_all, ctl->at.top[1][i * S::ROWS + r]);
            const float base = of_all == -CUDART_INF_F ? 0.0f : of_all;
#pragma unroll
            for (int i = 0; i < OF_ROW; ++i)
                sum += (ctl->at.top[0][i * S::ROWS + r] + ctl->at.top[0][128 + i * S::ROWS + r]) * fast_exp2(ctl->at.top[1][i * S::ROWS + r] - base);
            part_of = fast_exp2(m - base);
            m = of_all;
            l = sum;
        }
        const bool whole = it.flags & ITEM_WHOLE;
        float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (it.flags & ITEM_SECOND ? 1 : 0)) * PART;
        const bool none = m == -CUDART_INF_F && l == 0.0f, fixed = none || any_bad;
        const float instead = any_bad ? CUDART_NAN_F : 0.0f, out_scale = v_scale / l;
        if (half == 0 && copy == 0 && mine) {
            if (!whole) {
                part[r] = any_bad ? CUDART_NAN_F : m;
                part[S::ROWS + r] = l;
            } else if (p.lse) {
                p.lse[row_at] = any_bad ? CUDART_NAN_F : none ? -CUDART_INF_F : LN2 * (m + log2f(l));
            }
        }
        float odd = 0.0f;  // NaN if something is not finite
        // With copies all but the first leave theirs in q's place, which is free by now, some columns at a time.
        constexpr int AT_A_TIME = OF_ROW > 1 && D == 64 ? 16 : 32;
#pragma unroll 1
        for (int d0 = half * (D / HALVES); d0 < (half + 1) * (D / HALVES); d0 += AT_A_TIME) {
            float x[AT_A_TIME];
            __syncwarp();
            if (tiles) {
                uint32_t y[AT_A_TIME];
                if constexpr (AT_A_TIME == 32)
                    tc_ld32(y, tm_o + d0);
                else
                    tc_ld16(y, tm_o + d0);
#pragma unroll
                for (int k = 0; k < AT_A_TIME; ++k) x[k] = __uint_as_float(y[k]);
            } else {
#pragma unroll
                for (int k = 0; k < AT_A_TIME; ++k) x[k] = 0.0f;
            }
            if (OF_ROW > 1 && t0 < t1) {
                float *buf = reinterpret_cast<float *>(smem + (item - 1) % S::Q_PLACES * S::Q);
#pragma unroll
                for (int k = 0; k < AT_A_TIME; ++k) x[k] = part_of == 0.0f ? 0.0f : x[k] * part_of;  // a copy without keys: anything
                group_sync<GROUP>(group);
                if (copy > 0) {
                    float *to = buf + ((2 * copy - 2 + half) * S::ROWS + r) * AT_A_TIME;
#pragma unroll
                    for (int k = 0; k < AT_A_TIME; ++k) to[(k + r) % AT_A_TIME] = x[k];  // a column's rows on different banks
                }
                group_sync<GROUP>(group);
                if (copy == 0) {
#pragma unroll
                    for (int i = 0; i < OF_ROW - 1; ++i) {
                        const float *from = buf + ((2 * i + half) * S::ROWS + r) * AT_A_TIME;
#pragma unroll
                        for (int k = 0; k < AT_A_TIME; ++k) x[k] += from[(k + r) % AT_A_TIME];
                    }
                }
            }
            if (copy > 0) continue;
            if (!mine) continue;
            // 32 bytes a store: a thread's row is its own, and half a sector at a time costs twice the transactions
            if (!whole) {
#pragma unroll
                for (int k = 0; k < AT_A_TIME; ++k) {
                    x[k] = fixed ? 0.0f : x[k];
                    odd = fmaf(x[k], 0.0f, odd);
                }
#pragma unroll
                for (int k = 0; k < AT_A_TIME; k += 8) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(x[k + e]);
                    store_32bytes(part + 2 * S::ROWS + r * D + d0 + k, y);
                }
            } else {
#pragma unroll
                for (int k = 0; k < AT_A_TIME; ++k) {
                    x[k] = fixed ? instead : x[k] * out_scale;
                    odd = fmaf(x[k], 0.0f, odd);
                }
#pragma unroll
                for (int k = 0; k < AT_A_TIME; k += 16) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = S::WIDEN && p.q_bf16 ? pack_mma<__nv_bfloat16>(x[k + 2 * e], x[k + 2 * e + 1])
                                                    : pack_mma<M>(x[k + 2 * e], x[k + 2 * e + 1]);
                    store_32bytes(static_cast<char *>(p.out) + (row_at * D + d0 + k) * 2, y);
                }
            }
        }
        tc_fence_before();
        if (OF_ROW > 1 && t0 < t1) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->q_empty[(item - 1) % S::Q_PLACES]);
        }
        if (odd != odd && !any_bad) *reinterpret_cast<volatile int *>(&ctl->lost[group]) = 1;
    }
    group_sync<GROUP>(group);
    const bool again = *reinterpret_cast<volatile int *>(&ctl->lost[group]), stopped = *reinterpret_cast<volatile int *>(&ctl->stop[group]);
    if (again || stopped) tiles_finish<C, D, COPIES>(p, again, stopped ? k : 0x7fffffff, group, group_tid);
}

template <typename C, int D, int COPIES>
__global__ void __launch_bounds__(TILES_THREADS, 1)
    tiles_kernel(const TilesParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q, const int maps, const int q_map)
{
    using S = TilesShape<C, D, COPIES>;
    using Ctl = TilesCtl<S>;
    extern __shared__ __align__(1024) char smem[];  // the swizzle's rows of 128 bytes come in groups of eight
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::CTL_AT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned *err = p.error;
    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&ctl->full[i], 4);  // the loaders' warps
            mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], S::GROUP);
            mbar_init(&ctl->o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->item_full[i], 1);
            mbar_init(&ctl->item_empty[i], TILES_TAKERS);
            mbar_init(&ctl->q_full[i], S::ROWS_WIDEN ? 256 : TILES_PREPARE);
            mbar_init(&ctl->q_empty[i], 1 + 8);  // the products' end, and the row warps, when they need what lies beside q no more
            ctl->stop[i] = ctl->lost[i] = 0;
            for (int k = 0; k < S::ITEMS; ++k) ctl->bad[i][k] = 0;
        }
        mbar_init(&ctl->spare, 1);
        for (int i = 0; i < S::Q_PLACES; ++i) mbar_init(&ctl->q_raw[i], S::ROWS_WIDEN && !q_map ? TILES_PREPARE : 1);
        if (S::WIDEN)
            for (int i = 0; i < 4; ++i)
                for (int k = 0; k < S::RAW_STAGES; ++k) mbar_init(&ctl->raw_full[S::WIDEN ? i : 0][k], 1);
        ctl->dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tmem_alloc(&ctl->tmem, 512);
    chain_begin();
    const TileCursor c = tiles_find<S>(p, ctl, tid);
    if (tid < 2) p.split[blockIdx.x * 2 + tid].n = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c.at >= c.end) {  // the whole block
        if (warp == 8) tmem_free(ctl->tmem, 512);
        return;
    }
    // registers: launched with 128 a thread, 4 x 128 = 2 x 160 + 2 x 96
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        tiles_rows<C, D, COPIES>(p, smem, ctl, err, tid);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 8) {
            tiles_multiply<C, D, COPIES>(smem, ctl, err, lane);
            warp_commit(&ctl->spare);  // what was issued ends before the block may: others may have given up on it
            mbar_drain(&ctl->spare, 0);
        } else if (warp == 9) {
            tiles_items<S>(p, c, ctl, err, lane);
        } else {
            tiles_prepare<C, D, COPIES>(p, smem, ctl, err, tid - 320, q_map ? &map_q : nullptr);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        tiles_load<C, D, COPIES>(p, smem, ctl, err, tid - 384, maps ? &map_k : nullptr, maps ? &map_v : nullptr);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_free(ctl->tmem, 512);
}

template <typename C, int D, int COPIES> cudaError_t launch_tiles_of(TilesParams p, const KvLaunch &L, cudaStream_t st)
{
    using S = TilesShape<C, D, COPIES>;
    constexpr int SMEM = S::CTL_AT + static_cast<int>(sizeof(TilesCtl<S>));
    static_assert(SMEM <= 232448, "shared memory of a block");
    auto kernel = tiles_kernel<C, D, COPIES>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    p.w.tile = S::KEYS;
    p.w.row_tiles = (p.rows + S::ROWS - 1) / S::ROWS;
    CUtensorMap map_k{}, map_v{}, map_q{};
    const bool q_map = query_map(&map_q, p.q, L, p.group, S::PAIR ? 128 : S::ROWS);
    const int slots = S::WIDEN ? S::KEYS / 4 : S::KEYS;
    const bool maps = pool_map(&map_k, L, false, slots, S::WIDEN) && pool_map(&map_v, L, true, slots, S::WIDEN);
    e = launch_chained(kernel, dim3(ATT_SMS), TILES_THREADS, SMEM, st, p, map_k, map_v, map_q, static_cast<int>(maps), static_cast<int>(q_map));
    return e != cudaSuccess ? e : launch_join(p, L.dtype, D, S::ROWS, ATT_SMS, st);
}
template <typename C, int D> cudaError_t launch_tiles_dim(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    if (pairs) return launch_tiles_of<C, D, 0>(p, L, st);
    if constexpr (sizeof(C) == 2) {  // (of e4m3 so few rows are a rare prompt)
        if (p.rows <= 32) return launch_tiles_of<C, D, 4>(p, L, st);
    }
    if (p.rows <= 64) return launch_tiles_of<C, D, 2>(p, L, st);
    return launch_tiles_of<C, D, 1>(p, L, st);
}
template <typename C> cudaError_t launch_tiles_types(const TilesParams &p, const KvLaunch &L, bool pairs, cudaStream_t st)
{
    switch (L.cache.head_dim) {
    case 64: return launch_tiles_dim<C, 64>(p, L, pairs, st);
    case 128: return launch_tiles_dim<C, 128>(p, L, pairs, st);
    default: return launch_tiles_of<C, 256, 1>(p, L, st);
    }
}

}  // namespace spv
