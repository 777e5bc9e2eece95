// spv_attention_rows.cu -- attention over the paged cache for many query rows
// a key head (drafted chains with wide groups, draft trees): 5th-generation
// tensor cores, up to 128 rows at a time against tiles of 128 keys.
//
// One block an SM, with its equal range of all tiles (Work, Cursor), in roles
// that follow one another over shared and tensor memory:
//   * four warps bring K and four V, through the page table.  Whole tiles of a
//     16-bit cache with pages of eight slots or more come by the copy engine, a
//     box a page; other pages, and V's tiles with new tokens (whose infinities
//     are looked for), by asynchronous copies of the threads, in the permuted
//     layout the tensor cores read.  An e4m3 cache lands as it is and is widened
//     to f16 by the threads that loaded it (f16 holds every e4m3 value);
//   * one thread issues S = Q K^T, another O += P V, P from tensor memory, all
//     sums in 32 bits in tensor memory; two warps bring q of the next item;
//   * four warps hold a row a thread: running maximum, exponentials, sum, P
//     back to tensor memory.  O is only rescaled when a maximum has grown by
//     more than 2^8 (2^7 for f16 products), so p stays below 2^8 (2^14) and the
//     32-bit sums lose nothing.
// With 64 rows or fewer the rows stand in tensor memory two or four times,
// each copy taking half or a quarter of every tile's keys (its P is zero
// elsewhere): all four warps work whatever the number of rows, and the
// copies join at the end like pieces.  With more rows than that eight warps
// work, two on each row's keys: with four, the exponentials of 128 rows took
// 2,850 cycles a tile where its K and V take 2,300 (draft trees: 110 us).
//
// What bounds it, and what it takes: 40 rows of 64 sequences of up to 8,191
// slots, K and V 1.37 GB, 236 us (5.8 TB/s, 86% of a copy's rate: reading K and
// V, then starts, ends of items and joins); 84 rows of 32 sequences of up to
// 4,099 slots, 353 MB, 89 us: exponentials, 1,800 of a tile's 2,450 cycles when it
// took 94 us, and the ends of items.
//
// Every wait is bounded; one that gives up records SPV_ERR_TIMEOUT in the
// workspace, ends the block in order and leaves NaN in all that it still had to
// write, the pieces of shared items among them.
#include "spv_attention.cuh"
#include "spv_tcgen.cuh"
#include "spv_tma.cuh"

namespace spv {

constexpr int AR_KEYS = 128;
constexpr int AR_ROWS = 128;
constexpr int AR_PREPARE = 64;        // threads that bring q
constexpr int AR_ITEMS = 16;          // items whose flags can be in use at once

template <typename C, int D> struct RowsShape {
    static constexpr bool WIDEN = sizeof(C) == 1;
    static constexpr int TILE = AR_KEYS * D * 2;                             // q, K or V as multiplied
    static constexpr int RAW = AR_KEYS * D;                                  // e4m3 K or V
    // K's place is free once the scores are there, V's only after the outputs: at D = 128 there is room for two and
    // three. e4m3: one widened tile each, and stages of raw ones.
    static constexpr int K_STAGES = WIDEN ? 1 : D == 128 ? 2 : 5, V_STAGES = WIDEN ? 1 : D == 128 ? 3 : 5;
    static constexpr int RAW_STAGES = WIDEN ? (D == 128 ? 3 : 5) : 0;
    static constexpr int Q_AT = 0, K_AT = 2 * TILE, V_AT = K_AT + K_STAGES * TILE, RAW_AT = V_AT + V_STAGES * TILE;
    static constexpr int CTL_AT = RAW_AT + RAW_STAGES * 2 * RAW;
};

struct RowsCtl {
    uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];  // of a stage (e4m3: the one widened tile)
    uint64_t s_full[2], p_full[2], o_done[2], q_full[2], q_empty[2], spare[2];
    int odd[AR_ITEMS];                 // some new token's v has infinities or NaN
    unsigned long long sees[2][64];    // per place of q: what each new token sees
    int bad[AR_ITEMS];                 // a page id outside the pool
    float top[2 * AR_ROWS];            // a tile's maxima of the two halves
    // e4m3: what widening a tile needs to know of it, per loader warp and stage: the row of its first new token (128:
    // none), the item's flags.
    short tail[8][5][2];
    signed char q_power[2][AR_ROWS];   // e4m3: the rows of q are stored times 2^q_power
    uint32_t tmem;
    int dead, stop;
    int lost;                          // infinities or NaN of V are missing in some row's output, or may be there in vain
};

// Warps of a block: 4 for the rows, or 8 that share each row's keys where a row stands once; then 4 of products and q, 4
// of K, 4 of V.
template <int COLS> struct RowsWarps {
    static constexpr int HALVES = COLS == AR_ROWS ? 2 : 1, SOFTMAX = 128 * HALVES, THREADS = SOFTMAX + 384;
};

// What the warps of the rows exchange at the end of a piece, in the place of its q.
template <int D> struct RowsMerge {
    static constexpr int ROUNDS = D == 128 ? 2 : 1;  // buffers in turn, as many as fit
    float ms[2 * AR_ROWS], ls[2 * AR_ROWS];
    float x[ROUNDS][96 * 33];
};

// Bounded wait; false once a wait of the block has given up.
__device__ __forceinline__ bool rows_wait1(RowsCtl *ctl, uint64_t *bar, uint32_t parity, unsigned *err)
{
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63 && *reinterpret_cast<volatile int *>(&ctl->dead)) return false;
    }
    *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
    atomicExch(err, static_cast<unsigned>(STATUS_TIMEOUT));
    return false;
}
// The same of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool rows_wait(RowsCtl *ctl, uint64_t *bar, uint32_t parity, unsigned *err)
{
    return __all_sync(0xffffffffu, rows_wait1(ctl, bar, parity, err));
}

// Tiles of the cursor's item that this block has: [t0, t1); none for an item without keys.
__device__ __forceinline__ int first_tile(const Cursor &c) { return static_cast<int>(c.at - c.first); }
__device__ __forceinline__ int last_tile(const Cursor &c)
{
    if (c.s.total == 0) return first_tile(c);
    const long long e = c.first + c.tiles;
    return static_cast<int>((c.end < e ? c.end : e) - c.first);
}

__device__ __forceinline__ uint32_t panel_at(int row, int chunk)  // 16-byte chunk of a 16-bit row in an operand tile
{
    return (chunk >> 3) * (AR_KEYS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Clears infinities and NaN in 8 16-bit values.
template <typename C> __device__ __forceinline__ uint4 finite_only(uint4 x)
{
    const uint32_t e = std::is_same<C, __half>::value ? 0x7c00u : 0x7f80u;
    uint32_t *w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & e) == e) w[i] &= 0xffff0000u;
        if (((w[i] >> 16) & e) == e) w[i] &= 0x0000ffffu;
    }
    return x;
}

// The block's item that a loader or the multiplying thread is at, by number of
// items with tiles: the place of its flags.
__device__ __forceinline__ int item_flags(int item) { return item % AR_ITEMS; }

// ------------------------------------------------------------------ loaders
// One of two groups of four warps: K (kv = 0) or V.
template <typename C, int D, int kv>
__device__ void rows_load(const AttParams &p, Cursor c, char *smem, RowsCtl *ctl, unsigned *err, int lt, const CUtensorMap *map)
{
    using S = RowsShape<C, D>;
    constexpr int CH = D * static_cast<int>(sizeof(C)) / 16, RPI = 32 / CH;
    constexpr int NST = S::WIDEN ? S::RAW_STAGES : kv ? S::V_STAGES : S::K_STAGES, AT = kv ? S::V_AT : S::K_AT;
    const int lane = lt & 31, w = lt >> 5, chunk = lane % CH, sub = lane / CH;
    const uint32_t base = smem_u32(smem);
    const PoolView &pool = kv ? p.c.v : p.c.k;
    uint64_t *full = kv ? ctl->v_full : ctl->k_full, *empty = kv ? ctl->v_empty : ctl->k_empty;
    const int mask = (1 << p.c.page_shift) - 1;
    int n = 0, item = 0;  // tiles issued, items with tiles

    // e4m3: widens tile t, whose copies have landed; each thread what it has loaded.
    auto widen = [&](int t) -> bool {
        const int st = t % NST;
        const int row0 = ctl->tail[4 * kv + w][st][0], flags = ctl->tail[4 * kv + w][st][1];
        const char *raw = smem + S::RAW_AT + (st * 2 + kv) * S::RAW;
        char *to = smem + AT;
        if (t > 0 && !rows_wait(ctl, empty, (t - 1) & 1, err)) return false;
        // Two chunks at a time, not all eight unrolled: with the other roles' code the loop has to fit the instruction
        // caches (two sequences of 131,001 slots, 40 rows: 202 us; four at a time 216, all 287).
        constexpr int AT_ONCE = 2;
#pragma unroll 1
        for (int i0 = 0; i0 < CH; i0 += AT_ONCE) {
            uint4 in[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
                in[i] = *reinterpret_cast<const uint4 *>(raw + (32 * w + (i0 + i) * RPI + sub) * D + chunk * 16);
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int row = 32 * w + (i0 + i) * RPI + sub;
                uint32_t b[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                if (kv && row >= row0 && chunk_not_finite<C>(in[i])) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // bytes 0x7f and 0xff, to 0
                        b[k] &= ~(((((b[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
                    *reinterpret_cast<volatile int *>(&ctl->odd[flags]) = 1;
                }
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    y[2 * k] = e4m3x2_to_f16x2(b[k] & 0xffffu);
                    y[2 * k + 1] = e4m3x2_to_f16x2(b[k] >> 16);
                }
                // lanes of the two panels store their halves in opposite order: no two on one bank
                const bool swap = (chunk >> 2) & 1;
                const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
                *reinterpret_cast<uint4 *>(to + panel_at(row, 2 * chunk + swap)) = swap ? hi : lo;
                *reinterpret_cast<uint4 *>(to + panel_at(row, 2 * chunk + !swap)) = swap ? lo : hi;
            }
        }
        fence_async_shared();
        mbar_arrive(full);
        return true;
    };
    bool ok = true;
    for (; ok && c.at < c.end; next_item(c, p.w, p.c)) {
        const int t0 = first_tile(c), t1 = last_tile(c);
        if (t0 == t1) continue;
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        const int flags = item_flags(item++);
        const char *from = pool.base + c.h * pool.head_stride + chunk * 16;
        auto lookup = [&](int tile) {  // the page id of this lane's row of a tile, unchecked; -1: no such row
            const int j = tile * AR_KEYS + 32 * w + lane;
            return tile < t1 && j < c.s.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
        };
        // With a map, the first warp's lanes ask the copy engine for a box each: a page (or 128 slots of a large one)
        // by 64 elements.  V's tiles with new tokens still go through the threads, who look at them.
        const int box_slots = min(mask + 1, AR_KEYS), boxes = map ? AR_KEYS / box_slots * (D / 64) : 0;
        auto box_lookup = [&](int tile) {
            const int j = tile * AR_KEYS + lane / (D / 64) * box_slots;
            return w == 0 && lane < boxes && tile < t1 && j < c.s.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
        };
        int pg = -1, next = -1;
        if (map) {
            pg = box_lookup(t0);
            next = box_lookup(t0 + 1);
        } else {
            pg = lookup(t0);
            next = lookup(t0 + 1);
        }
        for (int tile = t0; tile < t1; ++tile, ++n) {
            const int st = n % NST, j0 = tile * AR_KEYS;
            if constexpr (!S::WIDEN) {
                if (map && (!kv || j0 + AR_KEYS <= c.s.ctx)) {
                    const int page = pg, slot = j0 + lane / (D / 64) * box_slots;
                    pg = next;
                    next = box_lookup(tile + 2);
                    if (w == 0 && lane < boxes && slot < c.s.total && static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.num_pages))
                        *reinterpret_cast<volatile int *>(&ctl->bad[flags]) = 1;
                    if (n >= NST && !(ok = rows_wait(ctl, &empty[st], (n / NST - 1) & 1, err))) break;
                    if (lt == 0)
                        mbar_arrive_expect_tx(&full[st], S::TILE);
                    else
                        mbar_arrive(&full[st]);
                    if (w == 0) {
                        __syncwarp();
                        if (lane < boxes)
                            tma_box(base + AT + st * S::TILE + (lane % (D / 64)) * (AR_KEYS * 128) + lane / (D / 64) * box_slots * 128,
                                    map, (lane % (D / 64)) * 64, slot & mask, c.h, page, &full[st]);
                    }
                    continue;
                }
                if (map) pg = lookup(tile);  // a tile of V with new tokens: by rows
            }
            const int row0 = min(max(0, c.s.ctx - j0), AR_KEYS);  // of the first new token
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.c.num_pages)) {
                if (j0 + 32 * w + lane < c.s.total) *reinterpret_cast<volatile int *>(&ctl->bad[flags]) = 1;
                pg = -1;
            }
            const int64_t mine = pg < 0 ? -1 : pg * pool.page_stride + ((j0 + 32 * w + lane) & mask) * pool.slot_stride;
            pg = map ? box_lookup(tile + 1) : next;
            next = map ? box_lookup(tile + 2) : lookup(tile + 2);  // two tiles ahead: its latency is behind that of the rows
            uint32_t to;
            if (S::WIDEN) {  // the raw stages are each thread's own
                if (n >= NST) {
                    cp_async_wait<NST - 1>();
                    if (!(ok = widen(n - NST))) break;
                }
                __syncwarp();
                if (lane == 0) {
                    ctl->tail[4 * kv + w][st][0] = row0;
                    ctl->tail[4 * kv + w][st][1] = flags;
                }
                __syncwarp();
                to = base + S::RAW_AT + (st * 2 + kv) * S::RAW;
            } else {
                if (n >= NST && !(ok = rows_wait(ctl, &empty[st], (n / NST - 1) & 1, err))) break;
                to = base + AT + st * S::TILE;
            }
#pragma unroll(S::WIDEN ? 2 : 1)
            for (int i = 0; i < CH; ++i) {
                const int row = 32 * w + i * RPI + sub;
                const int64_t at = __shfl_sync(0xffffffffu, mine, i * RPI + sub);
                cp_async16_zfill(to + (S::WIDEN ? row * D + chunk * 16 : panel_at(row, chunk)), at < 0 ? pool.base : from + at,
                                 at < 0 ? 0 : 16);
            }
            if (S::WIDEN) {
                cp_async_commit();
            } else if (kv && row0 < AR_KEYS) {
                // Infinities and NaN in a new token's v: cleared here, as 0 x inf would reach rows that do not see it;
                // the rows that do get them at the end of the range.
                asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
                for (int i = 0; i < CH; ++i) {
                    const int row = 32 * w + i * RPI + sub;
                    if (row < row0) continue;
                    uint4 *v = reinterpret_cast<uint4 *>(smem + (to - base) + panel_at(row, chunk));
                    const uint4 x = *v;
                    if (chunk_not_finite<C>(x)) {
                        *v = finite_only<C>(x);
                        *reinterpret_cast<volatile int *>(&ctl->odd[flags]) = 1;
                    }
                }
                fence_async_shared();
                mbar_arrive(&full[st]);
            } else {
                cp_async_arrive(&full[st]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (map && w == 0)  // the copy engine's, before the block may end: nobody else may have waited for them
        for (int t = max(0, n - NST); t < n; ++t) mbar_drain(&full[t % NST], (t / NST) & 1);
    if (S::WIDEN)  // the tiles still on their way
        for (int t = n >= NST ? n - NST : 0; ok && t < n; ++t) ok = widen(t);
}

// ------------------------------------------------------------------ products
// Two threads, one for the scores and one for the outputs: issuing a tile's 8
// products takes either of them 600 to 1,100 cycles, and the rows wait for the
// scores (one thread for both: 241 us for the verify batch against 232).  Their
// loops are unrolled by two only, and the loaders' not at all: all roles' loops
// together have to fit the instruction caches (draft trees 91 us otherwise, 88
// so).  With e4m3 they issue in time only when unrolled: two sequences of 131,001
// slots 204 us at 40 rows and 249 at 84 like the others, 194 and 240 so.
template <typename T, typename C, int D>
__device__ void rows_scores(const AttParams &p, Cursor c, char *smem, RowsCtl *ctl, unsigned *err)
{
    using S = RowsShape<C, D>;
    constexpr uint32_t SHAPE = mma_shape(std::is_same<typename MmaOf<T, C>::type, __nv_bfloat16>::value, false, AR_KEYS);
    constexpr int KST = S::K_STAGES;
    const uint32_t base = smem_u32(smem), tm_s = ctl->tmem;
    int n = 0, item = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        const int tiles = last_tile(c) - first_tile(c);
        if (tiles == 0) continue;
        const uint64_t q = desc_k_major(base + S::Q_AT + (item & 1) * S::TILE);
        if (!rows_wait1(ctl, &ctl->q_full[item & 1], (item >> 1) & 1, err)) return;
        for (int i = 0; i < tiles; ++i, ++n) {
            if (!rows_wait1(ctl, &ctl->k_full[n % KST], (n / KST) & 1, err)) return;
            if (n >= 2 && !rows_wait1(ctl, &ctl->p_full[n & 1], ((n - 2) >> 1) & 1, err)) return;  // its place has been read
            tc_fence_after();
            fence_async_shared();  // K was written by asynchronous copies of threads, q by threads
            const uint64_t k = desc_k_major(base + S::K_AT + (n % KST) * S::TILE);
#pragma unroll(S::WIDEN ? D / 16 : 2)
            for (int ks = 0; ks < D / 16; ++ks) {
                const int off = ((ks >> 2) * (AR_KEYS * 128) + (ks & 3) * 32) >> 4;
                tc_mma(tm_s + (n & 1) * AR_KEYS, q + off, k + off, SHAPE, ks > 0);
            }
            tc_commit(&ctl->s_full[n & 1]);
            tc_commit(&ctl->k_empty[n % KST]);
        }
        ++item;
    }
}
template <typename T, typename C, int D>
__device__ void rows_outputs(const AttParams &p, Cursor c, char *smem, RowsCtl *ctl, unsigned *err)
{
    using S = RowsShape<C, D>;
    constexpr uint32_t SHAPE = mma_shape(std::is_same<typename MmaOf<T, C>::type, __nv_bfloat16>::value, true, D);
    constexpr int VST = S::V_STAGES;
    const uint32_t base = smem_u32(smem), tm_p = ctl->tmem + 256, tm_o = ctl->tmem + 384;
    int n = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        const int tiles = last_tile(c) - first_tile(c);
        for (int i = 0; i < tiles; ++i, ++n) {
            if (!rows_wait1(ctl, &ctl->v_full[n % VST], (n / VST) & 1, err)) return;
            if (!rows_wait1(ctl, &ctl->p_full[n & 1], (n >> 1) & 1, err)) return;
            tc_fence_after();
            fence_async_shared();
            const uint64_t v = desc_n_major(base + S::V_AT + (n % VST) * S::TILE, AR_KEYS * 128);
#pragma unroll(S::WIDEN ? AR_KEYS / 16 : 2)
            for (int ks = 0; ks < AR_KEYS / 16; ++ks)
                tc_mma_ta(tm_o, tm_p + (n & 1) * (AR_KEYS / 2) + ks * 8, v + ks * (2048 >> 4), SHAPE, i > 0 || ks > 0);
            tc_commit(&ctl->o_done[n & 1]);
            tc_commit(&ctl->v_empty[n % VST]);
        }
    }
}

// ------------------------------------------------------------------ q
// Two warps, an item ahead of the others: q of every copy's rows, and what
// the new tokens see.  For an e4m3 cache each row by a power of two into f16's
// range.
template <typename T, typename C, int D, int COLS>
__device__ void rows_prepare(const AttParams &p, Cursor c, char *smem, RowsCtl *ctl, unsigned *err, int lt)
{
    using S = RowsShape<C, D>;
    using M = typename MmaOf<T, C>::type;
    int item = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        if (first_tile(c) == last_tile(c)) continue;
        if (item == p.give_up.item && static_cast<int>(blockIdx.x) == p.give_up.block) {  // the self-test
            *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
            atomicExch(err, static_cast<unsigned>(STATUS_TIMEOUT));
            return;
        }
        const int place = item & 1, row0 = c.row_tile * COLS, live = min(COLS, p.rows - row0);
        char *qs = smem + S::Q_AT + place * S::TILE;
        if (item >= 2 && !rows_wait(ctl, &ctl->q_empty[place], ((item >> 1) - 1) & 1, err)) return;
        for (int t = lt; t < p.w.T; t += AR_PREPARE)
            ctl->sees[place][t] = t < c.s.fresh ? visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, t) : 0ull;
        // rows at a time, 4 or 8; four loads of a thread on their way together (one by one they took 6 us)
        constexpr int CH = D / 8, STEP = AR_PREPARE / CH, AHEAD = 4;
        const int ch = lt % CH;
#pragma unroll 1
        for (int b0 = 0; b0 < COLS; b0 += AHEAD * STEP) {
            uint4 in[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int r = b0 + i * STEP + lt / CH, t = (row0 + r) / p.group, g = (row0 + r) - t * p.group;
                in[i] = make_uint4(0, 0, 0, 0);
                if (r < live && t < c.s.fresh)
                    in[i] = *reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.q) + ((static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g) * D + ch * 8);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int r = b0 + i * STEP + lt / CH;
                uint4 raw = in[i];
                if (S::WIDEN) {
                    const T *y = reinterpret_cast<const T *>(&raw);
                    float x[8], top = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = Num<T>::up(y[e]);
                        top = fabsf(x[e]) < CUDART_INF_F ? fmaxf(top, fabsf(x[e])) : top;
                    }
#pragma unroll
                    for (int o = CH / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int e2 = top > 0.0f ? max(-120, min(120, 14 - ilogbf(top))) : 0;
                    const float up = exp2f(static_cast<float>(e2));
                    if (ch == 0 && r < COLS)
#pragma unroll
                        for (int k = 0; k < AR_ROWS; k += COLS) ctl->q_power[place][k + r] = static_cast<signed char>(e2);
                    raw = make_uint4(pack_mma<M>(x[0] * up, x[1] * up), pack_mma<M>(x[2] * up, x[3] * up),
                                     pack_mma<M>(x[4] * up, x[5] * up), pack_mma<M>(x[6] * up, x[7] * up));
                }
                if (r < COLS)
#pragma unroll
                    for (int k = 0; k < AR_ROWS; k += COLS) *reinterpret_cast<uint4 *>(qs + panel_at(k + r, ch)) = raw;
            }
        }
        fence_async_shared();
        mbar_arrive(&ctl->q_full[place]);
        ++item;
    }
}

// ------------------------------------------------------------------ rows
// 32 bytes to a 16-byte aligned address: at once where it allows.
__device__ __forceinline__ void store32(void *at, const uint32_t (&y)[8])
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

template <int N> __device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory"); }

// The two warps that have the same rows.
__device__ __forceinline__ void pair_sync(int w) { asm volatile("bar.sync %0, 64;" ::"r"(2 + w) : "memory"); }

// Columns of an item's rows, or of the block's piece of them, that the products
// could not have: those where a new token that the row sees has an infinity or
// NaN in v (cleared there), and those that are NaN.  A warp a row, anew, key by
// key in 32 bits and without weights of keys that the row does not have.  Rows
// whose scores are NaN, or that have a bad page, stay as they are.
template <typename T, typename C, int D, int COLS>
__device__ __forceinline__ void rows_again(const AttParams &p, const Cursor &c, long long begin, int tid)
{
    constexpr int PER = D / 32;  // columns of a lane, next to one another
    const int lane = tid & 31, row0 = c.row_tile * COLS, live = min(COLS, p.rows - row0), t0 = first_tile(c), t1 = last_tile(c);
    if (t0 == t1) return;
    const bool whole = t0 == 0 && t1 == c.tiles;
    float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * (AR_ROWS * (D + 2));
    const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
    const int end = min(t1 * AR_KEYS, c.s.total);
    const float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
    auto row_of = [&](const PoolView &pool, int page, int j) {
        return reinterpret_cast<const C *>(row_ptr(p.c, pool, page, j, c.h)) + PER * lane;
    };
#pragma unroll 1
    for (int r = tid >> 5; r < live; r += RowsWarps<COLS>::SOFTMAX / 32) {
        const int token = (row0 + r) / p.group, g = row0 + r - token * p.group;
        const int64_t at = ((static_cast<int64_t>(c.b) * p.w.T + token) * p.q_heads + c.h * p.group + g) * D + PER * lane;
        const unsigned long long see =
            token < c.s.fresh ? visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, token) : 0ull;
        if (see == 0) continue;
        T *out = static_cast<T *>(p.out) + at;
        float *piece = part + 2 * AR_ROWS + r * D + PER * lane;
        unsigned redo = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float y = whole ? Num<T>::up(out[e]) : piece[e];
            if (y != y) redo |= 1u << e;
        }
#pragma unroll 1
        for (int j = max(c.s.ctx, t0 * AR_KEYS); j < end; ++j) {
            const int page = page_of(p.c, table, j);
            if (page < 0 || !(see >> (j - c.s.ctx) & 1)) continue;
            const C *v = row_of(p.c.v, page, j);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (!(fabsf(Num<C>::up(v[e])) < CUDART_INF_F)) redo |= 1u << e;
        }
        if (!__any_sync(0xffffffffu, redo != 0)) continue;
        float m = -CUDART_INF_F, l = 0.0f, q[PER], x[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            q[e] = Num<T>::up(static_cast<const T *>(p.q)[at + e]);
            x[e] = 0.0f;
        }
        bool fine = true;
#pragma unroll 1
        for (int j = t0 * AR_KEYS; fine && j < end; ++j) {
            const int page = page_of(p.c, table, j);
            fine = page >= 0;
            if (!fine || (j >= c.s.ctx && !(see >> (j - c.s.ctx) & 1))) continue;
            const C *k = row_of(p.c.k, page, j), *v = row_of(p.c.v, page, j);
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < PER; ++e) s += q[e] * Num<C>::up(k[e]);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= factor;
            fine = s == s;
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
            if (!(redo >> e & 1)) continue;
            if (whole)
                out[e] = Num<T>::down(x[e] * unit);
            else
                piece[e] = x[e] * unit;
        }
    }
}

// What is left of a block's range, from an item's beginning on, after a wait
// gave up: NaN for every row, the pieces of a shared item among them.  Items
// without keys have what they always have.
template <typename T, int D, int COLS> __device__ __forceinline__ void rows_lost(const AttParams &p, Cursor c, int tid)
{
    constexpr int THREADS = RowsWarps<COLS>::SOFTMAX;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        const AttRows rows{c.b, c.h, c.row_tile * COLS, min(COLS, p.rows - c.row_tile * COLS)};
        const bool empty = c.s.total == 0 && !c.s.bad;
        if (c.s.total == 0 || c.end >= c.first + c.tiles) {  // whole
            const float m = empty ? -CUDART_INF_F : CUDART_NAN_F;
            for (int i = tid; i < rows.live * (D / 4); i += THREADS)
                write_row<T, D>(p, rows, i / (D / 4), i % (D / 4) * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f), m, 0.0f, 1.0f);
            if (tid == 0 && p.row_status && c.h == 0 && c.row_tile == 0)
                p.row_status[c.b] = c.s.bad ? KV_STATUS_BAD : empty ? 0 : STATUS_TIMEOUT;
        } else {  // a piece in the second place; its maximum is enough
            float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * (AR_ROWS * (D + 2));
            for (int r = tid; r < rows.live; r += THREADS) {
                part[r] = CUDART_NAN_F;
                part[AR_ROWS + r] = 0.0f;
            }
            note_split(p, c, rows, c.first, tid);
        }
    }
}

// The items that begin before tile `done`, again; then, where that is not the
// range's end, NaN for those behind the one that a wait cost.  Out of line, away
// from the loops that have to fit the instruction caches.  (What few lines of it
// stood in the rows' epilogue cost the verify batch up to 25 us by the place
// alone that the loops then had.)
template <typename T, typename C, int D, int COLS>
__device__ __noinline__ void rows_finish(const AttParams &p, long long begin, long long done, int tid)
{
    Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid & 31);
    for (; c.at < done; next_item(c, p.w, p.c)) rows_again<T, C, D, COLS>(p, c, begin, tid);
    if (c.at >= c.end) return;
    next_item(c, p.w, p.c);
    rows_lost<T, D, COLS>(p, c, tid);
}

// COLS: rows of a copy, and its keys of a tile; a thread takes these, or half of them.
template <typename T, typename C, int D, int COLS>
__device__ void rows_softmax(const AttParams &p, Cursor c, char *smem, RowsCtl *ctl, unsigned *err, int tid)
{
    using S = RowsShape<C, D>;
    using M = typename MmaOf<T, C>::type;
    constexpr int COPIES = AR_ROWS / COLS, PART = AR_ROWS * (D + 2);
    using W = RowsWarps<COLS>;
    constexpr float UP = Weights<M>::UP;
    constexpr int HALVES = W::HALVES, KEYS = COLS / HALVES;
    const int half = tid / AR_ROWS, lane_row = tid % AR_ROWS, copy = lane_row / COLS, r = lane_row % COLS;
    const uint32_t quarter = static_cast<uint32_t>(lane_row & ~31) << 16;
    const uint32_t tm_s = ctl->tmem + quarter + copy * COLS + half * KEYS,
                   tm_p = ctl->tmem + quarter + 256 + copy * (COLS / 2) + half * (KEYS / 2), tm_o = ctl->tmem + quarter + 384;
    const long long begin = c.at;
    // An infinity in a cached slot of V, which all rows see, meets a weight of 0 in the copies that do not have its key:
    // rows with NaN are looked at again when the range is done.
    constexpr bool LOOK_AGAIN = COPIES > 1 && !S::WIDEN;
    // the keys of other copies never get a probability
    if (COPIES > 1) {
        uint32_t zero[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll
        for (int i = 0; i < 128; i += 32) tc_st32(ctl->tmem + quarter + 256 + i, zero);
        tc_wait_st();
    }
    int n = 0, item = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        const int t0 = first_tile(c), t1 = last_tile(c), row0 = c.row_tile * COLS, live = min(COLS, p.rows - row0);
        const AttRows rows{c.b, c.h, row0, live};
        const float v_scale = p.c.v_scale ? __ldg(p.c.v_scale + c.h) : 1.0f;
        const bool mine = r < live;
        const int token = (row0 + r) / p.group;
        unsigned long long see = 0;
        float m = -CUDART_INF_F, l = 0.0f;  // a maximum so far less UP: what l and O are sums against
        float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        bool any_bad = c.s.bad, ok = true;
        const int place = item & 1;
        using Merge = RowsMerge<D>;
        static_assert(sizeof(Merge) <= S::TILE, "the exchange fits q's place");
        Merge *merge = reinterpret_cast<Merge *>(smem + S::Q_AT + place * S::TILE);  // once all scores are there
        if (t0 < t1) {
            ok = rows_wait(ctl, &ctl->q_full[place], (item >> 1) & 1, err);
            if (mine && token < c.s.fresh) see = ctl->sees[place][token];
            if (S::WIDEN) factor *= exp2f(-static_cast<float>(ctl->q_power[place][lane_row]));
            const bool works = __any_sync(0xffffffffu, mine);
            for (int tile = t0; tile < t1; ++tile, ++n) {  // to its end even after a wait gave up: the halves meet at each tile
                ok = ok && rows_wait(ctl, &ctl->s_full[n & 1], (n >> 1) & 1, err);
                tc_fence_after();
                __syncwarp();
                if (works) {
                    float x[KEYS];
#pragma unroll
                    for (int i = 0; i < KEYS; i += 32) {
                        uint32_t y[32];
                        tc_ld32(y, tm_s + (n & 1) * AR_KEYS + i);
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[i + k] = __fmul_rn(__uint_as_float(y[k]), factor);  // as m is: not fused with the difference
                    }
                    const int j0 = tile * AR_KEYS + copy * COLS + half * KEYS;
                    if (j0 + KEYS > c.s.ctx) {
#pragma unroll
                        for (int i = 0; i < KEYS; i += 32) {
                            const int o = c.s.ctx - (j0 + i);  // the first new token's column, from here
                            unsigned bits = o >= 32 ? 0xffffffffu : o > 0 && see ? (1u << o) - 1u : 0u;
                            if (o < 32 && o > -64) bits |= static_cast<unsigned>(o >= 0 ? see << o : see >> -o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[i + k] = bits >> k & 1 ? x[i + k] : -CUDART_INF_F;
                        }
                    }
                    float top = x[0];
#pragma unroll
                    for (int i = 1; i + 1 < KEYS; i += 2) top = fmax3(top, x[i], x[i + 1]);
                    top = fmaxf(top, x[KEYS - 1]);
                    if (HALVES == 2) {  // the maximum of both halves, by the two warps that have these rows
                        pair_sync(lane_row / 32);  // the last tile's has been read
                        ctl->top[tid] = top;
                        pair_sync(lane_row / 32);
                        top = fmaxf(top, ctl->top[tid ^ AR_ROWS]);
                    }
                    if (tile == t0) {
                        m = top - UP;
                    } else if (__any_sync(0xffffffffu, top - m > UP + Weights<M>::LAG)) {  // as a difference: a sum may round up to a score 16 above
                        const float grown = fmaxf(m, top - UP), a = grown == -CUDART_INF_F ? 0.0f : fast_exp2(m - grown);
                        m = grown;
                        l *= a;
                        ok = ok && rows_wait(ctl, &ctl->o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err);
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
                    const float base = m == -CUDART_INF_F ? 0.0f : m;
                    float s0 = 0.0f, s1 = 0.0f;
                    uint32_t pk[KEYS / 2];
#pragma unroll
                    for (int i = 0; i < KEYS; i += 2) {
                        const float a = fast_exp2(x[i] - base), b = fast_exp2(x[i + 1] - base);
                        s0 += a;
                        s1 += b;
                        // rounded to 16 bits for the product (half a step of the type each); l keeps 32 bits
                        pk[i / 2] = pack_mma<M>(a, b);
                    }
                    l += s0 + s1;
                    // its place was read by the product two tiles ago
                    if (n >= 2) ok = ok && rows_wait(ctl, &ctl->o_done[n & 1], ((n - 2) >> 1) & 1, err);
                    tc_fence_after();
                    if (KEYS == 32) {
                        tc_st16(tm_p + (n & 1) * (AR_KEYS / 2), *reinterpret_cast<uint32_t(*)[16]>(pk));
                    } else {
#pragma unroll
                        for (int i = 0; i < KEYS / 2; i += 32)
                            tc_st32(tm_p + (n & 1) * (AR_KEYS / 2) + i, *reinterpret_cast<uint32_t(*)[32]>(pk + i));
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                mbar_arrive(&ctl->p_full[n & 1]);
            }
            if (ok) ok = rows_wait(ctl, &ctl->o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err);
            tc_fence_after();
            if (tid == 0 && *reinterpret_cast<volatile int *>(&ctl->odd[item_flags(item)])) *reinterpret_cast<volatile int *>(&ctl->lost) = 1;
            any_bad |= *reinterpret_cast<volatile int *>(&ctl->bad[item_flags(item)]) != 0;
            rows_sync<W::SOFTMAX>();  // all have read them, and all scores
        }
        if (see == 0) {
            m = -CUDART_INF_F;
            l = 0.0f;
        }
        const bool tiles = t0 < t1;
        if (tiles) {
            merge->ms[tid] = m;
            merge->ls[tid] = l;
        }
        if (tid == 0) {
            ctl->stop = *reinterpret_cast<volatile int *>(&ctl->dead);
            if (tiles) {
                ctl->odd[item_flags(item)] = 0;
                ctl->bad[item_flags(item)] = 0;
            }
        }
        rows_sync<W::SOFTMAX>();
        const bool stop = *reinterpret_cast<volatile int *>(&ctl->stop) != 0;
        any_bad |= stop;
        float all_m = -CUDART_INF_F, all_l = 0.0f;
        if (tiles) {
#pragma unroll
            for (int k = 0; k < COPIES * HALVES; ++k) all_m = fmaxf(all_m, merge->ms[k * COLS + r]);
        }
        const float base = all_m == -CUDART_INF_F ? 0.0f : all_m, of_pair = l + (HALVES == 2 && tiles ? merge->ls[tid ^ AR_ROWS] : 0.0f),
                    mine_a = of_pair == 0.0f ? 0.0f : fast_exp2(m - base);
        if (tiles) {
#pragma unroll
            for (int k = 0; k < COPIES * HALVES; ++k) {
                const float lk = merge->ls[k * COLS + r];
                if (lk != 0.0f) all_l += lk * fast_exp2(merge->ms[k * COLS + r] - base);
            }
        }
        const bool whole = c.s.total == 0 || (t0 == 0 && t1 == c.tiles);
        float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * PART;
        const float out_m = any_bad ? CUDART_NAN_F : all_m;
        // the row's place, and what is written where there is no sum (0) or a bad sequence (NaN)
        const int64_t row_at = (static_cast<int64_t>(c.b) * p.w.T + token) * p.q_heads + c.h * p.group + (row0 + r) - token * p.group;
        const bool none = all_m == -CUDART_INF_F && all_l == 0.0f, fixed = none || any_bad;
        const float instead = any_bad ? CUDART_NAN_F : 0.0f, out_scale = v_scale / all_l;
        if (copy == 0 && half == 0 && mine) {
            if (!whole) {
                part[r] = out_m;
                part[AR_ROWS + r] = all_l;
            } else if (p.lse) {
                p.lse[row_at] = any_bad ? CUDART_NAN_F : none ? -CUDART_INF_F : LN2 * (all_m + log2f(all_l));
            }
        }
#pragma unroll 1
        for (int d0 = half * (D / HALVES); d0 < (half + 1) * (D / HALVES); d0 += 32) {
            // each 32 columns are put together by another copy; of the halves each takes half the columns
            const int keeper = (d0 >> 5) % COPIES;
            float x[32];
            __syncwarp();
            if (tiles && !stop) {
                uint32_t y[32];
                tc_ld32(y, tm_o + d0);
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = mine_a == 0.0f ? 0.0f : __uint_as_float(y[k]) * mine_a;
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = 0.0f;
            }
            if (COPIES > 1 && tiles) {
                float *buf = merge->x[(d0 >> 5) % Merge::ROUNDS];
                if (Merge::ROUNDS == 1 && d0 > 0) rows_sync<W::SOFTMAX>();
                if (copy != keeper) {
                    float *to = buf + (((copy - keeper + COPIES) % COPIES - 1) * COLS + r) * 33;
#pragma unroll
                    for (int k = 0; k < 32; ++k) to[k] = x[k];
                }
                rows_sync<W::SOFTMAX>();
                if (copy == keeper) {
#pragma unroll
                    for (int q = 0; q < COPIES - 1; ++q)
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] += buf[(q * COLS + r) * 33 + k];
                }
            }
            if (copy != keeper || !mine) continue;
            if (LOOK_AGAIN) {
                float sum[4];  // NaN if one of them is
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] = x[k];
#pragma unroll
                for (int k = 4; k < 32; ++k) sum[k & 3] += x[k];
                const float any = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (any != any) *reinterpret_cast<volatile int *>(&ctl->lost) = 1;
            }
            // 32 bytes a store: a thread's row is its own, and half a sector at a time cost twice the transactions
            if (!whole) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(x[k + e]);
                    store32(part + 2 * AR_ROWS + r * D + d0 + k, y);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = fixed ? instead : x[k] * out_scale;
#pragma unroll
                for (int k = 0; k < 32; k += 16) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = pack_mma<T>(x[k + 2 * e], x[k + 2 * e + 1]);
                    store32(static_cast<T *>(p.out) + row_at * D + d0 + k, y);
                }
            }
        }
        tc_fence_before();
        if (!whole)
            note_split(p, c, rows, begin, tid);
        else if (tid == 0 && p.row_status && c.h == 0 && c.row_tile == 0)
            p.row_status[c.b] = c.s.bad ? KV_STATUS_BAD : stop ? STATUS_TIMEOUT : any_bad ? KV_STATUS_BAD : 0;
        if (tiles) {
            mbar_arrive(&ctl->q_empty[place]);
            ++item;
        }
        rows_sync<W::SOFTMAX>();
        if (stop) break;
    }
    // c.at before the end: a wait gave up
    if (*reinterpret_cast<volatile int *>(&ctl->lost) || c.at < c.end) rows_finish<T, C, D, COLS>(p, begin, c.at, tid);
}

template <typename T, typename C, int D, int COLS>
__global__ void __launch_bounds__(RowsWarps<COLS>::THREADS, 1)
    attention_rows_kernel(const AttParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const int maps)
{
    using S = RowsShape<C, D>;
    using W = RowsWarps<COLS>;
    extern __shared__ __align__(1024) char smem[];  // the swizzle's rows of 128 bytes come in groups of eight
    RowsCtl *ctl = reinterpret_cast<RowsCtl *>(smem + S::CTL_AT);
    const int tid = threadIdx.x, warp = tid >> 5;
    unsigned *err = p.error;
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) {
            mbar_init(&ctl->k_full[i], 128);
            mbar_init(&ctl->v_full[i], 128);
            mbar_init(&ctl->k_empty[i], 1);
            mbar_init(&ctl->v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], W::SOFTMAX);
            mbar_init(&ctl->o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->q_full[i], AR_PREPARE);
            mbar_init(&ctl->spare[i], 1);
            mbar_init(&ctl->q_empty[i], W::SOFTMAX);
        }
        for (int i = 0; i < AR_ITEMS; ++i) ctl->odd[i] = 0, ctl->bad[i] = 0;
        ctl->dead = ctl->stop = ctl->lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W::SOFTMAX / 32) tmem_alloc(&ctl->tmem, 512);
    chain_begin();
    const Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid & 31);
    if (tid < 2) p.split[blockIdx.x * 2 + tid].n = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c.at == c.end) {  // the whole block
        if (warp == W::SOFTMAX / 32) tmem_free(ctl->tmem, 512);
        return;
    }
    // registers: launched with 128 a thread, 4 x 128 = 208 + 80 + 2 x 112, or with 96, 5 x 96 = 2 x 128 + 80 + 2 x 72 and
    // 2 x 120 + 3 x 80 (more for the widening); what spills comes back from the L2, shared memory has most of the L1
    const int role = warp - W::SOFTMAX / 32;
    if (role < 0) {
        if (W::HALVES == 1)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else if (S::WIDEN)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        rows_softmax<T, C, D, COLS>(p, c, smem, ctl, err, tid);
    } else if (role < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (role < 2 && (tid & 31) == 0) {
            if (role == 0)
                rows_scores<T, C, D>(p, c, smem, ctl, err);
            else
                rows_outputs<T, C, D>(p, c, smem, ctl, err);
            // what was issued ends before the block may: others may have given up on it
            tc_commit(&ctl->spare[role]);
            mbar_drain(&ctl->spare[role], 0);
        }
        __syncwarp();
        if (role >= 2) rows_prepare<T, C, D, COLS>(p, c, smem, ctl, err, tid - W::SOFTMAX - 64);
    } else {
        if (W::HALVES == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        else if (S::WIDEN)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (role < 8)
            rows_load<C, D, 0>(p, c, smem, ctl, err, tid & 127, maps ? &map_k : nullptr);
        else
            rows_load<C, D, 1>(p, c, smem, ctl, err, tid & 127, maps ? &map_v : nullptr);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W::SOFTMAX / 32) tmem_free(ctl->tmem, 512);
}

template <typename T, typename C, int D, int COLS>
static cudaError_t launch_cols(AttParams p, const KvLaunch &L, cudaStream_t st)
{
    using S = RowsShape<C, D>;
    constexpr int SMEM = S::CTL_AT + static_cast<int>(sizeof(RowsCtl));
    static_assert(SMEM <= 232448, "shared memory of a block");
    auto kernel = attention_rows_kernel<T, C, D, COLS>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    p.w.tile = AR_KEYS;
    p.w.row_tiles = (p.rows + COLS - 1) / COLS;
    CUtensorMap map_k{}, map_v{};
    const bool maps = pool_map(&map_k, L, false) && pool_map(&map_v, L, true);
    e = launch_chained(kernel, dim3(ATT_SMS), RowsWarps<COLS>::THREADS, SMEM, st, p, map_k, map_v, static_cast<int>(maps));
    return e != cudaSuccess ? e : launch_join(p, std::is_same<T, __half>::value ? SPV_F16 : SPV_BF16, D, AR_ROWS, ATT_SMS, st);
}
template <typename T, typename C, int D> static cudaError_t launch_dim(const AttParams &p, const KvLaunch &L, cudaStream_t st)
{
    if constexpr (sizeof(C) == 2) {  // an e4m3 cache comes here with more than 32 rows
        if (p.rows <= 32) return launch_cols<T, C, D, 32>(p, L, st);
    }
    if (p.rows <= 64) return launch_cols<T, C, D, 64>(p, L, st);
    return launch_cols<T, C, D, 128>(p, L, st);
}
template <typename T, typename C> static cudaError_t launch_types(const AttParams &p, const KvLaunch &L, cudaStream_t st)
{
    return L.cache.head_dim == 64 ? launch_dim<T, C, 64>(p, L, st) : launch_dim<T, C, 128>(p, L, st);
}

size_t attention_rows_part_floats(int head_dim)
{
    return static_cast<size_t>(ATT_SMS) * 2 * AR_ROWS * (head_dim + 2);
}

cudaError_t launch_attention_rows(const AttParams &p, const KvLaunch &L, cudaStream_t st)
{
    const bool eight = L.cache.dtype == SPV_E4M3;
    if (L.dtype == SPV_BF16)
        return eight ? launch_types<__nv_bfloat16, __nv_fp8_e4m3>(p, L, st) : launch_types<__nv_bfloat16, __nv_bfloat16>(p, L, st);
    return eight ? launch_types<__half, __nv_fp8_e4m3>(p, L, st) : launch_types<__half, __half>(p, L, st);
}

}  // namespace spv
