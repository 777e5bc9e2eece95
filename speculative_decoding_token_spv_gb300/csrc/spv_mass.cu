// spv_mass.cu -- the attention weight that each cached key received from the
// tokens that stand after a verify step, added up.
//
// The weights are recomputed from q, K and the attention's log-sum-exp:
// exp(s - lse) needs no second pass and no maximum, so K is read once, no
// score is kept between the calls and no piece has to be joined.  Per 128-key
// tile the 5th-generation tensor cores give the transposed scores, a key a
// lane and a counted row a column of tensor memory: the sum over the rows is
// then a thread's own, with no exchange between threads.  (On warp-level tensor
// cores, whose lanes share a key's column, masks, exchanges and fragments came
// to 750 instructions per 16 keys: 329 us for the case below.)
//
// What bounds it is reading K, the old weights and writing the new ones once: 64
// sequences of up to 8,191 slots, 8 key heads of 8 query heads, D = 128, bf16,
// 704 MB: 128 us, 5.5 TB/s, 81% of a copy's rate.
//
// One block an SM has an equal range of all tiles (Work, Cursor).  Two groups
// of four loader warps take turns at the tiles, gathering K through the page
// table with asynchronous copies (e4m3 is widened to f16 by the thread that
// loaded it); three warps bring q and the rows' constants an item ahead; one
// thread issues the products; four warps, a key a thread, sum and write.
//
// Every wait is bounded; one that gives up ends the block in order: the weights
// that it still had to write become NaN, and the row_status of their sequences
// SPV_ERR_TIMEOUT.  So that no other block can overwrite that, a small kernel
// before this one writes all statuses.
#include "spv_mma.cuh"
#include "spv_tcgen.cuh"

namespace spv {

constexpr int MASS_SMS = 152;
constexpr int MASS_KEYS = 128;
constexpr int MASS_THREADS = 512;  // warps 0-3 keys, 4 products, 5-7 q, 8-11 and 12-15 K
constexpr int MASS_BUFFERS = 4;    // of scores in tensor memory, 128 columns each

struct MassParams {
    PagedView c;
    Work w;
    const void *q;
    const float *lse, *mass_in;
    const int32_t *parent, *accept, *nodes;
    float *mass_out;
    int64_t stride;
    int32_t *row_status;
    int q_heads, group;
    float scale_log2, decay;
    GiveUp give_up;
};

// Which new tokens of sequence b count; *bad if what says so is out of range.
__device__ __forceinline__ unsigned long long counted_tokens(const MassParams &p, int b, bool *bad)
{
    const int k = __ldg(p.accept + b);
    if (k < -1 || k > p.w.T - 1) {
        *bad = true;
        return 0;
    }
    if (k < 0) return 0;
    if (!p.nodes) return (2ull << k) - 1ull;
    unsigned long long m = 1;
    for (int i = 0; i < k; ++i) {
        const int n = __ldg(p.nodes + static_cast<int64_t>(b) * p.w.T + i);
        if (static_cast<unsigned>(n) >= static_cast<unsigned>(p.w.T)) {
            *bad = true;
            return 0;
        }
        m |= 1ull << n;
    }
    return m;
}

// The tokens that count and the rows that they make, of the item's sequence;
// no rows where they are out of range (`bad`).  Kept while the heads of a
// sequence pass by.
struct Counted {
    int b = -1, rows = 0;
    unsigned long long tokens = 0;
    bool bad = false;
    __device__ __forceinline__ void at(const MassParams &p, const Cursor &c)
    {
        if (c.b == b) return;
        b = c.b;
        bad = c.s.bad || c.s.total > p.stride;
        tokens = counted_tokens(p, b, &bad);
        if (c.s.fresh < 64) tokens &= (1ull << (c.s.fresh < 0 ? 0 : c.s.fresh)) - 1ull;
        rows = bad || c.s.total == 0 ? 0 : __popcll(tokens) * p.group;
    }
};

// row_status of every sequence, a block each.
__global__ void __launch_bounds__(128) mass_status_kernel(const MassParams p)
{
    const int b = blockIdx.x;
    chain_begin();
    const SeqLens s = seq_lens(p.w.ctx_lens, p.w.new_lens, b, p.w.T, p.c, p.w.idle);
    bool bad = s.bad || s.total > p.stride;
    counted_tokens(p, b, &bad);
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    int any = bad;
    for (int g = threadIdx.x; s.total > 0 && g <= (s.total - 1) >> p.c.page_shift; g += 128) any |= page_of(p.c, table, g << p.c.page_shift) < 0;
    any = __syncthreads_or(any);
    if (threadIdx.x == 0) p.row_status[b] = any ? KV_STATUS_BAD : 0;
}

// ROWS rows at once; more go in several passes over the item's tiles.
template <typename C, int D> struct MassShape {
    static constexpr bool WIDEN = sizeof(C) == 1;
    static constexpr int ROWS = D == 256 ? (WIDEN ? 32 : 64) : 128;
    static constexpr int Q = ROWS * D * 2, TILE = MASS_KEYS * D * 2, RAW = MASS_KEYS * D;
    // Both even: a stage is always the same group's, which so meets its barrier's phases one by one.
    static constexpr int K_STAGES = WIDEN ? (D == 64 ? 4 : 2) : (D == 64 ? 8 : D == 128 ? 4 : 2);
    static constexpr int RAW_STAGES = WIDEN ? (D == 64 ? 8 : D == 128 ? 4 : 2) : 0;
    static constexpr int Q_AT = 0, K_AT = 2 * Q, RAW_AT = K_AT + K_STAGES * TILE, CTL_AT = RAW_AT + RAW_STAGES * RAW;
};

template <int ROWS> struct MassCtl {
    uint64_t k_full[8], k_empty[8], s_full[MASS_BUFFERS], s_empty[MASS_BUFFERS], q_full[2], q_empty[2], spare;
    unsigned long long sees[2][ROWS];
    alignas(16) float2 row[2][ROWS];  // (read in pairs) what a unit of the stored q.k stands for, and the log-sum-exp, in powers of two
    int careful[2];       // number (from 1) of the last pass in which some row gives nothing: masks are then looked at everywhere
    uint32_t tmem;
    int dead;
};

template <typename Ctl> __device__ __forceinline__ bool mass_wait1(Ctl *ctl, uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63) == 63 && *reinterpret_cast<volatile int *>(&ctl->dead)) return false;
    }
    *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
    return false;
}
template <typename Ctl> __device__ __forceinline__ bool mass_wait(Ctl *ctl, uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mass_wait1(ctl, bar, parity));
}

__device__ __forceinline__ int mass_first(const Cursor &c) { return static_cast<int>(c.at - c.first); }
__device__ __forceinline__ int mass_last(const Cursor &c)
{
    if (c.s.total == 0) return mass_first(c);
    const long long e = c.first + c.tiles;
    return static_cast<int>((c.end < e ? c.end : e) - c.first);
}
// Byte of 16-byte chunk `chunk` of row `row` in an operand of ROWS rows.
template <int ROWS> __device__ __forceinline__ uint32_t mass_panel(int row, int chunk)
{
    return (chunk >> 3) * (ROWS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// One of the two groups of loader warps: the tiles of its parity.
template <typename C, int D, typename Ctl>
__device__ void mass_load(const MassParams &p, Cursor c, char *smem, Ctl *ctl, int lt, int turn)
{
    using S = MassShape<C, D>;
    constexpr int CH = D * static_cast<int>(sizeof(C)) / 16, CPL = CH > 32 ? 32 : CH, RPI = 32 / CPL, KST = S::K_STAGES;
    constexpr int RST = S::RAW_STAGES > 0 ? S::RAW_STAGES / 2 : 1;
    const int lane = lt & 31, w = lt >> 5, chunk = lane % CPL, sub = lane / CPL;
    const uint32_t base = smem_u32(smem);
    const int mask = (1 << p.c.page_shift) - 1;
    Counted count;
    int n = 0, mine_n = 0;  // tiles so far, and those of this group
    // e4m3: widens this group's tile number t (tile 2 t + turn of all), whose copies have landed.
    auto widen = [&](int t) -> bool {
        const int all = 2 * t + turn, st = all % KST;
        if (all >= KST && !mass_wait(ctl, &ctl->k_empty[st], (all / KST - 1) & 1)) return false;
        const char *raw = smem + S::RAW_AT + (turn * RST + t % RST) * S::RAW;
        char *to = smem + S::K_AT + st * S::TILE;
#pragma unroll 8
        for (int i = 0; i < 32 / RPI; ++i) {
            const int row = 32 * w + i * RPI + sub;
            const uint4 x = *reinterpret_cast<const uint4 *>(raw + row * D + chunk * 16);
            const uint32_t b[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = e4m3x2_to_f16x2(b[k] & 0xffffu);
                y[2 * k + 1] = e4m3x2_to_f16x2(b[k] >> 16);
            }
            const bool swap = (chunk >> 2) & 1;  // lanes of two panels store their halves in opposite order
            const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
            *reinterpret_cast<uint4 *>(to + mass_panel<MASS_KEYS>(row, 2 * chunk + swap)) = swap ? hi : lo;
            *reinterpret_cast<uint4 *>(to + mass_panel<MASS_KEYS>(row, 2 * chunk + !swap)) = swap ? lo : hi;
        }
        fence_async_shared();
        mbar_arrive(&ctl->k_full[st]);
        return true;
    };
    bool ok = true;
    for (; ok && c.at < c.end; next_item(c, p.w, p.c)) {
        count.at(p, c);
        const int t0 = mass_first(c), t1 = mass_last(c);
        if (count.rows == 0 || t0 == t1) continue;
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        const char *from = p.c.k.base + c.h * p.c.k.head_stride + chunk * 16;
        auto lookup = [&](int tile) {  // page id of this lane's row of a tile; -1: no such row
            const int j = tile * MASS_KEYS + 32 * w + lane;
            return tile < t1 && j < c.s.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
        };
        for (int r0 = 0; ok && r0 < count.rows; r0 += S::ROWS) {
            int tile = t0 + ((n ^ turn) & 1);  // this group's next
            int pg = lookup(tile), next = lookup(tile + 2);
            for (; ok && tile < t1; tile += 2, ++mine_n) {
                const int all = 2 * mine_n + turn, j0 = tile * MASS_KEYS;
                int64_t mine = -1;
                if (static_cast<unsigned>(pg) < static_cast<unsigned>(p.c.num_pages))
                    mine = pg * p.c.k.page_stride + ((j0 + 32 * w + lane) & mask) * p.c.k.slot_stride;
                pg = next;
                next = lookup(tile + 4);
                uint32_t to;
                if (S::WIDEN) {
                    if (mine_n >= RST) {
                        cp_async_wait<RST - 1>();
                        if (!(ok = widen(mine_n - RST))) break;
                    }
                    to = base + S::RAW_AT + (turn * RST + mine_n % RST) * S::RAW;
                } else {
                    const int st = all % KST;
                    if (all >= KST && !(ok = mass_wait(ctl, &ctl->k_empty[st], (all / KST - 1) & 1))) break;
                    to = base + S::K_AT + st * S::TILE;
                }
#pragma unroll 8
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int row = 32 * w + i * RPI + sub;
                    const int64_t at = __shfl_sync(0xffffffffu, mine, i * RPI + sub);
                    cp_async16_zfill(to + (S::WIDEN ? row * D + chunk * 16 : mass_panel<MASS_KEYS>(row, chunk)),
                                     at < 0 ? p.c.k.base : from + at, at < 0 ? 0 : 16);
                }
                if (S::WIDEN)
                    cp_async_commit();
                else
                    cp_async_arrive(&ctl->k_full[all % KST]);
            }
            n += t1 - t0;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (S::WIDEN)
        for (int t = mine_n >= RST ? mine_n - RST : 0; ok && t < mine_n; ++t) ok = widen(t);
}

// Three warps, an item ahead of the others: the counted rows of q and their
// constants.  For an e4m3 cache each row by a power of two into f16's range.
template <typename T, typename C, int D, typename Ctl>
__device__ void mass_prepare(const MassParams &p, Cursor c, char *smem, Ctl *ctl, int lt)
{
    using S = MassShape<C, D>;
    using M = typename MmaOf<T, C>::type;
    constexpr int CH = D / 8, STEP = 96 / CH, AHEAD = 6;  // rows at a time, loads of a thread on their way together
    Counted count;
    int unit_no = 0, item = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        count.at(p, c);
        if (count.rows == 0 || mass_first(c) == mass_last(c)) continue;
        if (item++ == p.give_up.item && static_cast<int>(blockIdx.x) == p.give_up.block) {  // the self-test
            *reinterpret_cast<volatile int *>(&ctl->dead) = 1;
            return;
        }
        const float unit = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        for (int r0 = 0; r0 < count.rows; r0 += S::ROWS, ++unit_no) {
            const int place = unit_no & 1, live = min(S::ROWS, count.rows - r0), padded = (live + 15) & ~15;
            char *qs = smem + S::Q_AT + place * S::Q;
            if (unit_no >= 2 && !mass_wait(ctl, &ctl->q_empty[place], ((unit_no >> 1) - 1) & 1)) return;
            const int ch = lt % CH;
#pragma unroll 1
            for (int b0 = 0; b0 < padded; b0 += AHEAD * STEP) {
                uint4 in[AHEAD];
                float z[AHEAD];
                int token[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int r = b0 + i * STEP + lt / CH;
                    in[i] = make_uint4(0, 0, 0, 0);
                    z[i] = CUDART_INF_F;
                    token[i] = -1;
                    if (r < live) {
                        const int nth = (r0 + r) / p.group, g = r0 + r - nth * p.group;
                        unsigned long long m = count.tokens;
                        for (int e = 0; e < nth; ++e) m &= m - 1;
                        token[i] = __ffsll(m) - 1;
                        const int64_t at = (static_cast<int64_t>(c.b) * p.w.T + token[i]) * p.q_heads + c.h * p.group + g;
                        in[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + at * D + ch * 8);
                        if (ch == 0) z[i] = __ldg(p.lse + at);
                    }
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int r = b0 + i * STEP + lt / CH;
                    uint4 raw = in[i];
                    float down = 1.0f;
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
                        down = exp2f(static_cast<float>(-e2));
                        raw = make_uint4(pack_mma<M>(x[0] * up, x[1] * up), pack_mma<M>(x[2] * up, x[3] * up),
                                         pack_mma<M>(x[4] * up, x[5] * up), pack_mma<M>(x[6] * up, x[7] * up));
                    }
                    if (r < padded) {
                        *reinterpret_cast<uint4 *>(qs + mass_panel<S::ROWS>(r, ch)) = raw;
                        if (ch == 0) {
                            unsigned long long see = 0;
                            if (token[i] >= 0) {
                                see = visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, token[i]);
                                if (z[i] == -CUDART_INF_F) see = 0;
                                if (see == 0) *reinterpret_cast<volatile int *>(&ctl->careful[place]) = unit_no + 1;
                            }
                            ctl->row[place][r] = make_float2(unit * down, z[i] * LOG2E);
                            ctl->sees[place][r] = see;
                        }
                    }
                }
            }
            fence_async_shared();
            mbar_arrive(&ctl->q_full[place]);
        }
    }
}

// One thread.
template <typename T, typename C, int D, typename Ctl>
__device__ void mass_multiply(const MassParams &p, Cursor c, char *smem, Ctl *ctl)
{
    using S = MassShape<C, D>;
    using M = typename MmaOf<T, C>::type;
    constexpr int KST = S::K_STAGES;
    const uint32_t base = smem_u32(smem), tmem = ctl->tmem;
    Counted count;
    int n = 0, unit_no = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        count.at(p, c);
        const int tiles = mass_last(c) - mass_first(c);
        if (count.rows == 0 || tiles == 0) continue;
        for (int r0 = 0; r0 < count.rows; r0 += S::ROWS, ++unit_no) {
            const int place = unit_no & 1, padded = (min(S::ROWS, count.rows - r0) + 15) & ~15;
            const uint32_t shape = mma_shape(std::is_same<M, __nv_bfloat16>::value, false, padded);
            if (!mass_wait1(ctl, &ctl->q_full[place], (unit_no >> 1) & 1)) return;
            for (int i = 0; i < tiles; ++i, ++n) {
                if (n >= MASS_BUFFERS && !mass_wait1(ctl, &ctl->s_empty[n % MASS_BUFFERS], (n / MASS_BUFFERS - 1) & 1)) return;
                if (!mass_wait1(ctl, &ctl->k_full[n % KST], (n / KST) & 1)) return;
                tc_fence_after();
                fence_async_shared();  // K was written by asynchronous copies of threads, q by threads
                const uint32_t k = base + S::K_AT + (n % KST) * S::TILE, q = base + S::Q_AT + place * S::Q;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma(tmem + (n % MASS_BUFFERS) * 128, desc_k_major(k + (ks >> 2) * (MASS_KEYS * 128) + (ks & 3) * 32),
                           desc_k_major(q + (ks >> 2) * (S::ROWS * 128) + (ks & 3) * 32), shape, ks > 0);
                tc_commit(&ctl->s_full[n % MASS_BUFFERS]);
                tc_commit(&ctl->k_empty[n % KST]);
            }
            tc_commit(&ctl->q_empty[place]);
        }
    }
}

// Four warps, a key of the tile a thread.  Returns the tile up to which the
// range is done: where its item began, if a wait gave up.  A warp that leaves so
// arrives on no barrier any more: 32 arrivals where a barrier lacks fewer (q's
// lacks 129) end in a fault.
template <typename Shape, typename Ctl> __device__ long long mass_sum(const MassParams &p, Cursor c, Ctl *ctl, int tid)
{
    constexpr int ROWS = Shape::ROWS;
    const int lane = tid & 31, warp = tid >> 5;
    const uint32_t quarter = ctl->tmem + (static_cast<uint32_t>(warp * 32) << 16);
    Counted count;
    int n = 0, unit_no = 0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        count.at(p, c);
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        const int t0 = mass_first(c), t1 = mass_last(c);
        if (count.bad) continue;
        const int64_t out_row = (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.stride;
        auto page_for = [&](int tile) {  // -1: nothing is written
            const int j = tile * MASS_KEYS + tid;
            return tile < t1 && j < c.s.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
        };
        for (int r0 = 0; r0 == 0 || r0 < count.rows; r0 += ROWS) {
            // what this thread's key has so far, to be multiplied by `keep` (where it is used: here it would wait)
            const float *so_far = r0 > 0 ? p.mass_out + out_row : p.mass_in ? p.mass_in + out_row : nullptr;
            const int held = so_far == nullptr ? 0 : r0 > 0 ? c.s.total : c.s.ctx;
            const float keep = r0 > 0 ? 1.0f : p.decay;
            auto mass_for = [&](int tile) {
                const int j = tile * MASS_KEYS + tid;
                return tile < t1 && j < held ? so_far[j] : 0.0f;
            };
            int pg = page_for(t0);  // both asked for a tile ahead
            float had = mass_for(t0);
            const int live = min(ROWS, count.rows - r0), place = unit_no & 1;
            bool careful = false;
            if (live > 0 && t0 < t1) {
                if (!mass_wait(ctl, &ctl->q_full[place], (unit_no >> 1) & 1)) return c.at;
                careful = *reinterpret_cast<volatile int *>(&ctl->careful[place]) == unit_no + 1;
            }
            for (int tile = t0; tile < t1; ++tile) {
                const int j = tile * MASS_KEYS + tid, page = pg;
                const float old = had;
                pg = page_for(tile + 1);
                had = mass_for(tile + 1);
                float sum = 0.0f;
                if (live > 0) {
                    if (!mass_wait(ctl, &ctl->s_full[n % MASS_BUFFERS], (n / MASS_BUFFERS) & 1)) return c.at;
                    tc_fence_after();
                    __syncwarp();
                    float s0 = 0.0f, s1 = 0.0f;
                    const bool masks = careful || (tile + 1) * MASS_KEYS > c.s.ctx;
                    for (int g = 0; g < live; g += 16) {
                        uint32_t y[16];
                        tc_ld16(y, quarter + (n % MASS_BUFFERS) * 128 + g);
                        const float4 *k = reinterpret_cast<const float4 *>(&ctl->row[place][g]);
                        if (!masks) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 u = k[i];
                                const float a = fast_exp2(__uint_as_float(y[2 * i]) * u.x - u.y);
                                const float b = fast_exp2(__uint_as_float(y[2 * i + 1]) * u.z - u.w);
                                if (g + 2 * i < live) s0 += a;
                                if (g + 2 * i + 1 < live) s1 += b;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int r = min(g + i, live - 1);
                                const unsigned long long see = ctl->sees[place][r];
                                const float2 u = ctl->row[place][r];
                                const bool seen = g + i < live && see != 0 &&
                                                  (j < c.s.ctx || (j < c.s.total && (see >> ((j - c.s.ctx) & 63) & 1)));
                                const float w = fast_exp2(__uint_as_float(y[i]) * u.x - u.y);
                                if (seen) s0 += w;
                            }
                        }
                        __syncwarp();
                    }
                    tc_fence_before();
                    mbar_arrive(&ctl->s_empty[n % MASS_BUFFERS]);
                    ++n;
                    sum = s0 + s1;
                }
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages)) p.mass_out[out_row + j] = old * keep + sum;
            }
            if (live > 0 && t0 < t1) {
                mbar_arrive(&ctl->q_empty[place]);
                ++unit_no;
            }
        }
    }
    return c.at;
}

// The items from tile `done` on, after a wait gave up: NaN where rows count, what
// does not depend on them as ever.  No barrier is touched any more.
__device__ __noinline__ void mass_lost(const MassParams &p, long long done, int tid)
{
    Counted count;
    for (Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid & 31); c.at < c.end; next_item(c, p.w, p.c)) {
        if (c.at < done) continue;
        count.at(p, c);
        if (count.bad) continue;
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        const int64_t out_row = (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.stride;
        const int end = min(mass_last(c) * MASS_KEYS, c.s.total);
        for (int j = mass_first(c) * MASS_KEYS + tid; j < end; j += MASS_KEYS) {
            if (page_of(p.c, table, j) < 0) continue;
            const float old = p.mass_in && j < c.s.ctx ? p.mass_in[out_row + j] : 0.0f;
            p.mass_out[out_row + j] = count.rows > 0 ? CUDART_NAN_F : old * p.decay;
        }
        if (count.rows > 0 && mass_first(c) < mass_last(c) && (tid & 31) == 0 && p.row_status) p.row_status[c.b] = STATUS_TIMEOUT;
    }
}

template <typename T, typename C, int D> __global__ void __launch_bounds__(MASS_THREADS, 1) mass_kernel(const MassParams p)
{
    using S = MassShape<C, D>;
    using Ctl = MassCtl<S::ROWS>;
    extern __shared__ char raw_smem[];
    char *smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::CTL_AT);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&ctl->k_full[i], 128);
            mbar_init(&ctl->k_empty[i], 1);
        }
        for (int i = 0; i < MASS_BUFFERS; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->s_empty[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->q_full[i], 96);
            mbar_init(&ctl->q_empty[i], 129);  // the products' end and the 128 readers of the constants
        }
        mbar_init(&ctl->spare, 1);
        ctl->dead = ctl->careful[0] = ctl->careful[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) tmem_alloc(&ctl->tmem, 512);
    chain_begin();
    const Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid & 31);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c.at == c.end) {  // the whole block
        if (warp == 4) tmem_free(ctl->tmem, 512);
        return;
    }
    if (warp < 4) {
        const long long done = mass_sum<S>(p, c, ctl, tid);
        if (done < c.end) mass_lost(p, done, tid);
    } else if (warp == 4) {
        if (tid == 128) {
            mass_multiply<T, C, D>(p, c, smem, ctl);
            // what was issued ends before the block may: others may have given up on it
            tc_commit(&ctl->spare);
            mbar_drain(&ctl->spare, 0);
        }
        __syncwarp();
    } else if (warp < 8) {
        mass_prepare<T, C, D>(p, c, smem, ctl, tid - 160);
    } else {
        mass_load<C, D>(p, c, smem, ctl, tid & 127, warp >= 12);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_free(ctl->tmem, 512);
}

template <typename T, typename C, int D> static cudaError_t launch_dim(const MassParams &p, cudaStream_t st)
{
    using S = MassShape<C, D>;
    auto kernel = mass_kernel<T, C, D>;
    constexpr int SMEM = S::CTL_AT + static_cast<int>(sizeof(MassCtl<S::ROWS>)) + 1024;
    static_assert(SMEM <= 232448, "shared memory of a block");
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    return launch_chained(kernel, dim3(MASS_SMS), MASS_THREADS, SMEM, st, p);
}
template <typename T, typename C> static cudaError_t launch_types(const MassParams &p, int D, cudaStream_t st)
{
    if (D == 64) return launch_dim<T, C, 64>(p, st);
    if (D == 128) return launch_dim<T, C, 128>(p, st);
    return launch_dim<T, C, 256>(p, st);
}

cudaError_t launch_mass(const MassLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    MassParams p{};
    p.c = paged_view(k);
    p.group = k.q_heads / k.cache.kv_heads;
    p.w = Work{k.B, k.T, 1, MASS_KEYS, k.ctx_lens, k.new_lens, true};
    p.q = L.q;
    p.lse = L.lse;
    p.mass_in = L.mass_in;
    p.parent = k.parent;
    p.accept = L.accept_count;
    p.nodes = L.nodes;
    p.mass_out = L.mass_out;
    p.stride = L.mass_stride;
    p.row_status = k.row_status;
    p.q_heads = k.q_heads;
    p.scale_log2 = k.scale * LOG2E;
    p.decay = L.decay;
    p.give_up = give_up();
    if (p.row_status) {
        const cudaError_t e = launch_chained(mass_status_kernel, dim3(k.B), 128, 0, st, p);
        if (e != cudaSuccess) return e;
    }
    const bool eight = k.cache.dtype == SPV_E4M3;
    const int D = k.cache.head_dim;
    if (k.dtype == SPV_BF16)
        return eight ? launch_types<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                     : launch_types<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_types<__half, __nv_fp8_e4m3>(p, D, st) : launch_types<__half, __half>(p, D, st);
}

}  // namespace spv
