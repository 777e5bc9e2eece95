// spv_evict.cu -- cuts each sequence's cache back to its budget by the
// accumulated attention weight, each key head by itself and in place.
//
// Selection, one block per (sequence, head): every slot gets an
// order-preserving 32-bit key (protected slots the largest) and the key of the
// last slot to stay is found digit by digit; bit masks of the kept slots and
// prefix counts over their words then match the i-th hole below the budget
// with the i-th kept slot above it.  Up to 16,384 slots the keys stay in
// registers (evict_select_few), up to 49,152 in shared memory, and are counted,
// two bits a round, until a count is exact, usually after about 12 rounds;
// beyond, a radix select reads the weights again for each of four digits
// (evict_select_many).
// evict_move_kernel, a dependent launch, copies the rows of the matched slots
// and writes the new lengths: all blocks of the selection have read the old ones
// by then, so the new may take their place.
//
// What bounds it: for many sequences the moves, read once and written once (32
// sequences of 8,191 slots, 8 heads of 128, bf16, cut to 4,096: 633 MB, 117 us,
// 5.4 TB/s, 80% of a copy's rate); for few the
// chain of the selection's rounds, each two barriers (4 sequences of 2,117 slots
// cut to 2,048: 14.6 us).
#include "spv_kv.cuh"

namespace spv {

constexpr int EV_THREADS = 1024;
constexpr int EV_MOVE_SLOTS = 256;     // slots that a block of the move looks at, one a thread
constexpr int EV_MOVE_AHEAD = 8;       // 16-byte pieces of a thread on their way
constexpr int EV_HELD_SLOTS = 49152;   // whose keys fit shared memory
constexpr int EV_FEW_SLOTS = 16384, EV_FEW_THREADS = 512;  // two blocks an SM for up to 8,192 slots

struct EvictParams {
    PagedView c;
    const int32_t *lens, *pos;
    const float *mass;
    float *mass_out;
    int32_t *pos_out, *new_lens, *slot_src, *row_status;
    int64_t stride, out_stride;
    int budget, sinks, recent, row_bytes, words;
    int piece_shift;  // log2 of the 16-byte pieces of a slot's K and V rows together; -1: no power of two
};

// Ascending order of the keys is ascending order of the weights: NaN lowest,
// -0 as 0; the largest key is kept for protected slots.
__device__ __forceinline__ unsigned mass_key(float x)
{
    if (x != x) return 0;
    const unsigned u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned slot_key(const EvictParams &p, const float *mass, const int32_t *pos, int j, long long top)
{
    const long long at = pos ? pos[j] : j;
    return at < p.sinks || at > top - p.recent ? 0xffffffffu : mass_key(mass[j]);
}

// Exclusive prefix of `x` over a block of WARPS warps; *all gets the sum.
template <int WARPS> __device__ __forceinline__ int block_prefix(int x, int *sh, int *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = upto;
    __syncthreads();
    // every warp by itself: the sums of all, and of those before it
    int s = lane < WARPS ? sh[lane] : 0;
    *all = __reduce_add_sync(0xffffffffu, s);
    s = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
    return upto - x + s;
}

// Whether a length is out of range.
__device__ __forceinline__ bool evict_bad(const EvictParams &p, int n)
{
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
    return n < 0 || n > cap || n > p.stride;
}

// What both selections begin with, for block (h, b): the length, whether it is
// bad, and the outputs that need no selection.  False: the item is done.
struct EvictItem {
    int b, h, n, m;  // slots in use, slots to keep
    const float *mass;
    const int32_t *pos;
    int32_t *src;
    float *mass_out;
    int32_t *pos_out;
};
__device__ __forceinline__ bool evict_begin(const EvictParams &p, EvictItem *it)
{
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const int64_t item = static_cast<int64_t>(b) * p.c.kv_heads + h;
    it->b = b;
    it->h = h;
    it->mass = p.mass + item * p.stride;
    it->pos = p.pos ? p.pos + item * p.stride : nullptr;
    it->src = p.slot_src + item * p.budget;
    it->mass_out = p.mass_out + item * p.out_stride;
    it->pos_out = p.pos_out ? p.pos_out + item * p.out_stride : nullptr;
    const int n = p.lens[b];
    const bool bad = evict_bad(p, n);
    if (h == 0 && p.row_status) {
        int any = bad;
        const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
        for (int g = tid; !bad && n > p.budget && g <= (n - 1) >> p.c.page_shift; g += static_cast<int>(blockDim.x))
            any |= page_of(p.c, table, g << p.c.page_shift) < 0;
        any = __syncthreads_or(any);
        if (tid == 0) p.row_status[b] = any ? KV_STATUS_BAD : 0;
    }
    it->n = n;
    it->m = bad ? 0 : n < p.budget ? n : p.budget;
    if (!bad && n > p.budget) return true;
    for (int i = tid; i < p.budget; i += static_cast<int>(blockDim.x)) {  // nothing moves
        it->src[i] = i < it->m ? i : -1;
        if (i < it->m) {
            it->mass_out[i] = it->mass[i];
            if (it->pos_out) it->pos_out[i] = it->pos ? it->pos[i] : i;
        }
    }
    return false;
}
__device__ __forceinline__ void evict_write(const EvictParams &p, const EvictItem &it, int i, int s)
{
    it.src[i] = s;
    if (s != i || p.mass_out != p.mass) it.mass_out[i] = it.mass[s];
    if (it.pos_out && (s != i || p.pos_out != p.pos)) it.pos_out[i] = it.pos ? it.pos[s] : s;
}

// The m largest keys: those from `least` on where that is exactly m (exact),
// else those above it and `want` of its equals.
struct EvictCut {
    unsigned least;
    int want;
    bool exact;
};
// `count(a, b, c, &x, &yz)` adds a thread's number of keys >= a to x, >= b and
// >= c to the low and high half of yz (each below 65,536 in the block).  Two bits
// a round; a round is two warp reductions on either side of one barrier.
template <int WARPS, typename Count> __device__ __forceinline__ EvictCut find_cut(int m, uint2 (*counts)[WARPS], Count &&count)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    EvictCut cut{0, 0, false};
    int turn = 0;
    auto count3 = [&](unsigned a, unsigned b, unsigned c, int *na, int *nb, int *nc) {
        unsigned x = 0, yz = 0;
        count(a, b, c, &x, &yz);
        x = __reduce_add_sync(0xffffffffu, x);
        yz = __reduce_add_sync(0xffffffffu, yz);
        if (lane == 0) counts[turn][warp] = make_uint2(yz, x);
        __syncthreads();
        const uint2 w = lane < WARPS ? counts[turn][lane] : make_uint2(0, 0);
        x = __reduce_add_sync(0xffffffffu, w.y);
        yz = __reduce_add_sync(0xffffffffu, w.x);
        *na = static_cast<int>(x);
        *nb = static_cast<int>(yz & 0xffffu);
        *nc = static_cast<int>(yz >> 16);
        turn ^= 1;  // who writes this turn's places again has passed the other's barrier
    };
    for (int bit = 30; bit >= 0 && !cut.exact; bit -= 2) {
        const unsigned a = cut.least | 1u << bit, b = cut.least | 2u << bit, c = cut.least | 3u << bit;
        int x, y, z;
        count3(a, b, c, &x, &y, &z);
        const int got = z >= m ? z : y >= m ? y : x >= m ? x : -1;
        cut.least = z >= m ? c : y >= m ? b : x >= m ? a : cut.least;
        cut.exact = got == m;
    }
    if (!cut.exact) {
        int x = 0, y, z;
        if (cut.least != 0xffffffffu) count3(cut.least + 1u, 0xffffffffu, 0xffffffffu, &x, &y, &z);
        cut.want = m - x;
    }
    return cut;
}

// Slots in registers: slot t + 512 i is thread t's i-th.
template <int PER> __global__ void __launch_bounds__(EV_FEW_THREADS) evict_select_few(const EvictParams p)
{
    constexpr int NT = EV_FEW_THREADS, WARPS = NT / 32, WORDS = PER * WARPS, WPT = (WORDS + NT - 1) / NT;
    static_assert(WORDS % NT == 0 || WPT == 1, "words of a thread");
    __shared__ unsigned kept[WORDS], before[WORDS];  // kept bits; equals, later holes before a word
    __shared__ unsigned short movers[WORDS * 16];            // kept slots at or above the budget, in order
    __shared__ int sh[32];
    __shared__ uint2 counts[2][WARPS];  // each warp's, in turn: at least b, c (16 bits each); at least a
    chain_begin();
    EvictItem it;
    if (!evict_begin(p, &it)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = it.n, m = it.m;
    unsigned key[PER];
    {
        float w[PER];
        int at[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = tid + i * NT;
            w[i] = j < n ? it.mass[j] : 0.0f;
            at[i] = j < n ? (it.pos ? it.pos[j] : j) : -1;
        }
        int top = -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = max(top, at[i]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) sh[warp] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, sh[lane % WARPS]);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = tid + i * NT;
            const bool always = at[i] < p.sinks || static_cast<long long>(at[i]) > static_cast<long long>(top) - p.recent;
            key[i] = j >= n ? 0u : always ? 0xffffffffu : mass_key(w[i]);
        }
    }
    const EvictCut cut = find_cut<WARPS>(m, counts, [&](unsigned a, unsigned b, unsigned c, unsigned *x, unsigned *yz) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            *x += key[i] >= a;
            *yz += (key[i] >= b ? 1u : 0u) + (key[i] >= c ? 0x10000u : 0u);
        }
    });
    const unsigned least = cut.least;
    const bool exact = cut.exact;
    const int want = cut.want;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = tid + i * NT;
        const unsigned gt = __ballot_sync(0xffffffffu, j < n && (exact ? key[i] >= least : key[i] > least));
        const unsigned eq = __ballot_sync(0xffffffffu, j < n && !exact && key[i] == least);
        if (lane == 0) {
            kept[i * WARPS + warp] = gt;
            before[i * WARPS + warp] = eq;
        }
    }
    __syncthreads();
    int all;
    if (!exact) {
        const int w0 = tid * WPT;  // this thread's words
        int mine = 0;
#pragma unroll
        for (int i = 0; i < WPT; ++i) mine += w0 + i < WORDS ? __popc(before[w0 + i]) : 0;
        int left = want - block_prefix<WARPS>(mine, sh, &all);
#pragma unroll
        for (int i = 0; i < WPT; ++i) {
            if (w0 + i >= WORDS) break;
            unsigned eq = before[w0 + i], k = kept[w0 + i];
            for (; eq; eq &= eq - 1)
                if (left-- > 0) k |= eq & -eq;
            kept[w0 + i] = k;
        }
        __syncthreads();
    }
    const int wm = m >> 5;
    const unsigned low = (1u << (m & 31)) - 1u;
    {
        const int w0 = tid * WPT;
        unsigned hole[WPT], mover[WPT];
        int packed = 0;
#pragma unroll
        for (int i = 0; i < WPT; ++i) {
            const int w = w0 + i;
            const unsigned k = w < WORDS ? kept[w] : 0;
            const unsigned below = w < wm ? 0xffffffffu : w == wm ? low : 0u;  // slots below the budget
            hole[i] = w < WORDS ? ~k & below : 0u;
            mover[i] = k & ~below;
            packed += __popc(hole[i]) | __popc(mover[i]) << 16;
        }
        int ahead = block_prefix<WARPS>(packed, sh, &all);
#pragma unroll
        for (int i = 0; i < WPT; ++i) {
            const int w = w0 + i;
            if (w < WORDS) before[w] = ahead & 0xffff;
            int at = ahead >> 16;
            for (unsigned left = mover[i]; left; left &= left - 1) movers[at++] = static_cast<unsigned short>(32 * w + __ffs(left) - 1);
            ahead += __popc(hole[i]) | __popc(mover[i]) << 16;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.budget; i += NT) {
        int s = i;
        if (i < m) {
            const unsigned k = kept[i >> 5], bit = 1u << (i & 31);
            if (!(k & bit)) s = movers[before[i >> 5] + __popc(~k & (bit - 1u))];
            evict_write(p, it, i, s);
        } else {
            it.src[i] = -1;
        }
    }
}

// HELD: the keys fit shared memory and are counted there; else the weights are
// read again for each digit of a radix select.
template <bool HELD> __global__ void __launch_bounds__(EV_THREADS) evict_select_many(const EvictParams p)
{
    extern __shared__ unsigned words[];  // kept bits, prefix counts; HELD: the keys
    __shared__ uint2 counts[2][EV_THREADS / 32];
    __shared__ unsigned hist[256];
    __shared__ int sh[32];
    __shared__ int tops[32];
    __shared__ unsigned found[2];
    chain_begin();
    EvictItem it;
    if (!evict_begin(p, &it)) return;
    const int tid = threadIdx.x, lane = tid & 31, n = it.n, m = it.m;
    const float *mass = it.mass;
    const int32_t *pos = it.pos;
    int top = pos ? -1 : n - 1;
    if (pos) {
        for (int j = tid; j < n; j += EV_THREADS) top = max(top, pos[j]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[tid >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, tops[lane]);
    }
    unsigned *keys = words + 2 * p.words;  // each thread's own: slots tid + 1024 i
    auto key_of = [&](int j) { return HELD ? keys[j] : slot_key(p, mass, pos, j, top); };
    // the key of the m-th largest; `want` of its equals stay
    unsigned prefix = 0;
    int want = m;
    if constexpr (HELD) {
#pragma unroll 8
        for (int j = tid; j < n; j += EV_THREADS) keys[j] = slot_key(p, mass, pos, j, top);
        const EvictCut cut = find_cut<EV_THREADS / 32>(m, counts, [&](unsigned a, unsigned b, unsigned c, unsigned *x, unsigned *yz) {
#pragma unroll 8
            for (int j = tid; j < n; j += EV_THREADS) {
                const unsigned k = keys[j];
                *x += k >= a;
                *yz += (k >= b ? 1u : 0u) + (k >= c ? 0x10000u : 0u);
            }
        });
        // exactly: all above the key before the least one
        prefix = cut.exact ? cut.least - 1u : cut.least;
        want = cut.exact ? 0 : cut.want;
    } else {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = tid; j < n; j += EV_THREADS) {
                const unsigned key = slot_key(p, mass, pos, j, top);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[key >> shift & 255u], 1u);
            }
            __syncthreads();
            const int x = tid < 256 ? static_cast<int>(hist[255 - tid]) : 0;
            int all;
            const int before = block_prefix<EV_THREADS / 32>(x, sh, &all);  // of larger digits
            if (tid < 256 && before < want && want <= before + x) {
                found[0] = 255 - tid;
                found[1] = want - before;
            }
            __syncthreads();
            prefix |= found[0] << shift;
            want = static_cast<int>(found[1]);
            __syncthreads();
        }
    }
    // kept bits: larger keys, and the first `want` equals
    const int nw = (n + 31) >> 5;
    unsigned *kept = words, *count = words + p.words;
    for (int w = tid >> 5; w < nw; w += EV_THREADS / 32) {
        const int j = 32 * w + lane;
        const unsigned key = j < n ? key_of(j) : 0;
        const unsigned gt = __ballot_sync(0xffffffffu, j < n && key > prefix);
        const unsigned eq = __ballot_sync(0xffffffffu, j < n && key == prefix);
        if (lane == 0) {
            kept[w] = gt;
            count[w] = eq;
        }
    }
    __syncthreads();
    int run = 0;
    for (int w0 = 0; w0 < nw; w0 += EV_THREADS) {
        const int w = w0 + tid;
        unsigned eq = w < nw ? count[w] : 0;
        int all;
        const int before = run + block_prefix<EV_THREADS / 32>(__popc(eq), sh, &all);
        if (w < nw) {
            for (int left = want - before; eq && left > 0; --left) {
                kept[w] |= eq & -eq;
                eq &= eq - 1;
            }
        }
        run += all;
    }
    __syncthreads();
    // prefix counts: holes in the words below m, movers in those above
    const int wm = m >> 5;
    const unsigned low = (1u << (m & 31)) - 1u;
    int holes = 0, movers = 0;
    for (int w0 = 0; w0 < nw; w0 += EV_THREADS) {
        const int w = w0 + tid;
        const unsigned k = w < nw ? kept[w] : 0;
        const int hole = w >= nw || w > wm ? 0 : w < wm ? __popc(~k) : __popc(~k & low);
        const int mover = w >= nw || w < wm ? 0 : w > wm ? __popc(k) : __popc(k & ~low);
        int all;
        const int hb = holes + block_prefix<EV_THREADS / 32>(hole, sh, &all);
        holes += all;
        const int mb = movers + block_prefix<EV_THREADS / 32>(mover, sh, &all);
        movers += all;
        if (w < nw) count[w] = w <= wm ? hb : mb;
    }
    __syncthreads();
    const int first_movers = wm < nw ? __popc(kept[wm] & ~low) : 0;
    for (int i = tid; i < m; i += EV_THREADS) {
        const unsigned k = kept[i >> 5], bit = 1u << (i & 31);
        int s = i;
        if (!(k & bit)) {
            int rank = static_cast<int>(count[i >> 5]) + __popc(~k & (bit - 1u));
            unsigned from;
            int w;
            if (rank < first_movers) {
                w = wm;
                from = kept[wm] & ~low;
            } else {
                int a = wm + 1, z = nw - 1;  // the last word whose count is <= rank
                while (a < z) {
                    const int mid = (a + z + 1) >> 1;
                    if (static_cast<int>(count[mid]) <= rank)
                        a = mid;
                    else
                        z = mid - 1;
                }
                w = a;
                from = kept[w];
                rank -= static_cast<int>(count[w]);
            }
            for (; rank > 0; --rank) from &= from - 1;
            s = 32 * w + __ffs(from) - 1;
        }
        evict_write(p, it, i, s);
    }
    for (int i = m + tid; i < p.budget; i += EV_THREADS) it.src[i] = -1;
}

__global__ void __launch_bounds__(EV_MOVE_SLOTS) evict_move_kernel(const EvictParams p)
{
    __shared__ int64_t from_k[EV_MOVE_SLOTS], to_k[EV_MOVE_SLOTS], from_v[EV_MOVE_SLOTS], to_v[EV_MOVE_SLOTS];
    __shared__ int per_warp[EV_MOVE_SLOTS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y % p.c.kv_heads, b = blockIdx.y / p.c.kv_heads, i = blockIdx.x * EV_MOVE_SLOTS + tid;
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    chain_begin();
    if (tid == 0 && blockIdx.x == 0 && h == 0) {
        const int n = p.lens[b];  // may be new_lens
        p.new_lens[b] = evict_bad(p, n) || n < p.budget ? n : p.budget;
    }
    // the block's moves, in a row
    const int s = i < p.budget ? p.slot_src[static_cast<int64_t>(blockIdx.y) * p.budget + i] : -1;
    bool moves = s >= 0 && s != i;
    int from = -1, to = -1;
    if (moves) {
        from = page_of(p.c, table, s);
        to = page_of(p.c, table, i);
        moves = from >= 0 && to >= 0;
    }
    const unsigned who = __ballot_sync(0xffffffffu, moves);
    if (lane == 0) per_warp[warp] = __popc(who);
    __syncthreads();
    int at = __popc(who & ((1u << lane) - 1u)), count = 0;
#pragma unroll
    for (int w = 0; w < EV_MOVE_SLOTS / 32; ++w) {
        if (w < warp) at += per_warp[w];
        count += per_warp[w];
    }
    if (moves) {
        from_k[at] = row_ptr(p.c, p.c.k, from, s, h) - p.c.k.base;
        to_k[at] = row_ptr(p.c, p.c.k, to, i, h) - p.c.k.base;
        from_v[at] = row_ptr(p.c, p.c.v, from, s, h) - p.c.v.base;
        to_v[at] = row_ptr(p.c, p.c.v, to, i, h) - p.c.v.base;
    }
    __syncthreads();
    const int per = p.row_bytes >> 4, pieces = 2 * per, all = count * pieces;  // 16-byte pieces of a row; K's, then V's
    for (int x0 = tid; x0 < all; x0 += EV_MOVE_AHEAD * EV_MOVE_SLOTS) {
        uint4 data[EV_MOVE_AHEAD];
        char *dst[EV_MOVE_AHEAD];
#pragma unroll
        for (int e = 0; e < EV_MOVE_AHEAD; ++e) {
            const int x = x0 + e * EV_MOVE_SLOTS;
            dst[e] = nullptr;
            if (x < all) {
                const int r = p.piece_shift >= 0 ? x >> p.piece_shift : x / pieces;
                int o = x - r * pieces;
                const bool v = o >= per;
                o = (v ? o - per : o) << 4;
                char *base = v ? p.c.v.base : p.c.k.base;
                data[e] = __ldcs(reinterpret_cast<const uint4 *>(base + (v ? from_v[r] : from_k[r]) + o));
                dst[e] = base + (v ? to_v[r] : to_k[r]) + o;
            }
        }
#pragma unroll
        for (int e = 0; e < EV_MOVE_AHEAD; ++e)
            if (dst[e]) *reinterpret_cast<uint4 *>(dst[e]) = data[e];
    }
}

cudaError_t launch_evict(const EvictLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    EvictParams p{};
    p.c = paged_view(k);
    p.lens = L.lens;
    p.pos = L.pos;
    p.mass = L.mass;
    p.mass_out = L.mass_out;
    p.pos_out = L.pos_out;
    p.new_lens = L.new_lens;
    p.slot_src = L.slot_src;
    p.row_status = k.row_status;
    p.stride = L.mass_stride;
    p.out_stride = L.out_stride;
    p.budget = L.budget;
    p.sinks = L.sinks;
    p.recent = L.recent;
    p.row_bytes = k.cache.head_dim * (k.cache.dtype == SPV_E4M3 ? 1 : 2);
    const int64_t cap = static_cast<int64_t>(k.max_pages) * k.cache.page_size;
    p.words = static_cast<int>(((cap < L.mass_stride ? cap : L.mass_stride) + 31) / 32);
    const int pieces = p.row_bytes / 8;
    p.piece_shift = (pieces & (pieces - 1)) == 0 ? log2_of(pieces) : -1;
    const dim3 items(k.cache.kv_heads, k.B);
    // Where the keys are kept.  Registers, as few as will do: 2,117 slots 14.6 us with 8 a thread, 25.7 with 32, 15.8 in
    // shared memory; 8,191 slots 117 us with 16, 131 with 32, 128 in shared memory; 16,001 slots 65 us with 32, 102 in
    // shared memory.  Then shared memory: 30,001 slots 151 us, read again from the cache for each digit 176.
    const int slots = p.words * 32;  // that a sequence can have
    cudaError_t e;
    if (slots <= 4096) {
        e = launch_chained(evict_select_few<8>, items, EV_FEW_THREADS, 0, st, p);
    } else if (slots <= 8192) {
        e = launch_chained(evict_select_few<16>, items, EV_FEW_THREADS, 0, st, p);
    } else if (slots <= EV_FEW_SLOTS) {
        e = launch_chained(evict_select_few<32>, items, EV_FEW_THREADS, 0, st, p);
    } else {
        const bool held = slots <= EV_HELD_SLOTS;
        const int smem = (p.words * 2 + (held ? slots : 0)) * static_cast<int>(sizeof(unsigned));
        auto kernel = held ? evict_select_many<true> : evict_select_many<false>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        e = launch_chained(kernel, items, EV_THREADS, smem, st, p);
    }
    if (e != cudaSuccess) return e;
    const dim3 moves((L.budget + EV_MOVE_SLOTS - 1) / EV_MOVE_SLOTS, k.B * k.cache.kv_heads);
    return launch_chained(evict_move_kernel, moves, EV_MOVE_SLOTS, 0, st, p);
}

}  // namespace spv
