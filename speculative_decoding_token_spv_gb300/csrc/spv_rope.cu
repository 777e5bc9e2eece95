// spv_rope.cu -- rotary positions of new tokens' q and k, joined with the
// write of k and v into the paged cache.
//
// A block takes one token, or four of a sequence in turn where there are
// enough to fill the GPU: its threads first compute the tokens' cosines and
// sines into shared memory, once for all heads.  A thread then keeps its place
// within a head -- 8 elements, 16 bytes, and their cosines and sines in
// registers -- and walks over the heads.  The angle is the integer product of
// the position with a 64-bit fraction of a turn: the wrap of the product is the
// reduction to one turn, exact at any position, with no 64-bit floating point.
//
// What bounds it is reading q, k, v and writing q, K, V once.  8 prompts of up
// to 2,011 tokens, 32 + 8 heads of 128, f16, 395 MB: 64.6 us, 6.1 TB/s, 90% of a
// copy's rate (the next token's elements are asked for while one is worked on;
// without that 88 us).  One token of one sequence: 2.8 us, of which the angle's
// sine, the page lookup and two trips to memory are a chain.
#include "spv_kv.cuh"

namespace spv {

struct RopeParams {
    const void *q, *k, *v;
    void *q_out;
    int64_t stride[6];
    PagedView c;
    const unsigned long long *freqs;
    const int32_t *positions, *ctx_lens, *new_lens;
    int32_t *slot_pos, *row_status;
    int64_t pos_stride;
    int B, T, q_heads, D, half, interleaved;  // half = rotary_dim / 2
    float mscale;
};

// 8 elements of T.
template <typename T> struct alignas(8 * sizeof(T)) Vec8 {
    T x[8];
};

template <typename T> __device__ __forceinline__ void load8(const T *src, float *y)
{
    const Vec8<T> a = *reinterpret_cast<const Vec8<T> *>(src);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = Num<T>::up(a.x[i]);
}
template <typename C> __device__ __forceinline__ void store8(C *dst, const float *y, float div)
{
    Vec8<C> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.x[i] = Num<C>::down(sizeof(C) == 1 ? y[i] / div : y[i]);
    *reinterpret_cast<Vec8<C> *>(dst) = o;
}

// How a head's elements are cut into tasks, so that each task reads all it
// needs before it writes (q may be rotated in place).
enum RopeMode {
    ROPE_PAIRS,   // interleaved, or nothing rotates: a task is 8 elements
    ROPE_PARTIAL, // the same where the rotation ends within a task's 8: what is behind its end keeps its bits
    ROPE_HALVES,  // a task is 8 elements and their partners half a rotation away; then 8 passing elements each
    ROPE_SCALAR   // halves whose length is no multiple of 8: the same, element by element
};
constexpr bool rope_pairs(int mode) { return mode == ROPE_PAIRS || mode == ROPE_PARTIAL; }
template <int MODE> __device__ __forceinline__ int head_tasks(const RopeParams &p)
{
    if (rope_pairs(MODE)) return p.D >> 3;
    return (p.half >> 3) + ((p.D - 2 * p.half) >> 3);
}

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TOKENS = 4;  // of a block, where there are many

// A thread's place within each head that it visits, and what turns it there.
template <int MODE> struct RopePlace {
    int d, other;            // its 8 elements begin here, their partners there (-1: none)
    float c[8], s[8];        // interleaved: of the 4 pairs, each twice
    bool turns;
    int n;                   // ROPE_PARTIAL: elements that turn, the first ones
};

template <int MODE, typename T> struct RopeData {
    uint4 x, y;
};
template <int MODE, typename T>
__device__ __forceinline__ void rope_read(RopeData<MODE, T> &v, const T *row, const RopePlace<MODE> &at)
{
    v.x = *reinterpret_cast<const uint4 *>(row + at.d);
    if (MODE == ROPE_HALVES && at.other >= 0) v.y = *reinterpret_cast<const uint4 *>(row + at.other);
}
template <int MODE, typename T, typename C>
__device__ __forceinline__ void rope_write(const RopeData<MODE, T> &v, C *row, const RopePlace<MODE> &at, float div)
{
    if constexpr (std::is_same<T, C>::value) {
        if (!at.turns) {
            *reinterpret_cast<uint4 *>(row + at.d) = v.x;
            return;
        }
    }
    const T *xs = reinterpret_cast<const T *>(&v.x);
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = Num<T>::up(xs[j]);
    if (MODE == ROPE_HALVES && at.other >= 0) {
        const T *ys = reinterpret_cast<const T *>(&v.y);
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u0 = u[j], w0 = Num<T>::up(ys[j]);
            u[j] = u0 * at.c[j] - w0 * at.s[j];
            w[j] = w0 * at.c[j] + u0 * at.s[j];
        }
        store8(row + at.other, w, div);
    }
    if (rope_pairs(MODE) && at.turns) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            if (MODE == ROPE_PARTIAL && j >= at.n) continue;
            const float u0 = u[j], w0 = u[j + 1];
            u[j] = u0 * at.c[j] - w0 * at.s[j];
            u[j + 1] = w0 * at.c[j] + u0 * at.s[j];
        }
    }
    if constexpr (MODE == ROPE_PARTIAL && std::is_same<T, C>::value) {
        Vec8<C> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.x[j] = j < at.n ? Num<C>::down(u[j]) : xs[j];
        *reinterpret_cast<Vec8<C> *>(row + at.d) = o;
        return;
    }
    store8(row + at.d, u, div);
}

constexpr int ROPE_AHEAD = 3;   // heads of a thread whose elements are asked for a token ahead

template <int MODE, int TOKENS, typename T, typename C>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams p)
{
    extern __shared__ float2 cs[];  // [token][pair]
    const int tid = threadIdx.x, blocks = (p.T + TOKENS - 1) / TOKENS, b = blockIdx.x / blocks;
    const int t0 = (blockIdx.x - b * blocks) * TOKENS, tokens = min(TOKENS, p.T - t0);
    const int n0 = b * p.T + t0, D8 = p.D >> 3, heads = p.q_heads + p.c.kv_heads;
    const T *q0 = static_cast<const T *>(p.q) + b * p.stride[0] + t0 * p.stride[1];
    const T *k0 = static_cast<const T *>(p.k) + b * p.stride[2] + t0 * p.stride[3];
    const T *v0 = static_cast<const T *>(p.v) + b * p.stride[4] + t0 * p.stride[5];
    // this thread's place in the heads that turn, and in v's, which pass
    RopePlace<MODE> at;
    RopePlace<ROPE_PAIRS> v_place;
    const int per = MODE == ROPE_SCALAR ? 1 : head_tasks<MODE>(p), step = ROPE_THREADS / per, h0 = tid / per < step ? tid / per : heads, e = tid % per;
    const int v_step = ROPE_THREADS / D8, v_h0 = tid / D8 < v_step ? tid / D8 : p.c.kv_heads;
    at.d = 8 * e;
    at.other = -1;
    at.turns = false;
    if (MODE == ROPE_HALVES) {
        at.turns = e < p.half >> 3;
        if (at.turns)
            at.other = at.d + p.half;
        else
            at.d += p.half;  // past both halves
    } else if (rope_pairs(MODE)) {
        at.turns = at.d < 2 * p.half;
        at.n = min(8, 2 * p.half - at.d);
    }
    v_place.d = 8 * (tid % D8);
    v_place.other = -1;
    v_place.turns = false;
    auto from = [&](int tk, int h) {
        return h < p.q_heads ? q0 + tk * p.stride[1] + h * p.D : k0 + tk * p.stride[3] + (h - p.q_heads) * p.D;
    };
    // The first heads of a token are asked for while the one before is worked on, and those of the first token before
    // lengths, pages and angles, a chain of loads of their own.
    RopeData<MODE, T> x[ROPE_AHEAD], x_next[ROPE_AHEAD];
    RopeData<ROPE_PAIRS, T> v, v_next;
    auto fetch = [&](int tk, RopeData<MODE, T> (&to)[ROPE_AHEAD], RopeData<ROPE_PAIRS, T> &to_v) {
        if (MODE == ROPE_SCALAR) return;
#pragma unroll
        for (int i = 0; i < ROPE_AHEAD; ++i)
            if (h0 + i * step < heads) rope_read(to[i], from(tk, h0 + i * step), at);
        if (v_h0 < p.c.kv_heads) rope_read(to_v, v0 + tk * p.stride[5] + v_h0 * p.D, v_place);
    };
    chain_begin();
    fetch(0, x, v);
    const SeqLens s = seq_lens(p.ctx_lens, p.new_lens, b, p.T, p.c);
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    if (t0 == 0 && p.row_status) {  // all pages that the sequence's new tokens touch
        int bad = s.bad;
        if (s.total > 0)
            for (int g = (s.ctx >> p.c.page_shift) + tid; g <= (s.total - 1) >> p.c.page_shift; g += ROPE_THREADS)
                bad |= page_of(p.c, table, g << p.c.page_shift) < 0;
        bad = __syncthreads_or(bad);
        if (tid == 0) p.row_status[b] = bad ? KV_STATUS_BAD : 0;
    }
    const int live = s.bad ? 0 : max(0, min(tokens, s.fresh - t0));
    for (int i = tid; i < live * p.half; i += ROPE_THREADS) {
        const int tk = TOKENS == 1 ? 0 : i / p.half, e = i - tk * p.half;
        const int pos = p.positions ? __ldg(p.positions + n0 + tk) : s.ctx + t0 + tk;
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * __ldg(p.freqs + e);
        // the top 32 bits, signed: half a turn either way, at most 2^-33 turns off
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>((turn + (1ull << 31)) >> 32)) * 0x1p-31f, &sn, &cn);
        cs[i] = make_float2(cn * p.mscale, sn * p.mscale);
    }
    if (p.slot_pos)
        for (int i = tid; i < live * p.c.kv_heads; i += ROPE_THREADS) {
            const int tk = i / p.c.kv_heads, h = i - tk * p.c.kv_heads, slot = s.ctx + t0 + tk;
            if (slot < p.pos_stride)
                p.slot_pos[(static_cast<int64_t>(b) * p.c.kv_heads + h) * p.pos_stride + slot] =
                    p.positions ? __ldg(p.positions + n0 + tk) : slot;
        }
    __syncthreads();
    for (int tk = 0; tk < tokens; ++tk) {
        if (TOKENS > 1 && tk + 1 < live) fetch(tk + 1, x_next, v_next);
        T *q_out = static_cast<T *>(p.q_out) + static_cast<int64_t>(n0 + tk) * p.q_heads * p.D;
        if (tk >= live) {
            for (int i = tid; i < p.q_heads * D8; i += ROPE_THREADS) reinterpret_cast<uint4 *>(q_out)[i] = uint4{};
            continue;
        }
        const int slot = s.ctx + t0 + tk, page = page_of(p.c, table, slot);
        char *k_row = const_cast<char *>(row_ptr(p.c, p.c.k, page < 0 ? 0 : page, slot, 0));
        char *v_row = const_cast<char *>(row_ptr(p.c, p.c.v, page < 0 ? 0 : page, slot, 0));
        const float2 *mine = cs + tk * p.half;
        auto k_at = [&](int h) { return reinterpret_cast<C *>(k_row + (h - p.q_heads) * p.c.k.head_stride); };
        auto k_div = [&](int h) { return sizeof(C) == 1 && p.c.k_scale ? __ldg(p.c.k_scale + h - p.q_heads) : 1.0f; };
        if constexpr (MODE == ROPE_SCALAR) {
            // halves whose length is no multiple of 8: element by element, partners by one thread
            const int each = p.half + p.D - 2 * p.half;
            for (int i = tid; i < heads * each; i += ROPE_THREADS) {
                const int h = i / each, e = i - h * each;
                const T *row = from(tk, h);
                const int d = e < p.half ? e : e + p.half, o = e < p.half ? e + p.half : -1;
                float u = Num<T>::up(row[d]), w = 0.0f;
                if (o >= 0) {
                    const float2 a = mine[e];
                    const float u0 = u, w0 = Num<T>::up(row[o]);
                    u = u0 * a.x - w0 * a.y;
                    w = w0 * a.x + u0 * a.y;
                }
                if (h < p.q_heads) {
                    q_out[h * p.D + d] = o >= 0 ? Num<T>::down(u) : row[d];  // what passes keeps its bits
                    if (o >= 0) q_out[h * p.D + o] = Num<T>::down(w);
                } else if (page >= 0) {
                    const float div = k_div(h);
                    if constexpr (std::is_same<T, C>::value)
                        k_at(h)[d] = o >= 0 ? Num<C>::down(u) : row[d];
                    else
                        k_at(h)[d] = Num<C>::down(u / div);
                    if (o >= 0) k_at(h)[o] = Num<C>::down(sizeof(C) == 1 ? w / div : w);
                }
            }
        } else {
            if (MODE == ROPE_HALVES && at.turns) {
#pragma unroll
                for (int j = 0; j < 8; ++j) at.c[j] = mine[at.d + j].x, at.s[j] = mine[at.d + j].y;
            }
            if (rope_pairs(MODE) && at.turns) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    if (MODE == ROPE_PARTIAL && j >= at.n) continue;
                    const float2 a = mine[(at.d + j) >> 1];
                    at.c[j] = a.x, at.s[j] = a.y;
                }
            }
            auto write = [&](int h, const RopeData<MODE, T> &data) {
                if (h < p.q_heads)
                    rope_write<MODE, T, T>(data, q_out + h * p.D, at, 1.0f);
                else if (page >= 0)
                    rope_write<MODE, T, C>(data, k_at(h), at, k_div(h));
            };
#pragma unroll
            for (int i = 0; i < ROPE_AHEAD; ++i)
                if (h0 + i * step < heads) write(h0 + i * step, x[i]);
            for (int h = h0 + ROPE_AHEAD * step; h < heads; h += step) {
                rope_read(x[0], from(tk, h), at);
                write(h, x[0]);
            }
        }
        if (page >= 0) {
            for (int h = v_h0; h < p.c.kv_heads; h += v_step) {
                if (MODE == ROPE_SCALAR || h != v_h0) rope_read(v, v0 + tk * p.stride[5] + h * p.D, v_place);
                rope_write<ROPE_PAIRS, T, C>(v, reinterpret_cast<C *>(v_row + h * p.c.v.head_stride), v_place,
                                             sizeof(C) == 1 && p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.0f);
            }
        }
        if (TOKENS > 1) {
#pragma unroll
            for (int i = 0; i < ROPE_AHEAD; ++i) x[i] = x_next[i];
            v = v_next;
        }
    }
}

template <int MODE, typename T, typename C> static cudaError_t launch_mode(const RopeParams &p, cudaStream_t st)
{
    // four tokens a block once that still gives every SM eight blocks: 8 prompts of up to 2,011 tokens take 64.6 us, with
    // one token a block 70.2; fewer tokens are spread over as many SMs as there are: the verify tokens of 64 sequences
    // take 5.5 us, with four a block 9.8
    const int smem = p.half * static_cast<int>(sizeof(float2));
    if (static_cast<int64_t>(p.B) * p.T >= 8 * 152 * ROPE_TOKENS)
        return launch_chained(rope_kernel<MODE, ROPE_TOKENS, T, C>, dim3(p.B * ((p.T + ROPE_TOKENS - 1) / ROPE_TOKENS)),
                              ROPE_THREADS, ROPE_TOKENS * smem, st, p);
    return launch_chained(rope_kernel<MODE, 1, T, C>, dim3(p.B * p.T), ROPE_THREADS, smem, st, p);
}
template <typename T, typename C> static cudaError_t launch(const RopeParams &p, cudaStream_t st)
{
    if (p.interleaved && p.half % 4 != 0) return launch_mode<ROPE_PARTIAL, T, C>(p, st);
    if (p.interleaved || p.half == 0) return launch_mode<ROPE_PAIRS, T, C>(p, st);
    if (p.half % 8 == 0) return launch_mode<ROPE_HALVES, T, C>(p, st);
    return launch_mode<ROPE_SCALAR, T, C>(p, st);
}

PagedView paged_view(const KvLaunch &L)
{
    const spv_kv_cache &c = L.cache;
    const int64_t e = c.dtype == SPV_E4M3 ? 1 : 2;
    PagedView v{};
    v.k = PoolView{static_cast<char *>(c.k), c.k_page_stride * e, c.k_slot_stride * e, c.k_head_stride * e};
    v.v = PoolView{static_cast<char *>(c.v), c.v_page_stride * e, c.v_slot_stride * e, c.v_head_stride * e};
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.table = L.page_table;
    v.max_pages = L.max_pages;
    v.num_pages = c.num_pages;
    v.page_shift = log2_of(c.page_size);
    v.kv_heads = c.kv_heads;
    return v;
}

cudaError_t launch_rope(const RopeLaunch &L, cudaStream_t st)
{
    RopeParams p{};
    p.q = L.q;
    p.k = L.k;
    p.v = L.v;
    p.q_out = L.q_out;
    for (int i = 0; i < 6; ++i) p.stride[i] = L.strides[i];
    p.c = paged_view(L.kv);
    p.freqs = reinterpret_cast<const unsigned long long *>(L.freqs);
    p.positions = L.positions;
    p.ctx_lens = L.kv.ctx_lens;
    p.new_lens = L.kv.new_lens;
    p.slot_pos = L.slot_pos;
    p.row_status = L.kv.row_status;
    p.pos_stride = L.pos_stride;
    p.B = L.kv.B;
    p.T = L.kv.T;
    p.q_heads = L.kv.q_heads;
    p.D = L.kv.cache.head_dim;
    p.half = L.rotary_dim / 2;
    p.interleaved = L.interleaved;
    p.mscale = L.mscale;
    const bool eight = L.kv.cache.dtype == SPV_E4M3;
    if (L.kv.dtype == SPV_BF16)
        return eight ? launch<__nv_bfloat16, __nv_fp8_e4m3>(p, st) : launch<__nv_bfloat16, __nv_bfloat16>(p, st);
    return eight ? launch<__half, __nv_fp8_e4m3>(p, st) : launch<__half, __half>(p, st);
}

}  // namespace spv
