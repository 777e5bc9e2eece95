// spv_norm_rope.cu -- norms of q and k for each head, their rotation by the
// positions of one or more axes, and the write of k and v into the paged cache,
// in one pass.
//
// Mathematics: y = w x / sqrt(mean(x^2) + eps) over a head's D elements, then
// the pairs of y turn by position[axis of the pair] times the pair's frequency.
// The angle is the integer product of the position with a 64-bit fraction of a
// turn, so its wrap is the reduction to one turn.  Everything between the load
// and the store is held in 32 bits.
//
// What bounds it is reading q, k, v and writing q, K, V once.  A block takes one
// token, or four of a sequence where there are enough to fill the GPU, and
// computes their cosines and sines once for all heads.  The heads of q, k and v
// of these tokens are one row of work: groups of lanes take a head each, a lane
// 8 elements and, of halves, their partners, so that the sum of squares is a few
// shuffles and the rotation needs no exchange; a head is asked for while the one
// before it is worked on.
#include "spv_kv.cuh"

namespace spv {

struct NormRopeParams {
    const void *q, *k, *v;
    void *q_out;
    int64_t stride[6];
    PagedView c;
    const float *q_weight, *k_weight;
    float eps;
    const unsigned long long *freqs;
    const int32_t *axes, *positions, *ctx_lens, *new_lens;
    int32_t *slot_pos, *row_status;
    int64_t pos_stride;
    int num_axes, B, T, q_heads, D, half;  // half = rotary_dim / 2
    float mscale;
};

constexpr int NORM_THREADS = 256;
constexpr int NORM_TOKENS = 4;  // of a block, where there are many

enum NormMode {
    NORM_PAIRS,   // interleaved, or nothing turns: a lane has 8 elements
    NORM_HALVES,  // a lane has 8 elements and their partners half a rotation away, or 8 that pass
    NORM_ODD      // halves whose length is no multiple of 8: the head passes through shared memory
};

// Lanes of a head's group that have work.
template <int MODE> __host__ __device__ inline int norm_tasks(int D, int half)
{
    return MODE == NORM_HALVES ? (half >> 3) + ((D - 2 * half) >> 3) : D >> 3;
}

template <typename T> __device__ __forceinline__ void widen8(float *y, const uint4 &raw)
{
    const T *x = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = Num<T>::up(x[i]);
}
// x times unit and the eight weights from w on.
__device__ __forceinline__ void weigh8(float *x, const float *w, float unit)
{
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(w + i);
        x[i] *= unit * a.x, x[i + 1] *= unit * a.y, x[i + 2] *= unit * a.z, x[i + 3] *= unit * a.w;
    }
}
// (u, z) turned by the angle whose cosine and sine are (c, s).
__device__ __forceinline__ void turn(float &u, float &z, float c, float s)
{
    const float x = u;
    u = x * c - z * s;
    z = z * c + x * s;
}
template <typename C> struct alignas(8 * sizeof(C)) Eight {
    C x[8];
};
template <typename C> __device__ __forceinline__ void narrow8(C *to, const float *y, float div)
{
    Eight<C> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.x[i] = Num<C>::down(sizeof(C) == 1 ? y[i] / div : y[i]);
    *reinterpret_cast<Eight<C> *>(to) = o;
}

template <int MODE, int TOKENS, typename T, typename C>
__global__ void __launch_bounds__(NORM_THREADS) norm_rope_kernel(const NormRopeParams p, const int width)
{
    extern __shared__ __align__(16) float shared[];
    __shared__ int pages[TOKENS];  // of the tokens; -1: not written
    const int D = p.D, half = p.half;
    float2 *cs = reinterpret_cast<float2 *>(shared);             // [token][pair], padded to 16 bytes
    const int cs_row = (half + 1) & ~1;
    float *weights = shared + 2 * TOKENS * cs_row;               // [q, k][D]
    float *odd = weights + 2 * D;                                // NORM_ODD: a head of each group
    const int tid = threadIdx.x, blocks = (p.T + TOKENS - 1) / TOKENS, b = blockIdx.x / blocks;
    const int t0 = (blockIdx.x - b * blocks) * TOKENS, tokens = min(TOKENS, p.T - t0);
    const int n0 = b * p.T + t0, kv_heads = p.c.kv_heads, heads = p.q_heads + 2 * kv_heads;
    const T *q0 = static_cast<const T *>(p.q) + b * p.stride[0] + t0 * p.stride[1];
    const T *k0 = static_cast<const T *>(p.k) + b * p.stride[2] + t0 * p.stride[3];
    const T *v0 = static_cast<const T *>(p.v) + b * p.stride[4] + t0 * p.stride[5];
    // this lane's place in its group and in a head: 8 elements from d on, and their partners from `other` on
    const int lane = tid & (width - 1), group = tid / width, groups = NORM_THREADS / width;
    const bool works = lane < norm_tasks<MODE>(D, half);
    const bool turns = MODE == NORM_HALVES ? lane < half >> 3 : 8 * lane < 2 * half;
    const int d = MODE == NORM_HALVES && !turns ? 8 * lane + half : 8 * lane, other = d + half;
    struct Data {
        uint4 x, y;
    };
    struct Where {
        int token, head;
    };
    // a group's heads are `groups` apart in the row of work
    const int step = TOKENS == 1 ? 0 : groups / heads, step_heads = groups - step * heads;
    auto after = [&](Where w) {
        w.token += step;
        w.head += step_heads;
        if (TOKENS > 1 && w.head >= heads) ++w.token, w.head -= heads;
        return w;
    };
    // v has no partners: its lanes take 8 elements at 8 lane, and where a group has fewer lanes than that, 8 more behind
    auto v_at = [&](int i) { return 8 * (lane + i * width); };
    auto fetch = [&](Where w, Data &to) {
        if (w.token >= tokens || w.head >= heads) return;
        if (w.head >= p.q_heads + kv_heads) {
            const T *row = v0 + w.token * p.stride[5] + (w.head - p.q_heads - kv_heads) * D;
            if (v_at(0) < D) to.x = *reinterpret_cast<const uint4 *>(row + v_at(0));
            if (v_at(1) < D) to.y = *reinterpret_cast<const uint4 *>(row + v_at(1));
            return;
        }
        const T *row = w.head < p.q_heads ? q0 + w.token * p.stride[1] + w.head * D
                                          : k0 + w.token * p.stride[3] + (w.head - p.q_heads) * D;
        if (works) to.x = *reinterpret_cast<const uint4 *>(row + d);
        if (MODE == NORM_HALVES && works && turns) to.y = *reinterpret_cast<const uint4 *>(row + other);
    };
    Data now{}, next{};
    chain_begin();
    Where w{TOKENS == 1 ? 0 : group / heads, 0};
    w.head = group - w.token * heads;
    fetch(w, now);
    const SeqLens s = seq_lens(p.ctx_lens, p.new_lens, b, p.T, p.c);
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    if (t0 == 0 && p.row_status) {  // all pages that the sequence's new tokens touch
        int bad = s.bad;
        if (s.total > 0)
            for (int g = (s.ctx >> p.c.page_shift) + tid; g <= (s.total - 1) >> p.c.page_shift; g += NORM_THREADS)
                bad |= page_of(p.c, table, g << p.c.page_shift) < 0;
        bad = __syncthreads_or(bad);
        if (tid == 0) p.row_status[b] = bad ? KV_STATUS_BAD : 0;
    }
    const int live = s.bad ? 0 : max(0, min(tokens, s.fresh - t0));
    auto position = [&](int tk, int axis) {
        return p.positions ? __ldg(p.positions + static_cast<int64_t>(n0 + tk) * p.num_axes + axis) : s.ctx + t0 + tk;
    };
    for (int i = tid; i < live * half; i += NORM_THREADS) {
        const int tk = TOKENS == 1 ? 0 : i / half, e = i - tk * half;
        const int axis = p.axes ? min(max(__ldg(p.axes + e), 0), p.num_axes - 1) : 0;
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(position(tk, axis))) * __ldg(p.freqs + e);
        // the top 32 bits, signed: half a turn either way, at most 2^-33 turns off
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>((turn + (1ull << 31)) >> 32)) * 0x1p-31f, &sn, &cn);
        cs[tk * cs_row + e] = make_float2(cn * p.mscale, sn * p.mscale);
    }
    for (int i = tid; i < 2 * D; i += NORM_THREADS) {
        const float *w = i < D ? p.q_weight : p.k_weight;
        weights[i] = w ? __ldg(w + (i < D ? i : i - D)) : 1.0f;
    }
    if (tid < live) pages[tid] = page_of(p.c, table, s.ctx + t0 + tid);
    if (p.slot_pos)
        for (int i = tid; i < live * kv_heads; i += NORM_THREADS) {
            const int tk = i / kv_heads, h = i - tk * kv_heads, slot = s.ctx + t0 + tk;
            if (slot < p.pos_stride) p.slot_pos[(static_cast<int64_t>(b) * kv_heads + h) * p.pos_stride + slot] = position(tk, 0);
        }
    __syncthreads();
    T *q_out = static_cast<T *>(p.q_out) + static_cast<int64_t>(n0) * p.q_heads * D;
    for (int i = live * p.q_heads * (D >> 3) + tid; i < tokens * p.q_heads * (D >> 3); i += NORM_THREADS)
        reinterpret_cast<uint4 *>(q_out)[i] = uint4{};
    const int todo = live * heads;
    const int rounds = (todo + groups - 1) / groups;  // of every group: shuffles need whole warps
    for (int round = 0; round < rounds; ++round) {
        const Where then = after(w);
        fetch(then, next);
        const bool here = round * groups + group < todo;
        if (!here) w = Where{0, 0};
        const bool is_q = w.head < p.q_heads, is_v = w.head >= p.q_heads + kv_heads;
        const int h = is_q ? w.head : is_v ? w.head - p.q_heads - kv_heads : w.head - p.q_heads;  // in its tensor
        const bool pair = MODE == NORM_HALVES && turns;
        float x[8], y[8];
        widen8<T>(x, now.x);
        widen8<T>(y, now.y);
        float sum = 0.0f;
        if (works) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += x[e] * x[e];
            if (pair) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += y[e] * y[e];
            }
        }
        for (int o = width >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!is_v) {
            if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
                const float unit = 1.0f / sqrtf(sum / static_cast<float>(D) + p.eps);
                const float *wt = weights + (is_q ? 0 : D);
                if (works) {
                    weigh8(x, wt + d, unit);
                    if (pair) weigh8(y, wt + other, unit);
                }
            }
            const float2 *mine = cs + w.token * cs_row;
            if (pair) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 a = *reinterpret_cast<const float4 *>(mine + d + e);
                    turn(x[e], y[e], a.x, a.y);
                    turn(x[e + 1], y[e + 1], a.z, a.w);
                }
            } else if (MODE == NORM_PAIRS && turns) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    if (d + e >= 2 * half) continue;
                    const float4 a = *reinterpret_cast<const float4 *>(mine + ((d + e) >> 1));
                    turn(x[e], x[e + 1], a.x, a.y);
                    if (d + e + 2 < 2 * half) turn(x[e + 2], x[e + 3], a.z, a.w);
                }
            }
        }
        if (MODE == NORM_ODD) {  // a lane's partners are in other lanes, at other places of their 8
            float *head = odd + group * D;
            if (works)
#pragma unroll
                for (int e = 0; e < 8; ++e) head[d + e] = x[e];
            __syncwarp();
            if (works && !is_v) {
                const float2 *mine = cs + w.token * cs_row;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = d + e;
                    if (at >= 2 * half) continue;
                    const float2 a = mine[at < half ? at : at - half];
                    x[e] = at < half ? x[e] * a.x - head[at + half] * a.y : x[e] * a.x + head[at - half] * a.y;
                }
            }
            __syncwarp();
        }
        if (here) {
            if (is_q) {
                T *row = q_out + (static_cast<int64_t>(w.token) * p.q_heads + h) * D;
                if (works) narrow8(row + d, x, 1.0f);
                if (works && pair) narrow8(row + other, y, 1.0f);
            } else {
                const int slot = s.ctx + t0 + w.token, page = pages[w.token];
                if (page >= 0) {
                    const PoolView &pool = is_v ? p.c.v : p.c.k;
                    C *row = reinterpret_cast<C *>(const_cast<char *>(row_ptr(p.c, pool, page, slot, h)));
                    const float *scale = is_v ? p.c.v_scale : p.c.k_scale;
                    const float div = sizeof(C) == 1 && scale ? __ldg(scale + h) : 1.0f;
                    if (is_v) {
                        if constexpr (std::is_same<T, C>::value) {
                            if (v_at(0) < D) *reinterpret_cast<uint4 *>(row + v_at(0)) = now.x;
                            if (v_at(1) < D) *reinterpret_cast<uint4 *>(row + v_at(1)) = now.y;
                        } else {
                            if (v_at(0) < D) narrow8(row + v_at(0), x, div);
                            if (v_at(1) < D) narrow8(row + v_at(1), y, div);
                        }
                    } else {
                        if (works) narrow8(row + d, x, div);
                        if (works && pair) narrow8(row + other, y, div);
                    }
                }
            }
        }
        now = next;
        w = then;
    }
}

template <int MODE, typename T, typename C> static cudaError_t launch_mode(const NormRopeParams &p, cudaStream_t st)
{
    int width = 1;
    while (width < norm_tasks<MODE>(p.D, p.half)) width *= 2;
    const int pairs = (p.half + 1) & ~1, odd = MODE == NORM_ODD ? NORM_THREADS / width * p.D : 0;
    auto bytes = [&](int tokens) { return (2 * tokens * pairs + 2 * p.D + odd) * static_cast<int>(sizeof(float)); };
    // four tokens a block once that still gives every SM eight blocks
    if (static_cast<int64_t>(p.B) * p.T >= 8 * 152 * NORM_TOKENS)
        return launch_chained(norm_rope_kernel<MODE, NORM_TOKENS, T, C>, dim3(p.B * ((p.T + NORM_TOKENS - 1) / NORM_TOKENS)),
                              NORM_THREADS, bytes(NORM_TOKENS), st, p, width);
    return launch_chained(norm_rope_kernel<MODE, 1, T, C>, dim3(p.B * p.T), NORM_THREADS, bytes(1), st, p, width);
}
template <typename T, typename C> static cudaError_t launch(const NormRopeParams &p, bool interleaved, cudaStream_t st)
{
    if (interleaved || p.half == 0) return launch_mode<NORM_PAIRS, T, C>(p, st);
    if (p.half % 8 == 0) return launch_mode<NORM_HALVES, T, C>(p, st);
    return launch_mode<NORM_ODD, T, C>(p, st);
}

cudaError_t launch_norm_rope(const NormRopeLaunch &L, cudaStream_t st)
{
    const RopeLaunch &r = L.rope;
    NormRopeParams p{};
    p.q = r.q;
    p.k = r.k;
    p.v = r.v;
    p.q_out = r.q_out;
    for (int i = 0; i < 6; ++i) p.stride[i] = r.strides[i];
    p.c = paged_view(r.kv);
    p.q_weight = L.q_weight;
    p.k_weight = L.k_weight;
    p.eps = L.eps;
    p.freqs = reinterpret_cast<const unsigned long long *>(r.freqs);
    p.axes = L.axes;
    p.positions = r.positions;
    p.ctx_lens = r.kv.ctx_lens;
    p.new_lens = r.kv.new_lens;
    p.slot_pos = r.slot_pos;
    p.row_status = r.kv.row_status;
    p.pos_stride = r.pos_stride;
    p.num_axes = L.num_axes;
    p.B = r.kv.B;
    p.T = r.kv.T;
    p.q_heads = r.kv.q_heads;
    p.D = r.kv.cache.head_dim;
    p.half = r.rotary_dim / 2;
    p.mscale = r.mscale;
    const bool eight = r.kv.cache.dtype == SPV_E4M3;
    if (r.kv.dtype == SPV_BF16)
        return eight ? launch<__nv_bfloat16, __nv_fp8_e4m3>(p, r.interleaved, st) : launch<__nv_bfloat16, __nv_bfloat16>(p, r.interleaved, st);
    return eight ? launch<__half, __nv_fp8_e4m3>(p, r.interleaved, st) : launch<__half, __half>(p, r.interleaved, st);
}

}  // namespace spv
