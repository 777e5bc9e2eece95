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
// token, or four or eight of a sequence where there are enough to fill the GPU,
// and computes their cosines and sines once for all heads.  Groups of lanes take
// every so many heads of one token each, a lane 8 elements and, of halves, their
// partners, so that the sum of squares is a few shuffles, the rotation needs no
// exchange, and a lane's cosines, sines and weights stay in its registers from
// head to head; a head is asked for while the one before it is worked on.
// Arithmetic is in pairs.  Measured (32 heads on 8 of 128, 16 bits): 16,088
// tokens 88 us, 4.5 TB/s, 74 us where a quarter of them is padding; 4,800 tokens
// 30 us, 2,400 (in L2) 15 us; one token 6.3 us.  Instructions and their waits are
// half of it: with no arithmetic 62 us are left of 77.  Rows by way of shared
// memory, all at once (77 us) or an item ahead in blocks that stay (102 us), two
// heads asked for ahead (76 us), positions and pages before the lengths are used
// (77 us), one token a block (158 us) and more blocks of fewer registers (78 us)
// were no faster.
#include "spv_mma.cuh"

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

// Floats of a token's cosines and sines, a multiple of four.
__host__ __device__ inline int norm_angles(int half) { return 2 * ((half + 1) & ~1); }

template <typename T> __device__ __forceinline__ void widen8(float *y, const uint4 &raw)
{
    const T *x = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = Num<T>::up(x[i]);
}
// Four pairs of floats, on each of which one instruction works.
__device__ __forceinline__ void pairs_of(unsigned long long (&y)[4], const float *x)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack2(x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void floats_of(float *x, const unsigned long long (&y)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(y[i], x[2 * i], x[2 * i + 1]);
}
// Eight floats of shared memory, 16 bytes at a time.
__device__ __forceinline__ void pairs_at(unsigned long long (&y)[4], const float *at)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 a = reinterpret_cast<const float4 *>(at)[i];
        y[2 * i] = pack2(a.x, a.y);
        y[2 * i + 1] = pack2(a.z, a.w);
    }
}
__device__ __forceinline__ unsigned long long add_squares(const float *x, unsigned long long sum)
{
    unsigned long long y[4];
    pairs_of(y, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = ffma2(y[i], y[i], sum);
    return sum;
}
// x times unit and eight weights.
__device__ __forceinline__ void weigh8(float *x, const unsigned long long (&w)[4], float unit)
{
    unsigned long long y[4];
    pairs_of(y, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(w[i], pack2(unit, unit)));
    floats_of(x, y);
}
// Eight (u, z) turned by the angles whose cosines and sines are (c, s).
__device__ __forceinline__ void turn8(float *u, float *z, const unsigned long long (&c)[4], const unsigned long long (&s)[4])
{
    unsigned long long a[4], b[4];
    pairs_of(a, u);
    pairs_of(b, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned long long x = a[i];
        a[i] = ffma2(mul2(b[i], s[i]), pack2(-1.0f, -1.0f), mul2(x, c[i]));
        b[i] = ffma2(x, s[i], mul2(b[i], c[i]));
    }
    floats_of(u, a);
    floats_of(z, b);
}
template <typename C> __device__ __forceinline__ void narrow8(C *to, const float *y, float div)
{
    if constexpr (sizeof(C) == 1) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] / div, y[2 * i + 1] / div), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2 *>(to) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    } else {
        *reinterpret_cast<uint4 *>(to) = make_uint4(pack_mma<C>(y[0], y[1]), pack_mma<C>(y[2], y[3]), pack_mma<C>(y[4], y[5]), pack_mma<C>(y[6], y[7]));
    }
}

template <int MODE, int TOKENS, typename T, typename C>
__global__ void __launch_bounds__(NORM_THREADS, 2) norm_rope_kernel(const NormRopeParams p, const int width)
{
    extern __shared__ __align__(16) float shared[];
    __shared__ int64_t rows[2][TOKENS];  // bytes from a head's first slot to the token's, of K and V; -1: not written
    const int D = p.D, half = p.half, kv_heads = p.c.kv_heads;
    const int tid = threadIdx.x, blocks = (p.T + TOKENS - 1) / TOKENS, b = blockIdx.x / blocks;
    const int t0 = (blockIdx.x - b * blocks) * TOKENS, tokens = min(TOKENS, p.T - t0), n0 = b * p.T + t0;
    const int lane = tid & (width - 1), group = tid / width, groups = NORM_THREADS / width;
    float *cs = shared;                         // [token]: pairs (cosine, sine), of NORM_HALVES all cosines before the sines
    const int cs_row = norm_angles(half);
    float *weights = shared + TOKENS * cs_row;  // [q, k][D]
    float *odd = weights + 2 * D;               // NORM_ODD: a head of each group
    // this lane's place in a head: 8 elements from d on, and their partners from `other` on
    const bool works = lane < norm_tasks<MODE>(D, half);
    const bool turns = MODE == NORM_HALVES ? lane < half >> 3 : 8 * lane < 2 * half, pair = MODE == NORM_HALVES && turns;
    const int d = MODE == NORM_HALVES && !turns ? 8 * lane + half : 8 * lane, other = d + half;
    // a group has one token, and every so many heads of it
    const int token = group % TOKENS, my_first = group / TOKENS, apart = groups / TOKENS;
    struct Data {
        uint4 x, y;
    };
    auto row_of = [&](const void *x, int64_t of_b, int64_t of_t) { return static_cast<const T *>(x) + b * of_b + (t0 + token) * of_t + my_first * D; };
    auto get = [&](bool there, Data &to, const T *row) {
        if (there && works) to.x = *reinterpret_cast<const uint4 *>(row + d);
        if (there && pair) to.y = *reinterpret_cast<const uint4 *>(row + other);
    };
    // v has no partners: 8 elements at 8 lane, and where a group has fewer lanes than that, 8 more behind
    const int v0 = 8 * lane, v1 = 8 * (lane + width);
    auto get_v = [&](bool there, Data &to, const T *row) {
        if (there && v0 < D) to.x = *reinterpret_cast<const uint4 *>(row + v0);
        if (there && v1 < D) to.y = *reinterpret_cast<const uint4 *>(row + v1);
    };
    const T *q_row = row_of(p.q, p.stride[0], p.stride[1]), *k_row = row_of(p.k, p.stride[2], p.stride[3]), *v_row = row_of(p.v, p.stride[4], p.stride[5]);
    Data q_now{}, k_now{}, v_now{};
    chain_begin();
    get(token < tokens && my_first < p.q_heads, q_now, q_row);
    get(token < tokens && my_first < kv_heads, k_now, k_row);
    get_v(token < tokens && my_first < kv_heads, v_now, v_row);
    const SeqLens s = seq_lens(p.ctx_lens, p.new_lens, b, p.T, p.c);
    auto position = [&](int tk, int axis) {
        return p.positions ? __ldg(p.positions + static_cast<int64_t>(n0 + tk) * p.num_axes + axis) : s.ctx + t0 + tk;
    };
    const int live = s.bad ? 0 : max(0, min(tokens, s.fresh - t0));
    for (int i = tid; i < live * half; i += NORM_THREADS) {
        const int tk = TOKENS == 1 ? 0 : i / half, e = i - tk * half;
        const int axis = p.axes ? min(max(__ldg(p.axes + e), 0), p.num_axes - 1) : 0;
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(position(tk, axis))) * __ldg(p.freqs + e);
        // the top 32 bits, signed: half a turn either way, at most 2^-33 turns off
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>((turn + (1ull << 31)) >> 32)) * 0x1p-31f, &sn, &cn);
        cn *= p.mscale, sn *= p.mscale;
        float *at = cs + tk * cs_row;
        if (MODE == NORM_HALVES)
            at[e] = cn, at[half + e] = sn;
        else
            reinterpret_cast<float2 *>(at)[e] = make_float2(cn, sn);
    }
    for (int i = tid; i < 2 * D; i += NORM_THREADS) {
        const float *w = i < D ? p.q_weight : p.k_weight;
        weights[i] = w ? __ldg(w + (i < D ? i : i - D)) : 1.0f;
    }
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    if (t0 == 0 && p.row_status) {  // all pages that the sequence's new tokens touch
        int bad = s.bad;
        if (s.total > 0)
            for (int g = (s.ctx >> p.c.page_shift) + tid; g <= (s.total - 1) >> p.c.page_shift; g += NORM_THREADS)
                bad |= page_of(p.c, table, g << p.c.page_shift) < 0;
        bad = __syncthreads_or(bad);
        if (tid == 0) p.row_status[b] = bad ? KV_STATUS_BAD : 0;
    }
    if (tid < live) {
        const int slot = s.ctx + t0 + tid, page = page_of(p.c, table, slot), in_page = slot & ((1 << p.c.page_shift) - 1);
        rows[0][tid] = page < 0 ? -1 : page * p.c.k.page_stride + in_page * p.c.k.slot_stride;
        rows[1][tid] = page < 0 ? -1 : page * p.c.v.page_stride + in_page * p.c.v.slot_stride;
    }
    if (p.slot_pos)
        for (int i = tid; i < live * kv_heads; i += NORM_THREADS) {
            const int tk = i / kv_heads, h = i - tk * kv_heads, slot = s.ctx + t0 + tk;
            if (slot < p.pos_stride) p.slot_pos[(static_cast<int64_t>(b) * kv_heads + h) * p.pos_stride + slot] = position(tk, 0);
        }
    T *q_out = static_cast<T *>(p.q_out) + static_cast<int64_t>(n0) * p.q_heads * D;
    const int64_t token_q = static_cast<int64_t>(p.q_heads) * D;
    for (int64_t i = live * token_q + 8 * tid; i < tokens * token_q; i += 8 * NORM_THREADS) *reinterpret_cast<uint4 *>(q_out + i) = uint4{};
    __syncthreads();
    if (live == 0) return;
    const bool there = token < live;
    const float *angles = cs + token * cs_row;
    unsigned long long cosines[4], sines[4];  // NORM_PAIRS: `cosines` has both
    if (pair) {
        pairs_at(cosines, angles + d);
        pairs_at(sines, angles + half + d);
    } else if (MODE == NORM_PAIRS && turns) {
        pairs_at(cosines, angles + d);
    }
    const float by_d = 1.0f / static_cast<float>(D);
    // now: this group's first head, which is at `row`; to: where head 0 goes; apart_by: from head to head
    auto turn_heads = [&](bool there, int count, Data now, const T *row, const float *weight, const float *in_shared, auto *to, int64_t apart_by, const float *scale) {
        unsigned long long wx[4], wy[4];
        if (weight && works) {
            pairs_at(wx, in_shared + d);
            if (pair) pairs_at(wy, in_shared + other);
        }
#pragma unroll 1
        for (int at = my_first, round = 0; round < count; round += apart, at += apart) {  // whole warps: shuffles need them
            const bool here = there && at < count;
            Data next;
            row += apart * D;
            get(there && at + apart < count, next, row);
            float x[8], y[8];
            widen8<T>(x, now.x);
            widen8<T>(y, now.y);
            now = next;
            if (weight) {
                float sum = 0.0f;
                if (works) {
                    unsigned long long squares = add_squares(x, 0);
                    if (pair) squares = add_squares(y, squares);
                    float more;
                    unpack2(squares, sum, more);
                    sum += more;
                }
                for (int o = width >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float unit = rsqrtf(fmaf(sum, by_d, p.eps));
                if (works) weigh8(x, wx, unit);
                if (works && pair) weigh8(y, wy, unit);
            }
            if (pair) {
                turn8(x, y, cosines, sines);
            } else if (MODE == NORM_PAIRS && turns) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    if (d + e >= 2 * half) continue;
                    float c, sn;
                    unpack2(cosines[e >> 1], c, sn);
                    const float u = x[e], z = x[e + 1];
                    x[e] = u * c - z * sn;
                    x[e + 1] = z * c + u * sn;
                }
            }
            if (MODE == NORM_ODD) {  // a lane's partners are in other lanes, at other places of their 8
                float *head = odd + group * D;
                if (works)
#pragma unroll
                    for (int e = 0; e < 8; ++e) head[d + e] = x[e];
                __syncwarp();
                if (works)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = d + e;
                        if (i >= 2 * half) continue;
                        const float2 a = reinterpret_cast<const float2 *>(angles)[i < half ? i : i - half];
                        x[e] = i < half ? x[e] * a.x - head[i + half] * a.y : x[e] * a.x + head[i - half] * a.y;
                    }
                __syncwarp();
            }
            if (here && works) {
                const float div = sizeof(*to) == 1 && scale ? __ldg(scale + at) : 1.0f;
                narrow8(to + at * apart_by + d, x, div);
                if (pair) narrow8(to + at * apart_by + other, y, div);
            }
        }
    };
    turn_heads(there, p.q_heads, q_now, q_row, p.q_weight, weights, q_out + static_cast<int64_t>(token) * p.q_heads * D, D, nullptr);
    const int64_t k_at = there ? rows[0][token] : -1, v_at = there ? rows[1][token] : -1;
    auto head_0 = [&](const PoolView &pool, int64_t at) { return reinterpret_cast<C *>(const_cast<char *>(pool.base) + at); };
    const int64_t element = sizeof(C);
    turn_heads(k_at >= 0, kv_heads, k_now, k_row, p.k_weight, weights + D, head_0(p.c.k, k_at), p.c.k.head_stride / element, p.c.k_scale);
    if (v_at < 0) return;
    for (int at = my_first; at < kv_heads; at += apart) {
        C *to = head_0(p.c.v, v_at) + at * (p.c.v.head_stride / element);
        Data next;
        v_row += apart * D;
        get_v(at + apart < kv_heads, next, v_row);
        if constexpr (std::is_same<T, C>::value) {
            if (v0 < D) *reinterpret_cast<uint4 *>(to + v0) = v_now.x;
            if (v1 < D) *reinterpret_cast<uint4 *>(to + v1) = v_now.y;
        } else {
            const float div = p.c.v_scale ? __ldg(p.c.v_scale + at) : 1.0f;
            float x[8];
            widen8<T>(x, v_now.x);
            if (v0 < D) narrow8(to + v0, x, div);
            widen8<T>(x, v_now.y);
            if (v1 < D) narrow8(to + v1, x, div);
        }
        v_now = next;
    }
}

template <int MODE, typename T, typename C> static cudaError_t launch_mode(const NormRopeParams &p, cudaStream_t st)
{
    int width = 1;
    while (width < norm_tasks<MODE>(p.D, p.half)) width *= 2;
    auto go = [&](auto kernel, int tokens) {
        const int floats = tokens * norm_angles(p.half) + 2 * p.D + (MODE == NORM_ODD ? NORM_THREADS / width * p.D : 0);
        return launch_chained(kernel, dim3(p.B * ((p.T + tokens - 1) / tokens)), NORM_THREADS, floats * static_cast<int>(sizeof(float)), st, p, width);
    };
    // More tokens a block once that still gives every SM three blocks: 16 x 300 tokens take 27 us by eight, 28 by four, 53 by one,
    // 2,400 take 15 us by four and 29 by one.  A block's tokens are one sequence's, and places that it has no tokens for take as
    // long: by eight only where that pads T by no more than a twentieth over four (300 x 17 tokens 36 us by eight, 34 by four,
    // 1,300 x 3: 45 and 30), by four not for single tokens (4,096: 117 us by eight, 77 by four, 51 by one; 2,000 x 2: 62, 41, 49).
    const int64_t blocks = static_cast<int64_t>(p.B) * p.T / (3 * 152), by_eight = (p.T + 7ll) / 8 * 8, by_four = (p.T + 3ll) / 4 * 4;
    if (blocks >= 8 && 20 * by_eight <= 21 * by_four) return go(norm_rope_kernel<MODE, 8, T, C>, 8);
    if (blocks >= 4 && p.T > 1) return go(norm_rope_kernel<MODE, 4, T, C>, 4);
    return go(norm_rope_kernel<MODE, 1, T, C>, 1);
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
