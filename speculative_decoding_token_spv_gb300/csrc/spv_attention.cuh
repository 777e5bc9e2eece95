// spv_attention.cuh -- what the two attention kernels share: their arguments,
// the pieces in the workspace and how they are joined.
#pragma once

#include "spv_mma.cuh"

namespace spv {

constexpr int ATT_SMS = 152;
constexpr int ATT_MAX_BLOCKS = 3 * ATT_SMS;

struct AttParams {
    PagedView c;
    Work w;
    const void *q;
    void *out;
    float *lse;
    const int32_t *parent;
    int32_t *row_status;
    // Pieces of the item that begins in block i and ends in a later one (there is at most one) that are done; zero
    // between calls.
    unsigned *arrived;
    unsigned *error;  // the workspace's error word
    float *parts;  // [block][2] pieces: m and l of each row, then o
    int q_heads, group, rows;
    float scale_log2;
};

template <typename T> __device__ __forceinline__ bool not_finite16(uint32_t two)
{
    const uint32_t e = sizeof(T) == 1 ? 0 : std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (two & e) == e || ((two >> 16) & e) == e;
}
// Whether a 16-byte chunk of the cache holds an infinity or NaN.
template <typename C> __device__ __forceinline__ bool chunk_not_finite(uint4 x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(C) == 1) {  // e4m3 has no infinities; NaN is 0x7f and 0xff
#pragma unroll
            for (int k = 0; k < 4; ++k) odd |= ((w[i] >> (8 * k)) & 0x7fu) == 0x7fu;
        } else {
            odd |= not_finite16<C>(w[i]);
        }
    }
    return odd;
}


// A tile of an item's rows: which they are, and what is written for them.
struct AttRows {
    int b, h, row0, live;  // rows row0 .. row0 + live - 1 of key head h
};

// Result of row r of the tile, columns d .. d + 3: out = x v_scale / l, or what
// stands for it (mr NaN: a bad sequence; no sum at all: 0 and minus infinity).
template <typename T, int D>
__device__ __forceinline__ void write_row(const AttParams &p, const AttRows &w, int r, int d, float4 x, float mr, float lr,
                                          float v_scale)
{
    const int t = (w.row0 + r) / p.group, g = (w.row0 + r) - t * p.group;
    const int64_t at = (static_cast<int64_t>(w.b) * p.w.T + t) * p.q_heads + w.h * p.group + g;
    const bool nan = mr != mr, none = mr == -CUDART_INF_F && lr == 0.0f;
    const float inv = v_scale / lr;
    x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
    if (none) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (nan) x = make_float4(mr, mr, mr, mr);
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + at * D + d) = make_uint2(pack_mma<T>(x.x, x.y), pack_mma<T>(x.z, x.w));
    if (d == 0 && p.lse) p.lse[at] = nan ? mr : none ? -CUDART_INF_F : LN2 * (mr + log2f(lr));
}

// Block i's piece of the item that begins in block b0: there it lies in the
// second place, in the later blocks in the first.
__device__ __forceinline__ float *piece_of(const AttParams &p, int i, int b0, int size)
{
    return p.parts + (static_cast<int64_t>(i) * 2 + (i == b0 ? 1 : 0)) * size;
}

// Called by all THREADS threads (whole warps) once their block's piece of the
// item is in the workspace; `sync` is their barrier.  True for the block that
// came last: it has joined the pieces, in their order, and written the rows.
// ms and ls hold R floats each.
template <typename T, int D, int R, int THREADS, typename Sync>
__device__ __forceinline__ bool join_pieces(const AttParams &p, const AttRows &w, const Cursor &c, int tid, float *ms,
                                            float *ls, int *flag, float v_scale, Sync &&sync)
{
    constexpr int PART = R * (D + 2);
    const int b0 = range_owner(c, c.first), b1 = range_owner(c, c.first + c.tiles - 1);
    __threadfence();
    sync();
    if (tid == 0) {
        const bool last = atomicAdd(p.arrived + b0, 1u) == static_cast<unsigned>(b1 - b0);
        if (last) p.arrived[b0] = 0;
        *flag = last;
    }
    sync();
    const bool last = *reinterpret_cast<volatile int *>(flag) != 0;
    sync();
    if (!last) return false;
    __threadfence();
    for (int r = tid >> 5; r < w.live; r += THREADS / 32) {
        float mr = -CUDART_INF_F, lr = 0.0f;
        bool nan = false;
        for (int i = b0 + (tid & 31); i <= b1; i += 32) {
            const float x = __ldcg(piece_of(p, i, b0, PART) + r);
            nan |= x != x;
            mr = fmaxf(mr, x);
        }
        mr = warp_max(mr);
        nan = __any_sync(0xffffffffu, nan);
        const float base = mr == -CUDART_INF_F ? 0.0f : mr;
        for (int i = b0 + (tid & 31); i <= b1; i += 32) {
            const float *x = piece_of(p, i, b0, PART);
            lr += __ldcg(x + R + r) * fast_exp2(__ldcg(x + r) - base);
        }
        lr = warp_sum(lr);
        if ((tid & 31) == 0) {
            ms[r] = nan ? CUDART_NAN_F : mr;
            ls[r] = lr;
        }
    }
    sync();
    for (int i = tid; i < w.live * (D / 4); i += THREADS) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        const float mr = ms[r], base = mr == -CUDART_INF_F ? 0.0f : mr;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = b0; k <= b1; ++k) {
            const float *y0 = piece_of(p, k, b0, PART);
            const float a = fast_exp2(__ldcg(y0 + r) - base);
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(y0 + 2 * R + r * D + d));
            x.x += a * y.x, x.y += a * y.y, x.z += a * y.z, x.w += a * y.w;
        }
        write_row<T, D>(p, w, r, d, x, mr, ls[r], v_scale);
    }
    return true;
}

cudaError_t launch_attention_rows(const AttParams &p, spv_dtype q, spv_dtype cache, int D, cudaStream_t st);
size_t attention_rows_part_floats(int head_dim);  // of all blocks' pieces

}  // namespace spv
