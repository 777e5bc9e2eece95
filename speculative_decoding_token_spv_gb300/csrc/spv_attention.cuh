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
    unsigned *error;  // the workspace's error word
    struct SplitItem *split;  // [block][2]: the items that the block has pieces of
    float *parts;             // [block][2] pieces: m and l of each row, then o
    int q_heads, group, rows;
    float scale_log2;
    GiveUp give_up;
};

// The weights of a product in M are 2^(s - m), m the running maximum less UP, which the largest score may pass by LAG: at
// most 2^14 in f16, whose smallest value is then 2^-32 of the largest weight and not 2^-25 -- a long cache of keys below
// that would add to the sum l, held in 32 bits, and not to the output (262,143 keys of 2^-25 beside one of 1: 2^-7 of the
// result).  bf16 has the exponents of 32 bits.
template <typename M> struct Weights {
    static constexpr bool F16 = std::is_same<M, __half>::value;
    static constexpr float UP = F16 ? 7.0f : 0.0f, LAG = F16 ? 7.0f : 8.0f;
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

// An item whose tiles more than one block has: blocks b0 .. b1.  Each of them
// leaves its piece in the workspace -- b0, where the item begins, in its
// second place, the others in their first -- and the join kernel puts them
// together.  A block's two entries are written by every call; n = 0: none.
struct SplitItem {
    int b0, n;  // n = b1 - b0 + 1
    AttRows rows;
};

__device__ __forceinline__ float *piece_of(const AttParams &p, int i, int b0, int size)
{
    return p.parts + (static_cast<int64_t>(i) * 2 + (i == b0 ? 1 : 0)) * size;
}

// Notes that this block has a piece of the cursor's item; `begin` is the start
// of its range.
template <typename Lens>
__device__ __forceinline__ void note_split(const AttParams &p, const CursorOf<Lens> &c, const AttRows &rows, long long begin, int tid)
{
    if (tid != 0) return;
    SplitItem s;
    s.b0 = range_owner(c, c.first);
    s.n = range_owner(c, c.first + c.tiles - 1) - s.b0 + 1;
    s.rows = rows;
    p.split[blockIdx.x * 2 + (c.first < begin ? 0 : 1)] = s;
}

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

// Joins the pieces of the items that blocks share, after the kernel that wrote
// them (a programmatic dependent launch of as many blocks as that had).  R:
// rows of a piece.
cudaError_t launch_join(const AttParams &p, spv_dtype q, int D, int R, int blocks, cudaStream_t st);

// Room for the entries of `blocks` blocks.
constexpr size_t split_bytes(int blocks) { return (static_cast<size_t>(blocks) * 2 * sizeof(SplitItem) + 255) / 256 * 256; }

// Workspace: header, the blocks' split items, their pieces.
constexpr size_t ATT_PARTS_AT = WS_HEADER + split_bytes(ATT_MAX_BLOCKS);

cudaError_t launch_attention_rows(const AttParams &p, const KvLaunch &L, cudaStream_t st);
size_t attention_rows_part_floats(int head_dim);  // of all blocks' pieces

}  // namespace spv
