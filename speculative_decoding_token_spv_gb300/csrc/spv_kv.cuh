// spv_kv.cuh -- shared pieces of the calls around the verify step: the paged
// cache as the kernels see it, which slots a new token sees, and how the work
// of the attention calls is cut into pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "spv_internal.h"

namespace spv {

constexpr int KV_STATUS_BAD = 4;  // SPV_ERR_BAD_ROW
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// One pool (K or V): byte strides.
struct PoolView {
    char *base;
    int64_t page_stride, slot_stride, head_stride;
};

struct PagedView {
    PoolView k, v;
    const float *k_scale, *v_scale;
    const int32_t *table;
    int max_pages, num_pages, page_shift, kv_heads;
};

// Page of slot j of the sequence whose table row is `row`; -1 if its id is
// outside the pool.  j must lie below max_pages << page_shift.
__device__ __forceinline__ int page_of(const PagedView &c, const int32_t *row, int j)
{
    const int p = __ldg(row + (j >> c.page_shift));
    return static_cast<unsigned>(p) < static_cast<unsigned>(c.num_pages) ? p : -1;
}

__device__ __forceinline__ const char *row_ptr(const PagedView &c, const PoolView &pool, int page, int j, int h)
{
    return pool.base + page * pool.page_stride + (j & ((1 << c.page_shift) - 1)) * pool.slot_stride +
           h * pool.head_stride;
}

// Lengths of sequence b: cached slots, new tokens, and their sum (0 when the
// lengths are bad -- negative, or beyond T or the table -- and, unless `idle`,
// when there is no new token).
struct SeqLens {
    int ctx, fresh, total;
    bool bad;
};
__device__ __forceinline__ SeqLens seq_lens(const int32_t *ctx_lens, const int32_t *new_lens, int b, int T,
                                            const PagedView &c, bool idle = false)
{
    SeqLens s;
    s.ctx = __ldg(ctx_lens + b);
    s.fresh = new_lens ? __ldg(new_lens + b) : T;
    const int64_t cap = static_cast<int64_t>(c.max_pages) << c.page_shift;
    s.bad = s.ctx < 0 || s.fresh < 0 || s.fresh > T || static_cast<int64_t>(s.ctx) + s.fresh > cap;
    s.total = s.bad || (s.fresh == 0 && !idle) ? 0 : s.ctx + s.fresh;
    return s;
}

// Bit u of the result: new token t sees new token u.  Chain (parent null):
// u <= t; tree: t and its ancestors.  0 when the path to the root leaves
// [0, node): the token then sees nothing at all.  t < 64.
__device__ __forceinline__ unsigned long long visible_mask(const int32_t *parent, int t)
{
    if (!parent) return (2ull << t) - 1ull;
    unsigned long long m = 1ull << t;
    while (t > 0) {
        const int p = __ldg(parent + t);
        if (p < 0 || p >= t) return 0ull;
        m |= 1ull << p;
        t = p;
    }
    return m;
}

// The attention calls cut their work into tiles of `tile` keys of an item (a
// sequence, a tile of query rows, a key head), number the tiles of all items
// in a row (sequence-major, then row tile, then head) and give each block of
// the grid an equal range of them, so that any mix of lengths fills the GPU
// evenly and the host needs to know no length.  An item of no keys still has
// one tile: its outputs have to be written.
struct Work {
    int B, T, row_tiles, tile;
    const int32_t *ctx_lens, *new_lens;
    bool idle;  // sequences without new tokens have work too
};
__device__ __forceinline__ SeqLens lens_of(const Work &w, int b, const PagedView &c)
{
    return seq_lens(w.ctx_lens, w.new_lens, b, w.T, c, w.idle);
}
// Tiles at a sequence's beginning that its new tokens do not see at all.
__device__ __forceinline__ int skipped_tiles(const Work &, const SeqLens &) { return 0; }
// The first slot that any of them sees; pages that end before it may be missing.
__device__ __forceinline__ int first_seen(const SeqLens &) { return 0; }

// A block's range [at, end) and the item that it is in: `first` is the number
// of the item's first tile, `tiles` how many it has.
template <typename Lens> struct CursorOf {
    long long all, at, end, first;
    long long part;  // tiles of a block; the first `more` blocks have one tile more
    int blocks, more;  // blocks that have work
    int b, row_tile, h, tiles;
    Lens s;
};
using Cursor = CursorOf<SeqLens>;
template <typename W, typename Lens> __device__ __forceinline__ int tiles_of(const W &w, const Lens &s)
{
    return s.total == 0 ? 1 : (s.total + w.tile - 1) / w.tile - skipped_tiles(w, s);
}
// a / b; in 32 bits, a tenth of the time, where a fits them (nearly always).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}
template <typename Lens> __device__ __forceinline__ long long range_begin(const CursorOf<Lens> &c, int block)
{
    return c.part * block + min(block, c.more);
}
// The block whose range holds tile x.
template <typename Lens> __device__ __forceinline__ int range_owner(const CursorOf<Lens> &c, long long x)
{
    const long long large = (c.part + 1) * c.more;  // tiles of the blocks that have one more
    return static_cast<int>(x < large ? quotient(x, c.part + 1) : c.more + quotient(x - large, c.part));
}

// Finds the range of block `block` of `grid`; one warp, all lanes get the
// same.  at == end: nothing to do.
template <typename W> __device__ __forceinline__ auto find_range(const W &w, const PagedView &v, int block, int grid, int lane)
{
    using Lens = decltype(lens_of(w, 0, v));
    const int per = w.row_tiles * v.kv_heads;
    // Tiles of sequences lane, lane + 32, ...: the first KEEP of them stay in registers, their loads all under way
    // at once (a load is about a microsecond when the lengths come from memory).
    constexpr int KEEP = 2;
    int tiles[KEEP];
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        const int b = 32 * i + lane;
        tiles[i] = b < w.B ? tiles_of(w, lens_of(w, b, v)) : 0;
        sum += tiles[i];
    }
    for (int b = 32 * KEEP + lane; b < w.B; b += 32) sum += tiles_of(w, lens_of(w, b, v));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum *= per;
    CursorOf<Lens> c{};
    c.all = sum;
    c.blocks = sum < grid ? static_cast<int>(sum) : grid;
    if (block >= c.blocks) return c;
    c.part = quotient(sum, c.blocks);
    c.more = static_cast<int>(sum - c.part * c.blocks);
    c.at = range_begin(c, block);
    c.end = range_begin(c, block + 1);
    long long before = 0;
    bool found = false;
    auto look = [&](int b0, int mine) {  // among sequences b0 .. b0 + 31, whose tiles the lanes have
        int upto = mine;  // 32 sequences' tiles fit 32 bits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned here = __ballot_sync(0xffffffffu, before + static_cast<long long>(upto) * per > c.at);
        if (here) {
            const int l = __ffs(here) - 1;
            c.b = b0 + l;
            before += static_cast<long long>(__shfl_sync(0xffffffffu, upto - mine, l)) * per;
            found = true;
        } else {
            before += static_cast<long long>(__shfl_sync(0xffffffffu, upto, 31)) * per;
        }
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (!found && 32 * i < w.B) look(32 * i, tiles[i]);
    for (int b0 = 32 * KEEP; !found && b0 < w.B; b0 += 32) {
        const int b = b0 + lane;
        look(b0, b < w.B ? tiles_of(w, lens_of(w, b, v)) : 0);
    }
    c.s = lens_of(w, c.b, v);
    c.tiles = tiles_of(w, c.s);
    const long long in = c.at - before;
    const int item = static_cast<int>(quotient(in, c.tiles));
    c.first = before + static_cast<long long>(item) * c.tiles;
    c.row_tile = item / v.kv_heads;
    c.h = item - c.row_tile * v.kv_heads;
    return c;
}
// To the next item (the range goes on behind the present one).
template <typename Lens, typename W> __device__ __forceinline__ void next_item(CursorOf<Lens> &c, const W &w, const PagedView &v)
{
    c.first += c.tiles;
    c.at = c.first;
    if (++c.h < v.kv_heads) return;
    c.h = 0;
    if (++c.row_tile < w.row_tiles) return;
    c.row_tile = 0;
    if (++c.b == w.B) return;  // the end of everything
    c.s = lens_of(w, c.b, v);
    c.tiles = tiles_of(w, c.s);
}

// All kernels of these calls are programmatic dependent launches of what is
// before them in the stream: launched, and set up as far as needs no memory,
// while that still runs.  Each begins with chain_begin: it waits until
// everything before it is done and visible, and lets the next one launch.
__device__ __forceinline__ void chain_begin()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, Args... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T> struct Num;
template <> struct Num<__nv_bfloat16> {
    __device__ static __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Num<__half> {
    __device__ static __forceinline__ float up(__half x) { return __half2float(x); }
    __device__ static __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <> struct Num<__nv_fp8_e4m3> {
    __device__ static __forceinline__ float up(__nv_fp8_e4m3 x) { return static_cast<float>(x); }
    __device__ static __forceinline__ __nv_fp8_e4m3 down(float x) { return __nv_fp8_e4m3(x); }  // saturates
};

}  // namespace spv
