// spv_rope.cu -- rotary positions of new tokens' q and k, joined with the
// write of k and v into the paged cache.
//
// A block takes one token: its threads first compute the token's rotary_dim / 2 cosines and sines into shared memory, once for all
// heads, then move the heads 8 elements (16 bytes) at a time.  The angle is
// the integer product of the position with a 64-bit fraction of a turn: the
// wrap of the product is the reduction to one turn, exact at any position,
// with no 64-bit floating point.
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
    ROPE_HALVES,  // a task is 8 elements and their partners half a rotation away; then 8 passing elements each
    ROPE_SCALAR   // halves whose length is no multiple of 8: the same, element by element
};
template <int MODE> __device__ __forceinline__ int head_tasks(const RopeParams &p)
{
    if (MODE == ROPE_PAIRS) return p.D >> 3;
    if (MODE == ROPE_HALVES) return (p.half >> 3) + ((p.D - 2 * p.half) >> 3);
    return ((p.half + 7) >> 3) + ((p.D - 2 * p.half + 7) >> 3);
}

template <int MODE, typename T, typename C>
__device__ __forceinline__ void rope_task(const T *src, C *dst, int i, const float2 *cs, const RopeParams &p, float div)
{
    if (MODE == ROPE_PAIRS) {
        float y[8];
        load8(src + 8 * i, y);
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            if (8 * i + j < 2 * p.half) {
                const float2 w = cs[4 * i + (j >> 1)];
                const float u = y[j], v = y[j + 1];
                y[j] = u * w.x - v * w.y;
                y[j + 1] = v * w.x + u * w.y;
            }
        store8(dst + 8 * i, y, div);
    } else if (MODE == ROPE_HALVES) {
        const int n = p.half >> 3;
        float y[8];
        if (i >= n) {
            const int d = 2 * p.half + 8 * (i - n);
            load8(src + d, y);
            store8(dst + d, y, div);
            return;
        }
        float z[8];
        load8(src + 8 * i, y);
        load8(src + 8 * i + p.half, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 w = cs[8 * i + j];
            const float u = y[j], v = z[j];
            y[j] = u * w.x - v * w.y;
            z[j] = v * w.x + u * w.y;
        }
        store8(dst + 8 * i, y, div);
        store8(dst + 8 * i + p.half, z, div);
    } else {
        const int n = (p.half + 7) >> 3;
        for (int j = 0; j < 8; ++j) {
            if (i >= n) {
                const int d = 2 * p.half + 8 * (i - n) + j;
                if (d < p.D) dst[d] = Num<C>::down(sizeof(C) == 1 ? Num<T>::up(src[d]) / div : Num<T>::up(src[d]));
                continue;
            }
            const int d = 8 * i + j;
            if (d >= p.half) return;
            const float2 w = cs[d];
            const float u = Num<T>::up(src[d]), v = Num<T>::up(src[d + p.half]);
            const float a = u * w.x - v * w.y, b = v * w.x + u * w.y;
            dst[d] = Num<C>::down(sizeof(C) == 1 ? a / div : a);
            dst[d + p.half] = Num<C>::down(sizeof(C) == 1 ? b / div : b);
        }
    }
}

template <int MODE, typename T, typename C> __global__ void __launch_bounds__(256) rope_kernel(const RopeParams p)
{
    __shared__ float2 cs[256];
    const int n = blockIdx.x, b = n / p.T, t = n - b * p.T;
    const SeqLens s = seq_lens(p.ctx_lens, p.new_lens, b, p.T, p.c);
    const int32_t *row = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    if (t == 0 && p.row_status) {  // all pages that the sequence's new tokens touch
        int bad = s.bad;
        if (s.total > 0)
            for (int g = (s.ctx >> p.c.page_shift) + threadIdx.x; g <= (s.total - 1) >> p.c.page_shift; g += blockDim.x)
                bad |= page_of(p.c, row, g << p.c.page_shift) < 0;
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) p.row_status[b] = bad ? KV_STATUS_BAD : 0;
    }
    T *q_out = static_cast<T *>(p.q_out) + static_cast<int64_t>(n) * p.q_heads * p.D;
    if (s.bad || t >= s.fresh) {
        for (int i = threadIdx.x; i < p.q_heads * (p.D >> 3); i += blockDim.x)
            reinterpret_cast<uint4 *>(q_out)[i] = uint4{};
        return;
    }
    const int slot = s.ctx + t;
    const int pos = p.positions ? __ldg(p.positions + n) : slot;
    for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * __ldg(p.freqs + i);
        // the top 32 bits, signed: half a turn either way, at most 2^-33 turns off
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>((turn + (1ull << 31)) >> 32)) * 0x1p-31f, &sn, &cn);
        cs[i] = make_float2(cn * p.mscale, sn * p.mscale);
    }
    const int page = page_of(p.c, row, slot);
    if (p.slot_pos && slot < p.pos_stride)
        for (int h = threadIdx.x; h < p.c.kv_heads; h += blockDim.x)
            p.slot_pos[(static_cast<int64_t>(b) * p.c.kv_heads + h) * p.pos_stride + slot] = pos;
    __syncthreads();
    const int per = head_tasks<MODE>(p), D8 = p.D >> 3;
    const T *q = static_cast<const T *>(p.q) + b * p.stride[0] + t * p.stride[1];
    for (int i = threadIdx.x; i < p.q_heads * per; i += blockDim.x) {
        const int h = i / per;
        rope_task<MODE>(q + h * p.D, q_out + h * p.D, i - h * per, cs, p, 1.0f);
    }
    if (page < 0) return;
    const T *k = static_cast<const T *>(p.k) + b * p.stride[2] + t * p.stride[3];
    for (int i = threadIdx.x; i < p.c.kv_heads * per; i += blockDim.x) {
        const int h = i / per;
        C *dst = reinterpret_cast<C *>(const_cast<char *>(row_ptr(p.c, p.c.k, page, slot, h)));
        rope_task<MODE>(k + h * p.D, dst, i - h * per, cs, p, sizeof(C) == 1 && p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.0f);
    }
    const T *v = static_cast<const T *>(p.v) + b * p.stride[4] + t * p.stride[5];
    for (int i = threadIdx.x; i < p.c.kv_heads * D8; i += blockDim.x) {
        const int h = i / D8, d = (i - h * D8) << 3;
        C *dst = reinterpret_cast<C *>(const_cast<char *>(row_ptr(p.c, p.c.v, page, slot, h)));
        float y[8];
        load8(v + h * p.D + d, y);
        store8(dst + d, y, sizeof(C) == 1 && p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.0f);
    }
}

template <typename T, typename C> static cudaError_t launch(const RopeParams &p, cudaStream_t st)
{
    const int grid = p.B * p.T;
    if (p.interleaved || p.half == 0)
        rope_kernel<ROPE_PAIRS, T, C><<<grid, 256, 0, st>>>(p);
    else if (p.half % 8 == 0)
        rope_kernel<ROPE_HALVES, T, C><<<grid, 256, 0, st>>>(p);
    else
        rope_kernel<ROPE_SCALAR, T, C><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
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
