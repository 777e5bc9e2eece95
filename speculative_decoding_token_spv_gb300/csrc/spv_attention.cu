// spv_attention.cu -- attention of a sequence's new tokens over its paged
// cache, in one pass over K and V.
//
// Mathematics: with scores in powers of two, s = q.k scale log2 e, a block
// keeps for each of its rows the running maximum m, l = sum 2^(s - m) and
// o = sum 2^(s - m) v over the keys of its piece; pieces of one item join as
// M = max m_i, l = sum l_i 2^(m_i - M), o likewise, out = o / l.  The last
// block of an item to finish joins its pieces in their order along the
// sequence, so the result does not depend on which block that is.
#include "spv_kv.cuh"

namespace spv {

constexpr int ATT_BLOCKS = 4 * 152;  // blocks of the grid
constexpr int ATT_ROWS = 16;         // query rows of a block's tile
constexpr int ATT_KEYS = 64;         // keys of a tile
constexpr int ATT_THREADS = 128;

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
    float *parts;       // [block][2] pieces: ATT_ROWS m, ATT_ROWS l, ATT_ROWS x D o
    int q_heads, group, rows;
    float scale_log2;
};

static int att_row_tiles(int T, int group) { return (T * group + ATT_ROWS - 1) / ATT_ROWS; }
// Workspace: header, arrival counters, pieces.  The counters' place is the
// same for every shape, so calls of different shapes can share a workspace.
constexpr size_t ATT_PARTS_AT = (WS_HEADER + ATT_BLOCKS * sizeof(unsigned) + 255) / 256 * 256;

size_t attention_ws_bytes(int, int, int, int, int head_dim)
{
    return ATT_PARTS_AT + static_cast<size_t>(ATT_BLOCKS) * 2 * ATT_ROWS * (head_dim + 2) * sizeof(float);
}

template <typename T, typename C, int D> __global__ void __launch_bounds__(ATT_THREADS) attention_kernel(const AttParams p)
{
    constexpr int R = ATT_ROWS, KT = ATT_KEYS, PART = R * (D + 2);
    constexpr int DPT = (D + ATT_THREADS - 1) / ATT_THREADS;  // output columns of a thread
    __shared__ float qs[R][D];
    __shared__ float ps[R][KT];
    __shared__ float ms[R], ls[R], as[R];
    __shared__ unsigned long long sees[64];
    __shared__ Cursor cur0;
    __shared__ int flag;
    const int tid = threadIdx.x;
    if (tid < 32) {
        const Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid);
        if (tid == 0) cur0 = c;
    }
    __syncthreads();
    Cursor c = cur0;
    const long long begin = c.at;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        const int row0 = c.row_tile * R;
        const long long item_end = c.first + c.tiles;
        const int t0 = static_cast<int>(c.at - c.first);
        const int t1 = static_cast<int>((c.end < item_end ? c.end : item_end) - c.first);
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        __syncthreads();
        if (tid == 0) flag = 0;
        for (int t = tid; t < p.w.T; t += ATT_THREADS) sees[t] = visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, t);
        for (int i = tid; i < R * D; i += ATT_THREADS) {
            const int r = i / D, d = i - r * D, t = (row0 + r) / p.group, g = (row0 + r) - t * p.group;
            float x = 0.0f;
            if (row0 + r < p.rows && t < c.s.fresh)
                x = Num<T>::up(static_cast<const T *>(p.q)[((static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g) * D + d]);
            qs[r][d] = x;
        }
        if (tid < R) {
            ms[tid] = -CUDART_INF_F;
            ls[tid] = 0.0f;
        }
        float o[R][DPT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < DPT; ++e) o[r][e] = 0.0f;
        const float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        bool bad = c.s.bad;
        __syncthreads();
        for (int tile = t0; tile < t1 && c.s.total > 0; ++tile) {
            const int j0 = tile * KT;
            const int j = j0 + tid % KT;
            int page = -1;
            if (j < c.s.total) {
                page = page_of(p.c, table, j);
                bad |= page < 0;
            }
            float acc[R / 2];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) acc[r] = 0.0f;
            if (page >= 0) {
                const C *k = reinterpret_cast<const C *>(row_ptr(p.c, p.c.k, page, j, c.h));
                for (int d = 0; d < D; d += 4) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = Num<C>::up(k[d + e]);
#pragma unroll
                    for (int r = 0; r < R / 2; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r] += x[e] * qs[(tid / KT) * (R / 2) + r][d + e];
                }
            }
#pragma unroll
            for (int r = 0; r < R / 2; ++r) {
                const int row = (tid / KT) * (R / 2) + r, t = (row0 + row) / p.group;
                bool seen = page >= 0 && row0 + row < p.rows && t < c.s.fresh;
                if (seen) seen = sees[t] != 0 && (j < c.s.ctx || (sees[t] >> (j - c.s.ctx) & 1));
                ps[row][tid % KT] = seen ? acc[r] * factor : -CUDART_INF_F;
            }
            __syncthreads();
            if (tid < R) {
                float m = ms[tid];
                for (int i = 0; i < KT; ++i) m = fmaxf(m, ps[tid][i]);
                const float m0 = m == -CUDART_INF_F ? 0.0f : m;
                as[tid] = exp2f(ms[tid] - m0);
                float l = ls[tid] * as[tid];
                for (int i = 0; i < KT; ++i) {
                    const float e = exp2f(ps[tid][i] - m0);
                    ps[tid][i] = e;
                    l += e;
                }
                ms[tid] = m;
                ls[tid] = l;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < DPT; ++e) {
                const int d = tid + e * ATT_THREADS;
                if (d < D) {
#pragma unroll
                    for (int r = 0; r < R; ++r) o[r][e] *= as[r];
                    for (int i = 0; i < KT && j0 + i < c.s.total; ++i) {
                        const int pg = page_of(p.c, table, j0 + i);
                        if (pg < 0) continue;
                        const float v = Num<C>::up(reinterpret_cast<const C *>(row_ptr(p.c, p.c.v, pg, j0 + i, c.h))[d]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (ps[r][i] != 0.0f) o[r][e] += ps[r][i] * v;
                    }
                }
            }
            __syncthreads();
        }
        if (bad) flag = 1;
        __syncthreads();
        const bool any_bad = flag != 0;
        const bool whole = t0 == 0 && t1 == c.tiles;
        if (!whole) {
            float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * PART;
            if (tid < R) {
                part[tid] = any_bad ? CUDART_NAN_F : ms[tid];
                part[R + tid] = ls[tid];
            }
#pragma unroll
            for (int e = 0; e < DPT; ++e) {
                const int d = tid + e * ATT_THREADS;
                if (d < D)
                    for (int r = 0; r < R; ++r) part[2 * R + r * D + d] = o[r][e];
            }
            __threadfence();
            __syncthreads();
            const int b0 = range_owner(c, c.first), b1 = range_owner(c, item_end - 1);
            if (tid == 0) flag = atomicAdd(p.arrived + b0, 1u) == static_cast<unsigned>(b1 - b0);
            __syncthreads();
            if (!flag) continue;
            __threadfence();
            if (tid == 0) p.arrived[b0] = 0;
            // join the pieces in order
            if (tid < R) {
                float m = -CUDART_INF_F;
                bool nan = false;
                for (int i = b0; i <= b1; ++i) {
                    const float x = p.parts[(static_cast<int64_t>(i) * 2 + (c.first < range_begin(c, i) ? 0 : 1)) * PART + tid];
                    nan |= x != x;
                    m = fmaxf(m, x);
                }
                const float m0 = m == -CUDART_INF_F ? 0.0f : m;
                float l = 0.0f;
                for (int i = b0; i <= b1; ++i) {
                    const float *x = p.parts + (static_cast<int64_t>(i) * 2 + (c.first < range_begin(c, i) ? 0 : 1)) * PART;
                    l += x[R + tid] * exp2f(x[tid] - m0);
                }
                ms[tid] = nan ? CUDART_NAN_F : m;
                ls[tid] = l;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < DPT; ++e) {
                const int d = tid + e * ATT_THREADS;
                if (d < D)
                    for (int r = 0; r < R; ++r) {
                        const float m0 = ms[r] == -CUDART_INF_F ? 0.0f : ms[r];
                        float x = 0.0f;
                        for (int i = b0; i <= b1; ++i) {
                            const float *y = p.parts + (static_cast<int64_t>(i) * 2 + (c.first < range_begin(c, i) ? 0 : 1)) * PART;
                            x += y[2 * R + r * D + d] * exp2f(y[r] - m0);
                        }
                        o[r][e] = x;
                    }
            }
        } else {
            if (any_bad && tid < R) ms[tid] = CUDART_NAN_F;
            __syncthreads();
        }
        const float v_scale = p.c.v_scale ? __ldg(p.c.v_scale + c.h) : 1.0f;
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= p.rows) break;
            const int t = (row0 + r) / p.group, g = (row0 + r) - t * p.group;
            const int64_t at = (static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g;
            const float m = ms[r], l = ls[r];
            const bool nan = m != m, none = m == -CUDART_INF_F && l == 0.0f;
#pragma unroll
            for (int e = 0; e < DPT; ++e) {
                const int d = tid + e * ATT_THREADS;
                if (d < D) static_cast<T *>(p.out)[at * D + d] = Num<T>::down(nan ? CUDART_NAN_F : none ? 0.0f : o[r][e] / l * v_scale);
            }
            if (tid == 0 && p.lse) p.lse[at] = nan ? CUDART_NAN_F : none ? -CUDART_INF_F : LN2 * (m + log2f(l));
        }
        if (tid == 0 && p.row_status && c.h == 0 && c.row_tile == 0) p.row_status[c.b] = ms[0] != ms[0] ? KV_STATUS_BAD : 0;
    }
}

template <typename T, typename C> static cudaError_t launch_dim(const AttParams &p, int D, cudaStream_t st)
{
    if (D == 64)
        attention_kernel<T, C, 64><<<ATT_BLOCKS, ATT_THREADS, 0, st>>>(p);
    else if (D == 128)
        attention_kernel<T, C, 128><<<ATT_BLOCKS, ATT_THREADS, 0, st>>>(p);
    else
        attention_kernel<T, C, 256><<<ATT_BLOCKS, ATT_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attention(const AttentionLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    AttParams p{};
    p.c = paged_view(k);
    p.group = k.q_heads / k.cache.kv_heads;
    p.w = Work{k.B, k.T, att_row_tiles(k.T, p.group), ATT_KEYS, k.ctx_lens, k.new_lens, false};
    p.q = L.q;
    p.out = L.out;
    p.lse = L.lse;
    p.parent = k.parent;
    p.row_status = k.row_status;
    p.q_heads = k.q_heads;
    p.rows = k.T * p.group;
    p.scale_log2 = k.scale * LOG2E;
    char *ws = static_cast<char *>(L.ws);
    p.arrived = reinterpret_cast<unsigned *>(ws + WS_HEADER);
    p.parts = reinterpret_cast<float *>(ws + ATT_PARTS_AT);
    const bool eight = k.cache.dtype == SPV_E4M3;
    const int D = k.cache.head_dim;
    if (k.dtype == SPV_BF16)
        return eight ? launch_dim<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st) : launch_dim<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_dim<__half, __nv_fp8_e4m3>(p, D, st) : launch_dim<__half, __half>(p, D, st);
}

}  // namespace spv
