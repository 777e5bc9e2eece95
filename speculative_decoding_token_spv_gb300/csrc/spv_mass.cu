// spv_mass.cu -- the attention weight that each cached key received from the
// tokens that stand after a verify step, added up.
//
// The weights are recomputed from q, K and the attention's log-sum-exp:
// exp(s - lse) needs no second pass, so K is read once and no score is kept
// between the calls.
#include "spv_kv.cuh"

namespace spv {

constexpr int MASS_BLOCKS = 4 * 152;
constexpr int MASS_KEYS = 128;
constexpr int MASS_ROWS = 16;

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

template <typename T, typename C, int D> __global__ void __launch_bounds__(MASS_KEYS) mass_kernel(const MassParams p)
{
    __shared__ float qs[MASS_ROWS][D];
    __shared__ float zs[MASS_ROWS];
    __shared__ unsigned long long see[MASS_ROWS];
    __shared__ Cursor cur0;
    const int tid = threadIdx.x;
    if (tid < 32) {
        const Cursor c = find_range(p.w, p.c, blockIdx.x, gridDim.x, tid);
        if (tid == 0) cur0 = c;
    }
    __syncthreads();
    Cursor c = cur0;
    for (; c.at < c.end; next_item(c, p.w, p.c)) {
        bool bad = c.s.bad || c.s.total > p.stride;
        unsigned long long counted = counted_tokens(p, c.b, &bad);
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        const long long item_end = c.first + c.tiles;
        const int t0 = static_cast<int>(c.at - c.first);
        const int t1 = static_cast<int>((c.end < item_end ? c.end : item_end) - c.first);
        if (p.row_status && t0 == 0 && c.h == 0) {
            int any = bad;
            for (int g = tid; c.s.total > 0 && g <= (c.s.total - 1) >> p.c.page_shift; g += MASS_KEYS)
                any |= page_of(p.c, table, g << p.c.page_shift) < 0;
            any = __syncthreads_or(any);
            if (tid == 0) p.row_status[c.b] = any ? KV_STATUS_BAD : 0;
        }
        if (bad) continue;
        if (c.s.fresh < 64) counted &= (1ull << c.s.fresh) - 1ull;
        const int rows = __popcll(counted) * p.group;
        const float factor = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        for (int tile = t0; tile < t1; ++tile) {
            const int j = tile * MASS_KEYS + tid;
            const int page = j < c.s.total ? page_of(p.c, table, j) : -1;
            const C *k = page < 0 ? nullptr : reinterpret_cast<const C *>(row_ptr(p.c, p.c.k, page, j, c.h));
            float sum = 0.0f;
            for (int r0 = 0; r0 < rows; r0 += MASS_ROWS) {
                __syncthreads();
                for (int i = tid; i < MASS_ROWS * D; i += MASS_KEYS) {
                    const int r = i / D, d = i - r * D;
                    float x = 0.0f;
                    if (r0 + r < rows) {
                        const int n = (r0 + r) / p.group, g = r0 + r - n * p.group;
                        unsigned long long m = counted;
                        for (int e = 0; e < n; ++e) m &= m - 1;
                        const int t = __ffsll(m) - 1;
                        const int64_t at = (static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g;
                        x = Num<T>::up(static_cast<const T *>(p.q)[at * D + d]);
                        if (d == 0) {
                            zs[r] = __ldg(p.lse + at) * LOG2E;
                            see[r] = visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, t);
                        }
                    }
                    qs[r][d] = x;
                }
                __syncthreads();
                if (page < 0) continue;
                float acc[MASS_ROWS];
#pragma unroll
                for (int r = 0; r < MASS_ROWS; ++r) acc[r] = 0.0f;
                for (int d = 0; d < D; d += 4) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = Num<C>::up(k[d + e]);
#pragma unroll
                    for (int r = 0; r < MASS_ROWS; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r] += x[e] * qs[r][d + e];
                }
#pragma unroll
                for (int r = 0; r < MASS_ROWS; ++r)
                    if (r0 + r < rows && zs[r] != -CUDART_INF_F && see[r] != 0 &&
                        (j < c.s.ctx || (see[r] >> (j - c.s.ctx) & 1)))
                        sum += exp2f(acc[r] * factor - zs[r]);
            }
            if (page >= 0) {
                const int64_t at = (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.stride + j;
                if (p.mass_in && j < c.s.ctx) sum += p.decay * p.mass_in[at];
                p.mass_out[at] = sum;
            }
        }
    }
}

template <typename T, typename C> static cudaError_t launch_dim(const MassParams &p, int D, cudaStream_t st)
{
    if (D == 64)
        mass_kernel<T, C, 64><<<MASS_BLOCKS, MASS_KEYS, 0, st>>>(p);
    else if (D == 128)
        mass_kernel<T, C, 128><<<MASS_BLOCKS, MASS_KEYS, 0, st>>>(p);
    else
        mass_kernel<T, C, 256><<<MASS_BLOCKS, MASS_KEYS, 0, st>>>(p);
    return cudaGetLastError();
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
    const bool eight = k.cache.dtype == SPV_E4M3;
    const int D = k.cache.head_dim;
    if (k.dtype == SPV_BF16)
        return eight ? launch_dim<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st) : launch_dim<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_dim<__half, __nv_fp8_e4m3>(p, D, st) : launch_dim<__half, __half>(p, D, st);
}

}  // namespace spv
