// spv_mass.cu -- the attention weight that each cached key received from the
// tokens that stand after a verify step, added up.
//
// The weights are recomputed from q, K and the attention's log-sum-exp:
// exp(s - lse) needs no second pass and no maximum, so K is read once, no
// score is kept between the calls and no piece has to be joined.  The work is
// cut along the cache as in the attention (Work, Cursor); each warp has its own
// ring of 16-key slices, filled by asynchronous copies, and takes a slice's
// fragments through the tensor cores against the counted rows, 16 at a time
// from shared memory.  What a slice's 16 keys received is a sum over rows: a
// thread's two rows, then a butterfly over the eight threads that share its
// columns.
#include "spv_mma.cuh"

namespace spv {

constexpr int MASS_WARPS = 4;
constexpr int MASS_THREADS = 32 * MASS_WARPS;
constexpr int MASS_KEYS = 16 * MASS_WARPS;
constexpr int MASS_SMS = 152;

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

// Rows that a block holds in shared memory at once; more go in several passes
// over the slices (from the L2, for the second time).
template <typename C, int D> struct MassShape {
    static constexpr int ROW_BYTES = D * static_cast<int>(sizeof(C));
    static constexpr int SLICE = 16 * ROW_BYTES;
    static constexpr int STAGES = 16384 / SLICE < 2 ? 2 : 16384 / SLICE > 8 ? 8 : 16384 / SLICE;
    static constexpr int ROWS = D == 256 ? 32 : 64;
    static constexpr int Q = ROWS * D * 2;
    static constexpr int SMEM = Q + MASS_WARPS * STAGES * SLICE;
    static constexpr int BLOCKS_PER_SM = SMEM * 3 <= 216 * 1024 ? 3 : 2;
};

template <typename T, typename C, int D>
__global__ void __launch_bounds__(MASS_THREADS, MassShape<C, D>::BLOCKS_PER_SM) mass_kernel(const MassParams p)
{
    using S = MassShape<C, D>;
    using M = typename MmaOf<T, C>::type;
    constexpr int NST = S::STAGES, ROWS = S::ROWS;
    extern __shared__ __align__(1024) char smem[];
    __shared__ float q_unit[ROWS], zs[ROWS];    // log-sum-exp in powers of two; infinity: a row that gives nothing
    __shared__ unsigned long long sees[ROWS];
    __shared__ Cursor cur0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t qs32 = smem_u32(smem), ring = smem_u32(smem + S::Q) + warp * (NST * S::SLICE);
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
        const int t1 = c.s.total > 0 ? static_cast<int>((c.end < item_end ? c.end : item_end) - c.first) : t0;
        if (p.row_status && t0 == 0 && c.h == 0) {
            int any = bad;
            for (int g = tid; c.s.total > 0 && g <= (c.s.total - 1) >> p.c.page_shift; g += MASS_THREADS)
                any |= page_of(p.c, table, g << p.c.page_shift) < 0;
            any = __syncthreads_or(any);
            if (tid == 0) p.row_status[c.b] = any ? KV_STATUS_BAD : 0;
        }
        if (bad) continue;
        if (c.s.fresh < 64) counted &= (1ull << c.s.fresh) - 1ull;
        const int rows = __popcll(counted) * p.group;
        const float unit = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        const int64_t out_row = (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.stride;
        // at least one pass: without counted rows the old mass is carried over
        for (int r0 = 0; r0 == 0 || r0 < rows; r0 += ROWS) {
            const int live = min(ROWS, rows - r0), groups = (live + 15) >> 4;
            const int t_end = rows > 0 ? t1 : t0;
            bool unused = false;
            SliceSource src = find_slice(p.c, table, t0 * MASS_KEYS + warp * 16, t0 < t_end ? c.s.total : 0, lane, &unused);
            auto issue = [&](int tile) {
                if (tile < t_end) {
                    const int j0 = tile * MASS_KEYS + warp * 16;
                    copy_slice<S::ROW_BYTES>(p.c, p.c.k, src, j0, c.h, ring + ((tile - t0) % NST) * S::SLICE, lane);
                    src = find_slice(p.c, table, j0 + MASS_KEYS, tile + 1 < t_end ? c.s.total : 0, lane, &unused);
                }
                cp_async_commit();
            };
            __syncthreads();  // q and the rings of the pass before are no longer read
#pragma unroll
            for (int i = 0; i < NST - 1; ++i) issue(t0 + i);
            for (int i = tid; i < groups * 16 * (D / 8); i += MASS_THREADS) {
                const int r = i / (D / 8), d = (i - r * (D / 8)) * 8;
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.0f;
                float z = CUDART_INF_F;
                unsigned long long see = 0;
                if (r < live) {
                    const int nth = (r0 + r) / p.group, g = r0 + r - nth * p.group;
                    unsigned long long m = counted;
                    for (int e = 0; e < nth; ++e) m &= m - 1;
                    const int t = __ffsll(m) - 1;
                    const int64_t at = (static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g;
                    const uint4 raw = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + at * D + d);
                    const T *y = reinterpret_cast<const T *>(&raw);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = Num<T>::up(y[e]);
                    if (d == 0) {
                        see = visible_mask(p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr, t);
                        z = __ldg(p.lse + at) * LOG2E;
                        if (z == -CUDART_INF_F || see == 0) z = CUDART_INF_F;
                    }
                }
                float down = 1.0f;
                if (sizeof(C) == 1) {
                    float top = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fabsf(x[e]) < CUDART_INF_F ? fmaxf(top, fabsf(x[e])) : top;
#pragma unroll
                    for (int o = D / 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int e2 = top > 0.0f ? max(-120, min(120, 14 - ilogbf(top))) : 0;
                    const float up = exp2f(static_cast<float>(e2));
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= up;
                    down = exp2f(static_cast<float>(-e2));
                }
                put_q8<M, C, D>(smem, r, d, x);
                if (d == 0) {
                    q_unit[r] = unit * down;
                    zs[r] = z;
                    sees[r] = see;
                }
            }
            __syncthreads();
            auto carried = [&](int j) {  // what key j has so far
                if (r0 > 0) return p.mass_out[out_row + j];
                return p.mass_in && j < c.s.ctx ? p.decay * p.mass_in[out_row + j] : 0.0f;
            };
            // lanes 0..15: the page (-1: nothing is written) and the old mass of this lane's key of a tile, asked for
            // a tile ahead
            auto page_for = [&](int tile) {
                const int j = tile * MASS_KEYS + warp * 16 + lane;
                return lane < 16 && tile < t_end && j < c.s.total ? __ldg(table + (j >> p.c.page_shift)) : -1;
            };
            auto mass_for = [&](int tile) {
                const int j = tile * MASS_KEYS + warp * 16 + lane;
                return lane < 16 && tile < t_end && j < c.s.total ? carried(j) : 0.0f;
            };
            int next_page = page_for(t0);
            float next_mass = mass_for(t0);
            for (int tile = t0; tile < t_end; ++tile) {
                __syncwarp();
                issue(tile + NST - 1);
                const int j0 = tile * MASS_KEYS + warp * 16;
                if (j0 >= c.s.total) break;
                const int j = j0 + lane, page = next_page;
                const float old = next_mass;
                next_page = page_for(tile + 1);
                next_mass = mass_for(tile + 1);
                cp_async_wait<NST - 1>();
                __syncwarp();
                const uint32_t slice = ring + ((tile - t0) % NST) * S::SLICE;
                uint32_t kf[D / 16][4];
                get_k<C, D>(kf, slice, lane);
                const bool tail = j0 + 16 > c.s.ctx;
                float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // [key tile][column]
                for (int g = 0; g < groups; ++g) {
                    float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t a[4];
                        get_q<D>(a, qs32, g, ks, lane);
                        mma16816<M>(s[0], a, kf[ks][0], kf[ks][1]);
                        mma16816<M>(s[1], a, kf[ks][2], kf[ks][3]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = g * 16 + i * 8 + (lane >> 2);
                        const float f = q_unit[r], z = zs[r];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float w = fast_exp2(s[k][2 * i + e] * f - z);
                                if (tail) {
                                    const int key = j0 + 8 * k + 2 * (lane & 3) + e;
                                    if (!(key < c.s.ctx || (key < c.s.total && (sees[r] >> (key - c.s.ctx) & 1)))) w = 0.0f;
                                }
                                if (z == CUDART_INF_F) w = 0.0f;
                                sum[k][e] += w;
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) sum[k][e] += __shfl_xor_sync(0xffffffffu, sum[k][e], o);
                    }
                // lane l < 16 writes key l: column l & 1 of the thread (l % 8) / 2 in key tile l / 8
                const int from = (lane & 7) >> 1;
                const float a = __shfl_sync(0xffffffffu, sum[0][0], from), b = __shfl_sync(0xffffffffu, sum[0][1], from);
                const float d = __shfl_sync(0xffffffffu, sum[1][0], from), e = __shfl_sync(0xffffffffu, sum[1][1], from);
                const float mine = (lane & 8) ? ((lane & 1) ? e : d) : ((lane & 1) ? b : a);
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages)) p.mass_out[out_row + j] = old + mine;
            }
            cp_async_wait<0>();
            if (rows == 0)
                for (int j = t0 * MASS_KEYS + tid; j < min(t1 * MASS_KEYS, c.s.total); j += MASS_THREADS)
                    if (page_of(p.c, table, j) >= 0) p.mass_out[out_row + j] = carried(j);
        }
    }
}

template <typename T, typename C, int D> static cudaError_t launch_dim(const MassParams &p, cudaStream_t st)
{
    using S = MassShape<C, D>;
    auto kernel = mass_kernel<T, C, D>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<MASS_SMS * S::BLOCKS_PER_SM, MASS_THREADS, S::SMEM, st>>>(p);
    return cudaGetLastError();
}
template <typename T, typename C> static cudaError_t launch_types(const MassParams &p, int D, cudaStream_t st)
{
    if (D == 64) return launch_dim<T, C, 64>(p, st);
    if (D == 128) return launch_dim<T, C, 128>(p, st);
    return launch_dim<T, C, 256>(p, st);
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
        return eight ? launch_types<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                     : launch_types<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_types<__half, __nv_fp8_e4m3>(p, D, st) : launch_types<__half, __half>(p, D, st);
}

}  // namespace spv
