// spv_evict.cu -- cuts each sequence's cache back to its budget by the
// accumulated attention weight, each key head by itself and in place.
//
// evict_select_kernel, one block per (sequence, head): every slot gets an
// order-preserving 32-bit key (protected slots the largest); a radix select
// over its digits finds the key of the last slot to stay and how many of its
// equals do; bit masks of the kept slots and prefix counts over their words
// then match the i-th hole below the budget with the i-th kept slot above.
// evict_move_kernel copies the rows of the matched slots.
#include "spv_kv.cuh"

namespace spv {

constexpr int EV_THREADS = 1024;
constexpr int EV_MOVE_SLOTS = 64;  // slots that a block of the move looks at

struct EvictParams {
    PagedView c;
    const int32_t *lens, *pos;
    const float *mass;
    float *mass_out;
    int32_t *pos_out, *new_lens, *slot_src, *row_status;
    int64_t stride, out_stride;
    int budget, sinks, recent, row_bytes, words;
};

// Ascending order of the keys is ascending order of the weights: NaN lowest,
// -0 as 0; the largest key is kept for protected slots.
__device__ __forceinline__ unsigned mass_key(float x)
{
    if (x != x) return 0;
    const unsigned u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned slot_key(const EvictParams &p, const float *mass, const int32_t *pos, int j, long long top)
{
    const long long at = pos ? pos[j] : j;
    return at < p.sinks || at > top - p.recent ? 0xffffffffu : mass_key(mass[j]);
}

// Exclusive prefix of `x` over the block; *all gets the sum.
__device__ __forceinline__ int block_prefix(int x, int *sh, int *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int s = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        sh[lane] = s;
    }
    __syncthreads();
    *all = sh[31];
    return upto - x + (warp ? sh[warp - 1] : 0);
}

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const EvictParams p)
{
    extern __shared__ unsigned words[];  // kept bits, then prefix counts
    __shared__ unsigned hist[256];
    __shared__ int sh[32];
    __shared__ int tops[32];
    __shared__ unsigned found[2];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int64_t item = static_cast<int64_t>(b) * p.c.kv_heads + h;
    const float *mass = p.mass + item * p.stride;
    const int32_t *pos = p.pos ? p.pos + item * p.stride : nullptr;
    int32_t *src = p.slot_src + item * p.budget;
    const int n = p.lens[b];
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
    const bool bad = n < 0 || n > cap || n > p.stride;
    if (h == 0) {
        int any = bad;
        const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
        if (p.row_status) {
            for (int g = tid; !bad && n > p.budget && g <= (n - 1) >> p.c.page_shift; g += EV_THREADS)
                any |= page_of(p.c, table, g << p.c.page_shift) < 0;
            any = __syncthreads_or(any);
            if (tid == 0) p.row_status[b] = any ? KV_STATUS_BAD : 0;
        }
        if (tid == 0) p.new_lens[b] = bad || n < p.budget ? n : p.budget;
    }
    const int m = bad ? 0 : n < p.budget ? n : p.budget;
    if (bad || n <= p.budget) {  // nothing moves
        for (int i = tid; i < p.budget; i += EV_THREADS) {
            src[i] = i < m ? i : -1;
            if (i < m) {
                p.mass_out[item * p.out_stride + i] = mass[i];
                if (p.pos_out) p.pos_out[item * p.out_stride + i] = pos ? pos[i] : i;
            }
        }
        return;
    }
    int top = pos ? -1 : n - 1;
    if (pos) {
        for (int j = tid; j < n; j += EV_THREADS) top = max(top, pos[j]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[tid >> 5] = top;
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, tops[lane]);
    }
    // the key of the m-th largest, digit by digit; `want` of its equals stay
    unsigned prefix = 0;
    int want = m;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += EV_THREADS) {
            const unsigned key = slot_key(p, mass, pos, j, top);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[key >> shift & 255u], 1u);
        }
        __syncthreads();
        const int x = tid < 256 ? static_cast<int>(hist[255 - tid]) : 0;
        int all;
        const int before = block_prefix(x, sh, &all);  // of larger digits
        if (tid < 256 && before < want && want <= before + x) {
            found[0] = 255 - tid;
            found[1] = want - before;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want = static_cast<int>(found[1]);
        __syncthreads();
    }
    // kept bits: larger keys, and the first `want` equals
    const int nw = (n + 31) >> 5;
    unsigned *kept = words, *count = words + p.words;
    for (int w = tid >> 5; w < nw; w += EV_THREADS / 32) {
        const int j = 32 * w + lane;
        const unsigned key = j < n ? slot_key(p, mass, pos, j, top) : 0;
        const unsigned gt = __ballot_sync(0xffffffffu, j < n && key > prefix);
        const unsigned eq = __ballot_sync(0xffffffffu, j < n && key == prefix);
        if (lane == 0) {
            kept[w] = gt;
            count[w] = eq;
        }
    }
    __syncthreads();
    int run = 0;
    for (int w0 = 0; w0 < nw; w0 += EV_THREADS) {
        const int w = w0 + tid;
        unsigned eq = w < nw ? count[w] : 0;
        int all;
        const int before = run + block_prefix(__popc(eq), sh, &all);
        if (w < nw) {
            for (int left = want - before; eq && left > 0; --left) {
                kept[w] |= eq & -eq;
                eq &= eq - 1;
            }
        }
        run += all;
    }
    __syncthreads();
    // prefix counts: holes in the words below m, movers in those above
    const int wm = m >> 5;
    const unsigned low = (1u << (m & 31)) - 1u;
    int holes = 0, movers = 0;
    for (int w0 = 0; w0 < nw; w0 += EV_THREADS) {
        const int w = w0 + tid;
        const unsigned k = w < nw ? kept[w] : 0;
        const int hole = w >= nw || w > wm ? 0 : w < wm ? __popc(~k) : __popc(~k & low);
        const int mover = w >= nw || w < wm ? 0 : w > wm ? __popc(k) : __popc(k & ~low);
        int all;
        const int hb = holes + block_prefix(hole, sh, &all);
        holes += all;
        const int mb = movers + block_prefix(mover, sh, &all);
        movers += all;
        if (w < nw) count[w] = w <= wm ? hb : mb;
    }
    __syncthreads();
    const int first_movers = wm < nw ? __popc(kept[wm] & ~low) : 0;
    for (int i = tid; i < m; i += EV_THREADS) {
        const unsigned k = kept[i >> 5], bit = 1u << (i & 31);
        int s = i;
        if (!(k & bit)) {
            int rank = static_cast<int>(count[i >> 5]) + __popc(~k & (bit - 1u));
            unsigned from;
            int w;
            if (rank < first_movers) {
                w = wm;
                from = kept[wm] & ~low;
            } else {
                int a = wm + 1, z = nw - 1;  // the last word whose count is <= rank
                while (a < z) {
                    const int mid = (a + z + 1) >> 1;
                    if (static_cast<int>(count[mid]) <= rank)
                        a = mid;
                    else
                        z = mid - 1;
                }
                w = a;
                from = kept[w];
                rank -= static_cast<int>(count[w]);
            }
            for (; rank > 0; --rank) from &= from - 1;
            s = 32 * w + __ffs(from) - 1;
        }
        src[i] = s;
        if (s != i || p.mass_out != p.mass) p.mass_out[item * p.out_stride + i] = mass[s];
        if (p.pos_out && (s != i || p.pos_out != p.pos)) p.pos_out[item * p.out_stride + i] = pos ? pos[s] : s;
    }
    for (int i = m + tid; i < p.budget; i += EV_THREADS) src[i] = -1;
}

__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p)
{
    const int h = blockIdx.y % p.c.kv_heads, b = blockIdx.y / p.c.kv_heads;
    const int32_t *table = p.c.table + static_cast<int64_t>(b) * p.c.max_pages;
    const int32_t *src = p.slot_src + static_cast<int64_t>(blockIdx.y) * p.budget;
    const int per = p.row_bytes >> 4, lanes = 2 * per;  // 16-byte pieces of a row, of K and V
    for (int x = threadIdx.x; x < EV_MOVE_SLOTS * lanes; x += blockDim.x) {
        const int i = blockIdx.x * EV_MOVE_SLOTS + x / lanes, e = x % lanes;
        if (i >= p.budget) break;
        const int s = src[i];
        if (s < 0 || s == i) continue;
        const int from = page_of(p.c, table, s), to = page_of(p.c, table, i);
        if (from < 0 || to < 0) continue;
        const PoolView &pool = e < per ? p.c.k : p.c.v;
        const int o = (e < per ? e : e - per) << 4;
        *reinterpret_cast<uint4 *>(const_cast<char *>(row_ptr(p.c, pool, to, i, h)) + o) =
            *reinterpret_cast<const uint4 *>(row_ptr(p.c, pool, from, s, h) + o);
    }
}

cudaError_t launch_evict(const EvictLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    EvictParams p{};
    p.c = paged_view(k);
    p.lens = L.lens;
    p.pos = L.pos;
    p.mass = L.mass;
    p.mass_out = L.mass_out;
    p.pos_out = L.pos_out;
    p.new_lens = L.new_lens;
    p.slot_src = L.slot_src;
    p.row_status = k.row_status;
    p.stride = L.mass_stride;
    p.out_stride = L.out_stride;
    p.budget = L.budget;
    p.sinks = L.sinks;
    p.recent = L.recent;
    p.row_bytes = k.cache.head_dim * (k.cache.dtype == SPV_E4M3 ? 1 : 2);
    const int64_t cap = static_cast<int64_t>(k.max_pages) * k.cache.page_size;
    p.words = static_cast<int>(((cap < L.mass_stride ? cap : L.mass_stride) + 31) / 32);
    const int smem = p.words * 2 * static_cast<int>(sizeof(unsigned));
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    evict_select_kernel<<<dim3(k.cache.kv_heads, k.B), EV_THREADS, smem, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    evict_move_kernel<<<dim3((L.budget + EV_MOVE_SLOTS - 1) / EV_MOVE_SLOTS, k.B * k.cache.kv_heads), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace spv
