// spv_scored.cu -- spv_paged_attention_scored for few rows a key head, and the
// statuses of scored calls.
#include <algorithm>

#include "spv_attention_warps.cuh"

namespace spv {

// A sequence is bad if its lengths are, or a page that its new tokens may see is outside the pool.
__global__ void __launch_bounds__(128) scored_status_kernel(const PagedView c, const ScoredWork w, int32_t *row_status)
{
    __shared__ int lowest;
    const int b = blockIdx.x;
    if (threadIdx.x == 0) lowest = 0x7fffffff;
    chain_begin();
    __syncthreads();
    SeqLens s = seq_lens(w.ctx_lens, w.new_lens, b, w.T, c, w.idle);
    if (w.sc.slot_pos && !s.bad && s.ctx + s.fresh > w.sc.pos_stride) {
        s.bad = true;
        s.total = 0;
    }
    int from = w.sc.window > 0 && !w.sc.slot_pos ? s.ctx - w.sc.window + 1 : 0;
    if (w.sc.first && s.total > 0) {
        int least = 0x7fffffff;
        for (int t = threadIdx.x; t < s.fresh; t += 128) least = min(least, __ldg(w.sc.first + static_cast<int64_t>(b) * w.T + t));
        atomicMin(&lowest, least);
        __syncthreads();
        from = max(from, lowest);
    }
    from = max(0, min(from, s.total - 1));
    const int32_t *table = c.table + static_cast<int64_t>(b) * c.max_pages;
    int any = s.bad;
    for (int g = (from >> c.page_shift) + threadIdx.x; s.total > 0 && g <= (s.total - 1) >> c.page_shift; g += 128)
        any |= page_of(c, table, g << c.page_shift) < 0;
    any = __syncthreads_or(any);
    if (threadIdx.x == 0) row_status[b] = any ? KV_STATUS_BAD : 0;
}

cudaError_t launch_scored_status(const PagedView &c, const ScoredWork &w, int32_t *row_status, cudaStream_t st)
{
    return launch_chained(scored_status_kernel, dim3(w.B), 128, 0, st, c, w, row_status);
}

ScoredParams scored_params(const AttentionLaunch &L)
{
    const KvLaunch &k = L.kv;
    ScoredParams p{};
    p.c = paged_view(k);
    p.group = k.q_heads / k.cache.kv_heads;
    p.w = Work{k.B, k.T, 1, ATT_KEYS, k.ctx_lens, k.new_lens, false};
    p.q = L.q;
    p.out = L.out;
    p.lse = L.lse;
    p.parent = k.parent;
    p.q_heads = k.q_heads;
    p.rows = k.T * p.group;
    p.scale_log2 = k.scale * LOG2E;
    p.give_up = give_up();
    p.sc = scores_view(L.scores);
    char *ws = static_cast<char *>(L.ws);
    p.error = reinterpret_cast<unsigned *>(ws);
    p.split = reinterpret_cast<SplitItem *>(ws + WS_HEADER);
    p.parts = reinterpret_cast<float *>(ws + ATT_PARTS_AT);
    return p;
}

cudaError_t launch_attention_scored(const AttentionLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    ScoredParams p = scored_params(L);
    const bool eight = k.cache.dtype == SPV_E4M3;
    const int D = k.cache.head_dim;
    if (k.row_status) {
        const cudaError_t e = launch_scored_status(p.c, work_of(p), k.row_status, st);
        if (e != cudaSuccess) return e;
    }
    // Many rows a key head: in tiles.  Few rows too where a 16-bit cache may be large: at D = 256 from 64 MB on (1 token, 2 rows,
    // 8 key heads: 8 x 500 slots 24.9 us there and 24.1 here, 1 x 30,000 65.7 and 72.0, 64 x 2,000 193 and 223), at D = 128 from
    // 1 GB on (64 x 2,000 124 and 121, 64 x 6,000 266 and 304), at D = 64 never (64 x 6,000 197 and 165); e4m3, whose rows pass
    // through shared memory twice there, never (64 x 2,000 of 128: 169 and 90).  How long the caches are the host does not know:
    // what the page table has room for counts, or the window.
    int64_t slots = static_cast<int64_t>(k.max_pages) << log2_of(k.cache.page_size);
    if (p.sc.window > 0 && !p.sc.slot_pos) slots = std::min<int64_t>(slots, static_cast<int64_t>(p.sc.window) + k.T);
    const double bytes = 4.0 * D * k.cache.kv_heads * k.B * static_cast<double>(slots);
    const bool large = !eight && (D == 256 ? bytes >= 64e6 : D == 128 && bytes >= 1e9);
    if (large || p.rows > (eight && D <= 128 ? 32 : 16)) return launch_tiles(p, k, false, st);
    if (k.dtype == SPV_BF16)
        return eight ? launch_types<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                     : launch_types<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_types<__half, __nv_fp8_e4m3>(p, D, st) : launch_types<__half, __half>(p, D, st);
}

}  // namespace spv
