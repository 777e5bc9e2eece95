// spv_attention.cu -- spv_paged_attention: its workspace, and which kernel takes
// a call.
#include "spv_attention_warps.cuh"

namespace spv {

size_t attention_ws_bytes(int, int, int, int, int head_dim)
{
    const size_t few = static_cast<size_t>(ATT_MAX_BLOCKS) * 2 * ATT_MAX_ROWS * (head_dim + 2);
    const size_t many = attention_rows_part_floats(head_dim);
    return ATT_PARTS_AT + (few > many ? few : many) * sizeof(float);
}

cudaError_t launch_attention(const AttentionLaunch &L, cudaStream_t st)
{
    const KvLaunch &k = L.kv;
    AttParams p{};
    p.c = paged_view(k);
    p.group = k.q_heads / k.cache.kv_heads;
    p.w = Work{k.B, k.T, 1, ATT_KEYS, k.ctx_lens, k.new_lens, false};
    p.q = L.q;
    p.out = L.out;
    p.lse = L.lse;
    p.parent = k.parent;
    p.row_status = k.row_status;
    p.q_heads = k.q_heads;
    p.rows = k.T * p.group;
    p.scale_log2 = k.scale * LOG2E;
    p.give_up = give_up();
    char *ws = static_cast<char *>(L.ws);
    p.error = reinterpret_cast<unsigned *>(ws);
    p.split = reinterpret_cast<SplitItem *>(ws + WS_HEADER);
    p.parts = reinterpret_cast<float *>(ws + ATT_PARTS_AT);
    const bool eight = k.cache.dtype == SPV_E4M3;
    const int D = k.cache.head_dim;
    // Over 16 rows the 5th-generation tensor cores, for an e4m3 cache over 32: its rows pass through shared memory
    // twice there.  Two sequences of 131,001 keys, 8 key heads, D = 128, from cold caches: bf16 at 16 rows 194 us there
    // and 200 here, at 20 rows 194 and 362 (16 sequences of up to 4,000: 61 and 56, 62 and 77); e4m3 at 32 rows 194 and
    // 173 (71 and 56), at 40 rows 192 there and two passes here.
    if (p.rows > (eight ? 32 : 16) && D <= 128) return launch_attention_rows(p, k, st);
    if (k.dtype == SPV_BF16)
        return eight ? launch_types<__nv_bfloat16, __nv_fp8_e4m3>(p, D, st)
                     : launch_types<__nv_bfloat16, __nv_bfloat16>(p, D, st);
    return eight ? launch_types<__half, __nv_fp8_e4m3>(p, D, st) : launch_types<__half, __half>(p, D, st);
}

}  // namespace spv
