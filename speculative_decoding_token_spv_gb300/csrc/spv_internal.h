// spv_internal.h -- host-side launch interface between spv_api.cu and the
// per-op kernel files.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "spv.h"

namespace spv {

// Workspace header: word 0 is the device error word (SPV_OK or
// SPV_ERR_TIMEOUT); sections start at multiples of 256 bytes.
constexpr size_t WS_HEADER = 256;
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int blocks_per_row(int V) { return (V + 1023) / 1024; }
inline int chunks_per_row(int V) { return (V + 8191) / 8192; }

struct ChainLaunch {
    const void *target, *draft;
    int dtype;  // 0 fp32, 1 bf16
    const int32_t *tokens;
    const float *r;
    const uint64_t *keys;
    int B, gamma, V;
    float T;
    int32_t *accept_count, *out_tokens;
    float *out_pq, *out_Z;
    int32_t *row_status;
    void *ws;
    bool tma;  // rows are 16-byte aligned and V * elem_bytes % 16 == 0
    // Optional speculation-cache lookup (null cache_ids: none).
    const int32_t *cache_ids;
    const int32_t *cache_fanout;  // host, gamma + 1 entries
    int32_t *cache_slot;
    // Top-k / top-p filter (spv_verify_chain_filtered only).
    int top_k;
    float top_p;
    // Saguaro sampling (spv_verify_chain_saguaro only): the cache lists are
    // the cached candidates whose draft probability was divided by sag_C.
    int sag;
    float sag_C;
};

struct TreeLaunch {
    const void *target, *draft;
    int dtype;
    const int32_t *parent, *tokens;
    const float *r;
    const uint64_t *keys;
    int B, N, V;
    float T;
    int32_t *accept_count, *out_tokens, *out_nodes, *row_status;
    void *ws;
    bool tma;
};

struct FanoutLaunch {
    const void *draft;
    int dtype;
    const int32_t *exclude;
    int F[64];
    int off[65];
    int Fmax;
    int B, K1, V;
    int32_t *out_ids, *row_status;
    void *ws;
    bool tma;
};

// The arguments spv_verify_chain shares with spv_verify_chain_noalloc.
struct ChainArgs {
    const void *target_logits, *draft_logits;
    spv_dtype dtype;
    const int32_t *draft_tokens;
    const float *r;
    const uint64_t *sample_keys;
    int B, gamma, V;
    float temperature;
    int32_t *accept_count, *out_tokens;
    float *out_pq, *out_resid_norm;
    int32_t *row_status;
};

// Host checks of those arguments (pointers, dtype, sizes, temperature):
// SPV_OK or the status the call returns before any launch.
spv_status check_chain_args(const ChainArgs &a);
// Scratch bytes the call needs (greedy layout at T == 0).
size_t chain_call_ws_bytes(const ChainArgs &a);
// The launch description of a checked call on scratch `ws` (no cache lookup,
// no Saguaro weights).
ChainLaunch chain_launch(const ChainArgs &a, void *ws);
// Enqueues the call: the greedy kernels at T == 0, else the chain kernels.
cudaError_t launch_chain_or_greedy(const ChainLaunch &L, cudaStream_t st);

// The calls around the verify step (checked arguments, see spv.h).
struct KvLaunch {
    spv_kv_cache cache;
    const int32_t *page_table;
    int max_pages;
    int B, T, q_heads;
    spv_dtype dtype;
    const int32_t *ctx_lens, *new_lens, *parent;
    float scale;
    int32_t *row_status;
};
struct RopeLaunch {
    KvLaunch kv;
    const void *q, *k, *v;
    int64_t strides[6];
    const uint64_t *freqs;
    int rotary_dim, interleaved;
    float mscale;
    const int32_t *positions;
    int32_t *slot_pos;
    int64_t pos_stride;
    void *q_out;
};
struct NormRopeLaunch {
    RopeLaunch rope;
    const float *q_weight, *k_weight;
    float eps;
    const int32_t *axes;
    int num_axes;
};
struct AttentionLaunch {
    KvLaunch kv;
    const void *q;
    void *out;
    float *lse;
    void *ws;
    spv_scores scores;  // of the calls that take them
};
struct MassLaunch {
    KvLaunch kv;
    const void *q;
    const float *lse;
    const int32_t *accept_count, *nodes;
    float decay;
    const float *mass_in;
    float *mass_out;
    int64_t mass_stride;
    spv_scores scores;  // of the call that takes them
};
struct EvictLaunch {
    KvLaunch kv;
    const int32_t *lens;
    int budget, sinks, recent;
    const float *mass;
    const int32_t *pos;
    int64_t mass_stride;
    float *mass_out;
    int32_t *pos_out;
    int64_t out_stride;
    int32_t *new_lens, *slot_src;
};
// Self-test: in block `block` of an attention or mass kernel a wait gives up at
// its item `item` (block -1: nowhere).
struct GiveUp {
    int block, item;
};
GiveUp give_up();

inline int log2_of(int pow2)
{
    int s = 0;
    while ((1 << s) < pow2) ++s;
    return s;
}

size_t chain_ws_bytes(int B, int gamma, int V);
size_t greedy_ws_bytes(int B, int gamma, int V);
size_t fanout_ws_bytes(int B, int K1, int V, int Fmax);
size_t filtered_ws_bytes(int B, int gamma, int V);
size_t tree_ws_bytes(int B, int N, int V);

cudaError_t launch_chain(const ChainLaunch &L, cudaStream_t st);
cudaError_t launch_greedy(const ChainLaunch &L, cudaStream_t st);
cudaError_t launch_fanout(const FanoutLaunch &L, cudaStream_t st);
cudaError_t launch_filtered(const ChainLaunch &L, cudaStream_t st);
cudaError_t launch_selftest_wait(void *ws, unsigned polls, cudaStream_t st);
cudaError_t launch_tree(const TreeLaunch &L, cudaStream_t st);

size_t attention_ws_bytes(int B, int T, int q_heads, int kv_heads, int head_dim);
struct PagedView paged_view(const KvLaunch &L);
cudaError_t launch_rope(const RopeLaunch &L, cudaStream_t st);
cudaError_t launch_norm_rope(const NormRopeLaunch &L, cudaStream_t st);
cudaError_t launch_attention(const AttentionLaunch &L, cudaStream_t st);
cudaError_t launch_attention_scored(const AttentionLaunch &L, cudaStream_t st);
cudaError_t launch_prompt(const AttentionLaunch &L, cudaStream_t st);
size_t prompt_ws_bytes(int B, int T, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_mass(const MassLaunch &L, cudaStream_t st);
cudaError_t launch_mass_scored(const MassLaunch &L, cudaStream_t st);
cudaError_t launch_evict(const EvictLaunch &L, cudaStream_t st);

}  // namespace spv
