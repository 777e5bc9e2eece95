// spv_kv_api.cu -- the C entry points of the calls around the verify step
// (rotary positions, paged attention, attention mass, eviction): argument
// checks on the host and dispatch to the kernels.
#include "spv.h"
#include "spv_internal.h"

#include <atomic>
#include <cmath>
#include <cstdint>

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
spv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SPV_OK : SPV_ERR_CUDA; }
int elem_bytes(spv_dtype d) { return d == SPV_E4M3 ? 1 : 2; }

// The cache struct and the page table.
spv_status check_cache(const spv_kv_cache *c, const int32_t *page_table, int max_pages)
{
    if (!c || !c->k || !c->v || !page_table) return SPV_ERR_INVALID_ARG;
    if (c->dtype != SPV_BF16 && c->dtype != SPV_F16 && c->dtype != SPV_E4M3) return SPV_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->kv_heads < 1 || c->head_dim < 1 || max_pages < 1) return SPV_ERR_INVALID_ARG;
    if (c->page_size < 1 || (c->page_size & (c->page_size - 1)) != 0) return SPV_ERR_INVALID_ARG;
    if (c->head_dim % 8 != 0 || c->kv_heads > 1024) return SPV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * c->page_size > (1ll << 30)) return SPV_ERR_UNSUPPORTED;  // slots fit an int
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SPV_ERR_INVALID_ARG;
    const int e = elem_bytes(c->dtype);
    if (c->head_dim * e % 16 != 0) return SPV_ERR_UNSUPPORTED;
    const int64_t strides[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                                c->v_page_stride, c->v_slot_stride, c->v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s * e % 16 != 0) return SPV_ERR_INVALID_ARG;
    return SPV_OK;
}

// What the three calls on q share.
spv_status check_tokens(const void *q, spv_dtype dtype, int B, int T, int q_heads, const spv_kv_cache *c,
                        const int32_t *page_table, int max_pages, const int32_t *ctx_lens)
{
    if (!q || !ctx_lens || (dtype != SPV_BF16 && dtype != SPV_F16)) return SPV_ERR_INVALID_ARG;
    const spv_status st = check_cache(c, page_table, max_pages);
    if (st != SPV_OK) return st;
    if (c->dtype != SPV_E4M3 && c->dtype != dtype) return SPV_ERR_INVALID_ARG;
    if (c->dtype != SPV_E4M3 && (c->k_scale || c->v_scale)) return SPV_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || q_heads < 1 || q_heads % c->kv_heads != 0) return SPV_ERR_INVALID_ARG;
    if (!aligned(q, 16)) return SPV_ERR_INVALID_ARG;
    return SPV_OK;
}

// The shapes that the attention kernels are built for.
spv_status check_attention_sizes(int B, int T, int q_heads, int kv_heads, int head_dim)
{
    if (T > SPV_MAX_NEW_TOKENS || q_heads / kv_heads > SPV_MAX_GROUP || B > 65535) return SPV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return SPV_ERR_UNSUPPORTED;
    return SPV_OK;
}

spv::KvLaunch kv_launch(const spv_kv_cache *cache, const int32_t *page_table, int max_pages, int B, int T, int q_heads,
                        spv_dtype dtype, const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *parent,
                        float scale, int32_t *row_status)
{
    return spv::KvLaunch{*cache, page_table, max_pages, B, T, q_heads, dtype, ctx_lens, new_lens, parent, scale,
                         row_status};
}

// The checks and the launch that the two rotary calls share.
spv_status rope_launch(spv::RopeLaunch *out, const void *q, const void *k, const void *v, spv_dtype dtype,
                       const int64_t *strides, int B, int T, int q_heads, const uint64_t *freqs, int rotary_dim,
                       int interleaved, float mscale, const int32_t *positions, const int32_t *ctx_lens,
                       const int32_t *new_lens, const int32_t *page_table, int max_pages, const spv_kv_cache *cache,
                       int32_t *slot_pos, int64_t pos_stride, void *q_out, int32_t *row_status)
{
    const spv_status st = check_tokens(q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens);
    if (st != SPV_OK) return st;
    const int D = cache->head_dim, kv_heads = cache->kv_heads;
    if (!k || !v || !q_out || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16)) return SPV_ERR_INVALID_ARG;
    if (D > 512) return SPV_ERR_UNSUPPORTED;
    if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 2 != 0 || (rotary_dim > 0 && !freqs)) return SPV_ERR_INVALID_ARG;
    if (!std::isfinite(mscale)) return SPV_ERR_INVALID_ARG;
    if (slot_pos && pos_stride < 1) return SPV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(B) * T > 0x7fffffffll) return SPV_ERR_UNSUPPORTED;
    spv::RopeLaunch &L = *out;
    const int64_t qd = static_cast<int64_t>(q_heads) * D, kd = static_cast<int64_t>(kv_heads) * D;
    const int64_t packed[6] = {T * qd, qd, T * kd, kd, T * kd, kd};
    for (int i = 0; i < 6; ++i) {
        L.strides[i] = strides ? strides[i] : packed[i];
        if (L.strides[i] < 0 || L.strides[i] % 8 != 0) return SPV_ERR_INVALID_ARG;
    }
    if (q_out == q && (L.strides[0] != packed[0] || L.strides[1] != packed[1])) return SPV_ERR_INVALID_ARG;
    L.kv = kv_launch(cache, page_table, max_pages, B, T, q_heads, dtype, ctx_lens, new_lens, nullptr, 0.0f, row_status);
    L.q = q;
    L.k = k;
    L.v = v;
    L.freqs = freqs;
    L.rotary_dim = rotary_dim;
    L.interleaved = interleaved != 0;
    L.mscale = mscale;
    L.positions = positions;
    L.slot_pos = slot_pos;
    L.pos_stride = pos_stride;
    L.q_out = q_out;
    return SPV_OK;
}

// The scores of a call; `tree`: its new tokens are one.
spv_status check_scores(const spv_scores *s, bool tree)
{
    if (!s || !(s->cap >= 0.0f) || std::isinf(s->cap) || s->window < 0) return SPV_ERR_INVALID_ARG;
    if (s->cap > 0.0f && s->cap < 1e-30f) return SPV_ERR_INVALID_ARG;  // 2 / cap has to be a number
    if (s->last && tree) return SPV_ERR_INVALID_ARG;
    if (s->slot_pos && s->pos_stride < 1) return SPV_ERR_INVALID_ARG;
    return SPV_OK;
}

// The checks and the launch that the paged attention calls share.
spv_status attention_launch(spv::AttentionLaunch *out_launch, const void *q, spv_dtype dtype, int B, int T, int q_heads,
                            const spv_kv_cache *cache, const int32_t *page_table, int max_pages, const int32_t *ctx_lens,
                            const int32_t *new_lens, const int32_t *parent, float scale, void *out, float *lse,
                            int32_t *row_status, void *workspace, size_t workspace_bytes)
{
    spv_status st = check_tokens(q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens);
    if (st != SPV_OK) return st;
    st = check_attention_sizes(B, T, q_heads, cache->kv_heads, cache->head_dim);
    if (st != SPV_OK) return st;
    if (!out || !aligned(out, 16) || !workspace || !aligned(workspace, 256) || !std::isfinite(scale))
        return SPV_ERR_INVALID_ARG;
    if (workspace_bytes < spv::attention_ws_bytes(B, T, q_heads, cache->kv_heads, cache->head_dim))
        return SPV_ERR_INVALID_ARG;
    spv::AttentionLaunch &L = *out_launch;
    L.kv = kv_launch(cache, page_table, max_pages, B, T, q_heads, dtype, ctx_lens, new_lens, parent, scale, row_status);
    L.q = q;
    L.out = out;
    L.lse = lse;
    L.ws = workspace;
    return SPV_OK;
}

// The same of the weights of cached keys.
spv_status mass_launch(spv::MassLaunch *out, const void *q, spv_dtype dtype, int B, int T, int q_heads, const float *lse,
                       const spv_kv_cache *cache, const int32_t *page_table, int max_pages, const int32_t *ctx_lens,
                       const int32_t *new_lens, const int32_t *parent, float scale, const int32_t *accept_count,
                       const int32_t *nodes, float decay, const float *mass_in, float *mass_out, int64_t mass_stride,
                       int32_t *row_status)
{
    spv_status st = check_tokens(q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens);
    if (st != SPV_OK) return st;
    st = check_attention_sizes(B, T, q_heads, cache->kv_heads, cache->head_dim);
    if (st != SPV_OK) return st;
    if (!lse || !accept_count || !mass_out || mass_stride < 1) return SPV_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(decay)) return SPV_ERR_INVALID_ARG;
    spv::MassLaunch &L = *out;
    L.kv = kv_launch(cache, page_table, max_pages, B, T, q_heads, dtype, ctx_lens, new_lens, parent, scale, row_status);
    L.q = q;
    L.lse = lse;
    L.accept_count = accept_count;
    L.nodes = nodes;
    L.decay = decay;
    L.mass_in = mass_in;
    L.mass_out = mass_out;
    L.mass_stride = mass_stride;
    return SPV_OK;
}

// The shapes that the prompt kernels are built for.
spv_status check_prompt_sizes(int B, int T, int q_heads, int kv_heads, int head_dim)
{
    if (q_heads / kv_heads > SPV_MAX_GROUP || B > 65535) return SPV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(T) * (q_heads / kv_heads) > (1ll << 24)) return SPV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return SPV_ERR_UNSUPPORTED;
    return SPV_OK;
}

std::atomic<int64_t> give_up_at{-1};  // block << 32 | item

}  // namespace

namespace spv {
GiveUp give_up()
{
    const int64_t x = give_up_at.load(std::memory_order_relaxed);
    return GiveUp{static_cast<int>(x >> 32), static_cast<int>(x & 0x7fffffff)};
}
}  // namespace spv

extern "C" {

spv_status spv_selftest_give_up(int block, int item)
{
    if (block < -1 || item < 0) return SPV_ERR_INVALID_ARG;
    give_up_at.store(block < 0 ? -1 : static_cast<int64_t>(block) << 32 | item, std::memory_order_relaxed);
    return SPV_OK;
}

spv_status spv_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double low, double high,
                                double original_len, uint64_t *out)
{
    if (!out || rotary_dim < 2 || rotary_dim > 1024 || rotary_dim % 2 != 0) return SPV_ERR_INVALID_ARG;
    if (!(base > 0.0) || std::isinf(base) || !(factor > 0.0) || std::isinf(factor)) return SPV_ERR_INVALID_ARG;
    if (scaling < SPV_ROPE_PLAIN || scaling > SPV_ROPE_BY_PARTS) return SPV_ERR_INVALID_ARG;
    if (scaling == SPV_ROPE_BASE && rotary_dim == 2) return SPV_ERR_INVALID_ARG;
    if (scaling == SPV_ROPE_BY_PARTS &&
        (!(low < high) || std::isinf(low) || std::isinf(high) || !(original_len > 0.0) || std::isinf(original_len)))
        return SPV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    if (scaling == SPV_ROPE_BASE) base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == SPV_ROPE_LINEAR) f /= factor;
        if (scaling == SPV_ROPE_BY_PARTS) {
            double g = (original_len * f / two_pi - low) / (high - low);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = g * f + (1.0 - g) * f / factor;
        }
        double turns = f / two_pi;
        turns -= std::floor(turns);                          // whole turns change nothing
        const double scaled = std::nearbyint(std::ldexp(turns, 64));
        out[i] = scaled >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(scaled);
    }
    return SPV_OK;
}

spv_status spv_rope_append(const void *q, const void *k, const void *v, spv_dtype dtype, const int64_t *strides, int B,
                           int T, int q_heads, const uint64_t *freqs, int rotary_dim, int interleaved, float mscale,
                           const int32_t *positions, const int32_t *ctx_lens, const int32_t *new_lens,
                           const int32_t *page_table, int max_pages, const spv_kv_cache *cache, int32_t *slot_pos,
                           int64_t pos_stride, void *q_out, int32_t *row_status, void *stream)
{
    spv::RopeLaunch L{};
    const spv_status st = rope_launch(&L, q, k, v, dtype, strides, B, T, q_heads, freqs, rotary_dim, interleaved, mscale,
                                      positions, ctx_lens, new_lens, page_table, max_pages, cache, slot_pos, pos_stride, q_out,
                                      row_status);
    if (st != SPV_OK) return st;
    return cuda_status(spv::launch_rope(L, static_cast<cudaStream_t>(stream)));
}

spv_status spv_norm_rope_append(const void *q, const void *k, const void *v, spv_dtype dtype, const int64_t *strides,
                                int B, int T, int q_heads, const float *q_weight, const float *k_weight, float eps,
                                const uint64_t *freqs, const int32_t *axes, int num_axes, int rotary_dim,
                                int interleaved, float mscale, const int32_t *positions, const int32_t *ctx_lens,
                                const int32_t *new_lens, const int32_t *page_table, int max_pages,
                                const spv_kv_cache *cache, int32_t *slot_pos, int64_t pos_stride, void *q_out,
                                int32_t *row_status, void *stream)
{
    spv::NormRopeLaunch L{};
    const spv_status st = rope_launch(&L.rope, q, k, v, dtype, strides, B, T, q_heads, freqs, rotary_dim, interleaved, mscale,
                                      positions, ctx_lens, new_lens, page_table, max_pages, cache, slot_pos, pos_stride, q_out,
                                      row_status);
    if (st != SPV_OK) return st;
    if (cache->head_dim > 256) return SPV_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || std::isinf(eps) || num_axes < 1 || num_axes > 8) return SPV_ERR_INVALID_ARG;
    if (num_axes > 1 && !positions) return SPV_ERR_INVALID_ARG;
    L.q_weight = q_weight;
    L.k_weight = k_weight;
    L.eps = eps;
    L.axes = axes;
    L.num_axes = num_axes;
    return cuda_status(spv::launch_norm_rope(L, static_cast<cudaStream_t>(stream)));
}

size_t spv_attention_workspace_bytes(int B, int T, int q_heads, int kv_heads, int head_dim)
{
    if (B < 1 || T < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
    if (check_attention_sizes(B, T, q_heads, kv_heads, head_dim) != SPV_OK) return 0;
    return spv::attention_ws_bytes(B, T, q_heads, kv_heads, head_dim);
}

spv_status spv_paged_attention(const void *q, spv_dtype dtype, int B, int T, int q_heads, const spv_kv_cache *cache,
                               const int32_t *page_table, int max_pages, const int32_t *ctx_lens,
                               const int32_t *new_lens, const int32_t *parent, float scale, void *out, float *lse,
                               int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream)
{
    spv::AttentionLaunch L{};
    const spv_status st = attention_launch(&L, q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens, new_lens, parent,
                                           scale, out, lse, row_status, workspace, workspace_bytes);
    if (st != SPV_OK) return st;
    return cuda_status(spv::launch_attention(L, static_cast<cudaStream_t>(stream)));
}

spv_status spv_paged_attention_scored(const void *q, spv_dtype dtype, int B, int T, int q_heads,
                                      const spv_kv_cache *cache, const int32_t *page_table, int max_pages,
                                      const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *parent,
                                      float scale, const spv_scores *scores, void *out, float *lse,
                                      int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream)
{
    spv::AttentionLaunch L{};
    spv_status st = attention_launch(&L, q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens, new_lens, parent,
                                     scale, out, lse, row_status, workspace, workspace_bytes);
    if (st != SPV_OK) return st;
    st = check_scores(scores, parent != nullptr);
    if (st != SPV_OK) return st;
    L.scores = *scores;
    return cuda_status(spv::launch_attention_scored(L, static_cast<cudaStream_t>(stream)));
}

size_t spv_prompt_workspace_bytes(int B, int T, int q_heads, int kv_heads, int head_dim)
{
    if (B < 1 || T < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return 0;
    if (check_prompt_sizes(B, T, q_heads, kv_heads, head_dim) != SPV_OK) return 0;
    return spv::prompt_ws_bytes(B, T, q_heads, kv_heads, head_dim);
}

spv_status spv_prompt_attention(const void *q, spv_dtype dtype, int B, int T, int q_heads, const spv_kv_cache *cache,
                                const int32_t *page_table, int max_pages, const int32_t *ctx_lens,
                                const int32_t *new_lens, float scale, const spv_scores *scores, void *out, float *lse,
                                int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream)
{
    spv_status st = check_tokens(q, dtype, B, T, q_heads, cache, page_table, max_pages, ctx_lens);
    if (st != SPV_OK) return st;
    st = check_prompt_sizes(B, T, q_heads, cache->kv_heads, cache->head_dim);
    if (st != SPV_OK) return st;
    if (!out || !aligned(out, 16) || !workspace || !aligned(workspace, 256) || !std::isfinite(scale))
        return SPV_ERR_INVALID_ARG;
    if (workspace_bytes < spv::prompt_ws_bytes(B, T, q_heads, cache->kv_heads, cache->head_dim)) return SPV_ERR_INVALID_ARG;
    spv::AttentionLaunch L{};
    if (scores) {
        st = check_scores(scores, false);
        if (st != SPV_OK) return st;
        L.scores = *scores;
    }
    L.kv = kv_launch(cache, page_table, max_pages, B, T, q_heads, dtype, ctx_lens, new_lens, nullptr, scale, row_status);
    L.q = q;
    L.out = out;
    L.lse = lse;
    L.ws = workspace;
    return cuda_status(spv::launch_prompt(L, static_cast<cudaStream_t>(stream)));
}

spv_status spv_attention_mass(const void *q, spv_dtype dtype, int B, int T, int q_heads, const float *lse,
                              const spv_kv_cache *cache, const int32_t *page_table, int max_pages,
                              const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *parent, float scale,
                              const int32_t *accept_count, const int32_t *nodes, float decay, const float *mass_in,
                              float *mass_out, int64_t mass_stride, int32_t *row_status, void *stream)
{
    spv::MassLaunch L{};
    const spv_status st = mass_launch(&L, q, dtype, B, T, q_heads, lse, cache, page_table, max_pages, ctx_lens, new_lens, parent,
                                      scale, accept_count, nodes, decay, mass_in, mass_out, mass_stride, row_status);
    if (st != SPV_OK) return st;
    return cuda_status(spv::launch_mass(L, static_cast<cudaStream_t>(stream)));
}

spv_status spv_attention_mass_scored(const void *q, spv_dtype dtype, int B, int T, int q_heads, const float *lse,
                                     const spv_kv_cache *cache, const int32_t *page_table, int max_pages,
                                     const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *parent,
                                     float scale, const spv_scores *scores, const int32_t *accept_count,
                                     const int32_t *nodes, float decay, const float *mass_in, float *mass_out,
                                     int64_t mass_stride, int32_t *row_status, void *stream)
{
    spv::MassLaunch L{};
    spv_status st = mass_launch(&L, q, dtype, B, T, q_heads, lse, cache, page_table, max_pages, ctx_lens, new_lens, parent, scale,
                                accept_count, nodes, decay, mass_in, mass_out, mass_stride, row_status);
    if (st != SPV_OK) return st;
    st = check_scores(scores, parent != nullptr);
    if (st != SPV_OK) return st;
    L.scores = *scores;
    return cuda_status(spv::launch_mass_scored(L, static_cast<cudaStream_t>(stream)));
}

spv_status spv_kv_evict(const spv_kv_cache *cache, const int32_t *page_table, int max_pages, int B,
                        const int32_t *lens, int budget, int sinks, int recent, const float *mass, const int32_t *pos,
                        int64_t mass_stride, float *mass_out, int32_t *pos_out, int64_t out_stride, int32_t *new_lens,
                        int32_t *slot_src, int32_t *row_status, void *stream)
{
    const spv_status st = check_cache(cache, page_table, max_pages);
    if (st != SPV_OK) return st;
    if (B < 1 || budget < 1 || sinks < 0 || recent < 0 || sinks > budget - recent) return SPV_ERR_INVALID_ARG;
    if (!lens || !mass || !mass_out || !new_lens || !slot_src || mass_stride < 1) return SPV_ERR_INVALID_ARG;
    if (out_stride < (budget < mass_stride ? budget : mass_stride)) return SPV_ERR_INVALID_ARG;
    if (mass_out == mass && out_stride != mass_stride) return SPV_ERR_INVALID_ARG;
    if (pos && pos_out == pos && out_stride != mass_stride) return SPV_ERR_INVALID_ARG;
    if (mass_stride > SPV_MAX_EVICT_SLOTS || budget > SPV_MAX_EVICT_SLOTS ||
        static_cast<int64_t>(B) * cache->kv_heads > 65535)
        return SPV_ERR_UNSUPPORTED;
    spv::EvictLaunch L{};
    L.kv = kv_launch(cache, page_table, max_pages, B, 0, 0, cache->dtype, nullptr, nullptr, nullptr, 0.0f, row_status);
    L.lens = lens;
    L.budget = budget;
    L.sinks = sinks;
    L.recent = recent;
    L.mass = mass;
    L.pos = pos;
    L.mass_stride = mass_stride;
    L.mass_out = mass_out;
    L.pos_out = pos_out;
    L.out_stride = out_stride;
    L.new_lens = new_lens;
    L.slot_src = slot_src;
    return cuda_status(spv::launch_evict(L, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
