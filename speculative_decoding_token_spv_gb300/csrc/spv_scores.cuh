// spv_scores.cuh -- scores and masks of attention that is not plain (spv_scores
// of spv.h) as the kernels see them.  Scores are in powers of two throughout: a
// score s stands for 2^s.
#pragma once

#include "spv_mma.cuh"

namespace spv {

struct ScoresView {
    float cap2, cap_in, cap_inv;  // cap log2 e (0: none), 2 / cap, 1 / cap2
    const float *slopes;
    int window;
    const int32_t *first, *last, *slot_pos;
    int64_t pos_stride;
};
inline ScoresView scores_view(const spv_scores &s)
{
    ScoresView v{};
    v.cap2 = s.cap > 0.0f ? s.cap * LOG2E : 0.0f;
    v.cap_in = s.cap > 0.0f ? 2.0f / s.cap : 0.0f;
    v.cap_inv = s.cap > 0.0f ? 1.0f / v.cap2 : 0.0f;
    v.slopes = s.slopes;
    v.window = s.window;
    v.first = s.first;
    v.last = s.last;
    v.slot_pos = s.slot_pos;
    v.pos_stride = s.pos_stride;
    return v;
}
// Whether positions come from memory: needed for a bias or a window over moved slots.
__host__ __device__ __forceinline__ bool moved_slots(const ScoresView &v) { return v.slot_pos && (v.slopes || v.window > 0); }

// cap tanh(x / cap), x and the result in powers of two.  Where |x| stays below
// CAP_SMALL of the cap: x times a polynomial in (x / cap)^2 (tanh(u) / u
// interpolated at the Chebyshev nodes of u^2 in [0, CAP_SMALL^2], 1.2e-7 off),
// so that a cap far above the scores changes nothing in them.  Beyond: cap - 2
// cap / (1 + e^(2 x / cap)), 2^-22 cap off, which is 2^-21 of a result there.
constexpr float CAP_SMALL = 0.625f;
constexpr float CAP_0 = 0.999999896f, CAP_1 = -0.333319736f, CAP_2 = 0.133047715f, CAP_3 = -0.0518318566f, CAP_4 = 0.0150636728f;
__device__ __forceinline__ float capped_small(const ScoresView &v, float x)
{
    const float u = x * v.cap_inv, w = u * u;
    return x * fmaf(w, fmaf(w, fmaf(w, fmaf(w, CAP_4, CAP_3), CAP_2), CAP_1), CAP_0);
}
__device__ __forceinline__ float capped_large(const ScoresView &v, float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp2(x * v.cap_in)));
    return fmaf(-2.0f * v.cap2, r, v.cap2);
}
// N values of each lane; one way for the whole warp where all of them are small.
template <int N> __device__ __forceinline__ void cap_all(const ScoresView &v, float (&x)[N])
{
    float top = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
    const float edge = CAP_SMALL * v.cap2;
    if (__any_sync(0xffffffffu, top >= edge)) {  // NaN is not above; the polynomial keeps it
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fabsf(x[i]) >= edge ? capped_large(v, x[i]) : capped_small(v, x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = capped_small(v, x[i]);
    }
}

__device__ __forceinline__ float2 unpair(unsigned long long x)
{
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}
// x f P((x f / cap)^2) of pairs, P of N coefficients.
template <int M, int N> __device__ __forceinline__ void cap_polynomial(const ScoresView &v, unsigned long long (&x)[M], float f, const float (&c)[N])
{
    const float u = f * v.cap_inv;
    const unsigned long long u2 = pack2(u, u);
    unsigned long long k[N];
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = pack2(c[i] * f, c[i] * f);
    constexpr int TOGETHER = M < 8 ? M : 8;  // pairs whose chains of operations go side by side
#pragma unroll
    for (int i0 = 0; i0 < M; i0 += TOGETHER) {
        unsigned long long w[TOGETHER], t[TOGETHER];
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) w[i] = mul2(x[i0 + i], u2);
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) w[i] = mul2(w[i], w[i]);
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) t[i] = ffma2(w[i], k[N - 1], k[N - 2]);
#pragma unroll
        for (int j = N - 3; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < TOGETHER; ++i) t[i] = ffma2(w[i], t[i], k[j]);
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) x[i0 + i] = mul2(x[i0 + i], t[i]);
    }
}
// The same of N pairs of products, whose scores are f times them.  Up to 1.25 of
// the cap a polynomial of more terms serves all of them (2e-7 off): packed, its
// ten operations for two scores cost less than two exponentials and reciprocals.
template <int N> __device__ __forceinline__ void cap_pairs(const ScoresView &v, unsigned long long (&x)[N], float f = 1.0f)
{
    float large[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 y = unpair(x[i]);
        large[i & 1] = fmax3(large[i & 1], fabsf(y.x), fabsf(y.y));
    }
    const float edge = CAP_SMALL * v.cap2;
    large[0] = fmaxf(large[0], large[1]) * fabsf(f);
    if (__any_sync(0xffffffffu, large[0] >= 2.0f * edge)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 y = unpair(x[i]);
            const float a = y.x * f, b = y.y * f;
            x[i] = pack2(fabsf(a) >= edge ? capped_large(v, a) : capped_small(v, a), fabsf(b) >= edge ? capped_large(v, b) : capped_small(v, b));
        }
    } else if (__any_sync(0xffffffffu, large[0] >= edge)) {
        constexpr float MEDIUM[8] = {0.999999929f, -0.333327294f, 0.133248116f, -0.0535018186f, 0.0205778305f, -0.006815299f, 0.00159693103f,
                                     -0.000184196065f};
        cap_polynomial(v, x, f, MEDIUM);
    } else {
        constexpr float SMALL[5] = {CAP_0, CAP_1, CAP_2, CAP_3, CAP_4};
        cap_polynomial(v, x, f, SMALL);
    }
}

// Lengths of a sequence, with the first slot that any of its new tokens can
// see, and the one from which on all of them see all cached slots.
struct SpanLens : SeqLens {
    int from, solid;
};

// The cut of the work for scored calls of up to 64 new tokens: tiles before
// `from` have none.
struct ScoredWork : Work {
    ScoresView sc;
};
__device__ __forceinline__ SpanLens lens_of(const ScoredWork &w, int b, const PagedView &c)
{
    SpanLens s;
    static_cast<SeqLens &>(s) = seq_lens(w.ctx_lens, w.new_lens, b, w.T, c, w.idle);
    if (w.sc.slot_pos && !s.bad && s.ctx + s.fresh > w.sc.pos_stride) {
        s.bad = true;
        s.total = 0;
    }
    s.from = s.solid = 0;
    if (s.total == 0) return s;
    const bool sliding = w.sc.window > 0 && !w.sc.slot_pos;
    if (sliding) {
        s.from = s.ctx - w.sc.window + 1;
        s.solid = s.from + s.fresh - 1;  // no node is deeper
    }
    if (w.sc.first) {
        int lowest = s.total, highest = 0;
        for (int t = 0; t < s.fresh; ++t) {
            const int f = __ldg(w.sc.first + static_cast<int64_t>(b) * w.T + t);
            lowest = min(lowest, f);
            highest = max(highest, f);
        }
        s.from = sliding ? max(s.from, lowest) : lowest;
        s.solid = max(s.solid, highest);
    }
    s.from = max(0, min(s.from, s.total - 1));
    s.solid = w.sc.window > 0 && w.sc.slot_pos ? s.total : max(s.solid, 0);
    return s;
}
__device__ __forceinline__ int skipped_tiles(const ScoredWork &w, const SpanLens &s) { return s.from / w.tile; }
__device__ __forceinline__ int first_seen(const SpanLens &s) { return s.from; }

// What new token t of sequence b sees, t < 64: of the new tokens those in the
// bits, of the cached slots those from `lo` on (of a token without bits none).
// Windows over moved slots are not in it.
struct TokenView {
    unsigned long long bits;
    int lo, depth;
};
__device__ __forceinline__ TokenView token_view(const ScoresView &v, const int32_t *parent, const SeqLens &s, int b, int T, int t)
{
    TokenView r;
    const bool sliding = v.window > 0 && !v.slot_pos;
    r.lo = 0;
    if (parent) {
        r.bits = 1ull << t;
        r.depth = 0;
        for (int u = t; u > 0;) {
            const int p = __ldg(parent + u);
            if (p < 0 || p >= u) {
                r.bits = 0;
                break;
            }
            ++r.depth;
            if (!sliding || r.depth < v.window) r.bits |= 1ull << p;
            u = p;
        }
    } else {
        r.bits = (2ull << t) - 1ull;
        r.depth = t;
        if (v.last) {
            const int end = __ldg(v.last + static_cast<int64_t>(b) * T + t);  // any value: compared before it is a difference
            if (end > s.ctx) r.bits |= end - s.ctx >= 64 ? ~0ull : (1ull << (end - s.ctx)) - 1ull;
        }
        if (sliding && t >= v.window) r.bits &= ~((1ull << (t - v.window + 1)) - 1ull);
    }
    if (sliding) r.lo = max(0, s.ctx + r.depth - v.window + 1);  // (far below 0 a slot's distance to it would not fit 32 bits)
    if (v.first) {
        const int f = __ldg(v.first + static_cast<int64_t>(b) * T + t);
        r.lo = max(r.lo, f);
        if (f > s.ctx) r.bits = f - s.ctx >= 64 ? 0ull : r.bits & ~((1ull << (f - s.ctx)) - 1ull);
    }
    return r;
}

// row_status of every sequence of a scored call, a block each.
cudaError_t launch_scored_status(const PagedView &c, const ScoredWork &w, int32_t *row_status, cudaStream_t st);

}  // namespace spv
