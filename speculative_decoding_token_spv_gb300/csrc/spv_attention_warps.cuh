// spv_attention_warps.cuh -- attention of a sequence's new tokens over its paged
// cache, in one pass over K and V.
//
// Mathematics: with scores in powers of two, s = q.k scale log2 e, a warp
// keeps for each of its rows the running maximum m, l = sum 2^(s - m) and
// o = sum 2^(s - m) v over the keys it takes; partial results join as
// M = max m_i, l = sum l_i 2^(m_i - M), o likewise, out = o / l.
//
// What bounds it is reading K and V once.  The work is cut along the cache
// (Work, Cursor), so the grid is the same for any lengths.  A block's four
// warps take 16 keys each of a 64-key tile and share nothing until the end of
// the piece: each has its own ring of K and V slices filled by asynchronous
// copies, so that no warp waits for another and up to 190 KB an SM are on
// their way.  All rows of a key head (new tokens x query heads of its group)
// go through the tensor cores against the slice together, 16 or 32 of them.
// Blocks leave what they have of a shared item in the workspace; a dependent
// launch joins the pieces in their order along the sequence.
//
// 64 sequences of up to 8,191 slots, one token, 32 query heads on 8 key heads, D
// = 128, bf16, 1.36 GB: 214 us, 6.3 TB/s, 94% of a copy's rate.  Two sequences of
// 131,001 slots in e4m3, 32 rows a key head, 537 MB: 163 us, bound by issuing the
// conversions and products, about 600 instructions for 16 keys.  One token of
// one sequence of 777 slots, captured: 10.0 us, the chain from lengths to page ids
// to keys, the join's launch and its loads.
//
// The same kernel serves calls with scores and masks (spv_scores): these are
// then made from the products, in powers of two, before the running maximum,
// and masks are looked at in the slices where some row may not see a slot.  That
// one token, capped and captured: 11.7 us, with its status 13.0; 64 sequences of
// up to 8,191 slots, 16 heads on 8 of 256, capped: 484 us (441 plain), which
// spv_scored.cu gives to tiles.
#pragma once

#include "spv_scored.cuh"

namespace spv {

constexpr int ATT_WARPS = 4;
constexpr int ATT_THREADS = 32 * ATT_WARPS;
constexpr int ATT_KEYS = 16 * ATT_WARPS;  // keys of a tile: a slice for each warp
constexpr int ATT_MAX_ROWS = 32;

__device__ __forceinline__ ScoresView p_scores(const AttParams &) { return ScoresView{}; }
__device__ __forceinline__ const ScoresView &p_scores(const ScoredParams &p) { return p.sc; }

// Sizes of a variant: MT tiles of 16 rows.
template <typename C, int D, int MT> struct AttShape {
    static constexpr int R = 16 * MT;
    static constexpr int ROW_BYTES = D * static_cast<int>(sizeof(C));
    static constexpr int SLICE = 16 * ROW_BYTES;
    static constexpr int STAGES = SLICE >= 4096 ? 2 : 4;
    static constexpr int RING = ATT_WARPS * STAGES * 2 * SLICE;
    static constexpr int PAD = D + 8;  // row of the merge buffer: 8 rows on different banks
    static constexpr int MERGE = ATT_WARPS * R * PAD * 4;
    static constexpr int Q = R * D * 2;
    static constexpr int SMEM = Q + (RING > MERGE ? RING : MERGE);
    static constexpr int BLOCKS_PER_SM = SMEM * 3 <= 216 * 1024 ? 3 : SMEM * 2 <= 216 * 1024 ? 2 : 1;
    static constexpr bool Q_IN_REGISTERS = MT == 1 && D <= 128;
};

template <typename T, typename C, int D, int MT, typename P>
__global__ void __launch_bounds__(ATT_THREADS, AttShape<C, D, MT>::BLOCKS_PER_SM) attention_kernel(const P p)
{
    constexpr bool SCORED = std::is_same<P, ScoredParams>::value;
    using S = AttShape<C, D, MT>;
    using M = typename MmaOf<T, C>::type;
    constexpr int R = S::R, PART = R * (D + 2), NST = S::STAGES;
    constexpr float UP = Weights<M>::UP;
    extern __shared__ __align__(1024) char smem[];
    __shared__ float ms[ATT_WARPS][R], ls[ATT_WARPS][R];
    __shared__ float q_unit[R];                // what a unit of the stored q row stands for
    __shared__ unsigned long long sees[R];     // new tokens that each row sees; 0: a row that sees nothing
    const auto &work = work_of(p);
    using Cur = CursorOf<decltype(lens_of(work, 0, p.c))>;
    __shared__ Cur cur0;
    __shared__ int flag;
    // of a call with scores: the first cached slot that each row sees, its position, its slope; depths of a tree's nodes
    __shared__ int row_lo[SCORED ? R : 1], row_pos[SCORED ? R : 1], depths[SCORED ? 64 : 1];
    __shared__ float row_slope[SCORED ? R : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    char *qs = smem;
    float *merge = reinterpret_cast<float *>(smem + S::Q);
    const uint32_t qs32 = smem_u32(qs), ring = smem_u32(smem + S::Q) + warp * (NST * 2 * S::SLICE);
    chain_begin();
    if (tid < 32) {
        const Cur c = find_range(work, p.c, blockIdx.x, gridDim.x, tid);
        if (tid == 0) cur0 = c;
    }
    __syncthreads();
    Cur c = cur0;
    const long long begin = c.at;
    if (tid < 2) p.split[blockIdx.x * 2 + tid].n = 0;
    for (; c.at < c.end; next_item(c, work, p.c)) {
        const int row0 = c.row_tile * R, live = min(R, p.rows - row0);
        const long long item_end = c.first + c.tiles;
        const int t0 = static_cast<int>(c.at - c.first);
        const int t1 = c.s.total > 0 ? static_cast<int>((c.end < item_end ? c.end : item_end) - c.first) : t0;
        const int32_t *table = p.c.table + static_cast<int64_t>(c.b) * p.c.max_pages;
        bool bad = c.s.bad;
        const int skip = skipped_tiles(work, c.s);  // tiles are counted from the first that is seen

        // the first slices, as early as the page table allows
        SliceSource src = find_slice(p.c, table, (t0 + skip) * ATT_KEYS + warp * 16, t0 < t1 ? c.s.total : 0, first_seen(c.s), lane, &bad);
        auto issue = [&](int tile) {
            if (tile < t1) {
                const int j0 = (tile + skip) * ATT_KEYS + warp * 16;
                const uint32_t dst = ring + ((tile - t0) % NST) * (2 * S::SLICE);
                copy_slice<S::ROW_BYTES>(p.c, p.c.k, src, j0, c.h, dst, lane);
                copy_slice<S::ROW_BYTES>(p.c, p.c.v, src, j0, c.h, dst + S::SLICE, lane);
                src = find_slice(p.c, table, j0 + ATT_KEYS, tile + 1 < t1 ? c.s.total : 0, first_seen(c.s), lane, &bad);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) issue(t0 + i);

        // Scores are q.k times a factor, which is kept positive (its sign goes into q; a scale of 0 makes q 0), so that
        // the largest product is the largest score.  (The product is rounded as m was, not fused with the difference:
        // of scores beyond 2^27 the largest would else miss m by more than p can hold.)
        const float signed_unit = p.scale_log2 * (p.c.k_scale ? __ldg(p.c.k_scale + c.h) : 1.0f);
        const float turn = signed_unit < 0.0f ? -1.0f : signed_unit == 0.0f ? 0.0f : 1.0f;
        const float unit = signed_unit == 0.0f ? 1.0f : fabsf(signed_unit);
        // q of the tile's rows; for an e4m3 cache each row by a power of two into f16's range
        for (int i = tid; i < R * (D / 8); i += ATT_THREADS) {
            const int r = i / (D / 8), d = (i - r * (D / 8)) * 8, t = (row0 + r) / p.group, g = (row0 + r) - t * p.group;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.0f;
            if (r < live && t < c.s.fresh && !c.s.bad) {
                const T *q = static_cast<const T *>(p.q) +
                             ((static_cast<int64_t>(c.b) * p.w.T + t) * p.q_heads + c.h * p.group + g) * D + d;
                const uint4 raw = *reinterpret_cast<const uint4 *>(q);
                const T *y = reinterpret_cast<const T *>(&raw);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = Num<T>::up(y[e]) * turn;
            }
            if (sizeof(C) == 1) {
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fabsf(x[e]) < CUDART_INF_F ? fmaxf(top, fabsf(x[e])) : top;
#pragma unroll
                for (int o = D / 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e2 = 0;
                if (top > 0.0f) e2 = 14 - ilogbf(top);  // the largest below 2^15
                e2 = max(-120, min(120, e2));           // both scales normal numbers
                const float up = exp2f(static_cast<float>(e2));
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= up;
                if (d == 0) q_unit[r] = exp2f(static_cast<float>(-e2));
            }
            put_q8<M, C, D>(qs, r, d, x);
        }
        if (tid < R) {
            const int t = (row0 + tid) / p.group;
            const bool there = tid < live && t < c.s.fresh && !c.s.bad;
            const int32_t *parent = p.parent ? p.parent + static_cast<int64_t>(c.b) * p.w.T : nullptr;
            if constexpr (SCORED) {
                sees[tid] = 0;
                if (there) {
                    const TokenView view = token_view(p.sc, parent, c.s, c.b, p.w.T, t);
                    sees[tid] = view.bits;
                    row_lo[tid] = view.lo;
                    row_pos[tid] = p.sc.slot_pos ? __ldg(p.sc.slot_pos + (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p.sc.pos_stride + c.s.ctx + t)
                                                 : c.s.ctx + view.depth;
                    row_slope[tid] = p.sc.slopes ? __ldg(p.sc.slopes + c.h * p.group + row0 + tid - t * p.group) * LOG2E : 0.0f;
                } else {
                    row_lo[tid] = row_pos[tid] = 0;
                    row_slope[tid] = 0.0f;
                }
            } else {
                sees[tid] = there ? visible_mask(parent, t) : 0ull;
            }
        }
        if constexpr (SCORED) {
            if (p.parent && p.sc.slopes && !p.sc.slot_pos && tid < c.s.fresh)
                depths[tid] = token_view(p.sc, p.parent + static_cast<int64_t>(c.b) * p.w.T, c.s, c.b, p.w.T, tid).depth;
        }
        if (tid == 0) flag = 0;
        __syncthreads();

        uint32_t qr[S::Q_IN_REGISTERS ? D / 16 : 1][4];
        if (S::Q_IN_REGISTERS) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) get_q<D>(qr[S::Q_IN_REGISTERS ? ks : 0], qs32, 0, ks, lane);
        }
        auto q_fragment = [&](int mt, int ks, uint32_t (&a)[4]) {
            if (S::Q_IN_REGISTERS) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = qr[S::Q_IN_REGISTERS ? ks : 0][i];
            } else {
                get_q<D>(a, qs32, mt, ks, lane);
            }
        };
        float factor[MT][2], m[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                factor[mt][i] = sizeof(C) == 1 ? unit * q_unit[mt * 16 + i * 8 + (lane >> 2)] : unit;
                m[mt][i] = -CUDART_INF_F;
                l[mt][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.0f;
        }
        // positions of this lane's four keys of a slice, a tile ahead
        const bool moved = SCORED && moved_slots(p_scores(p));
        const bool shaped = SCORED && (p_scores(p).cap2 != 0.0f || p_scores(p).slopes || moved);  // scores are more than products
        const int32_t *pos = moved ? p_scores(p).slot_pos + (static_cast<int64_t>(c.b) * p.c.kv_heads + c.h) * p_scores(p).pos_stride : nullptr;
        int key_pos[4], next_pos[4];
        auto positions = [&](int tile, int (&to)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = (tile + skip) * ATT_KEYS + warp * 16 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                to[i] = moved && tile < t1 && j < c.s.total ? __ldg(pos + j) : j;
            }
        };
        if constexpr (SCORED) positions(t0, next_pos);
        for (int tile = t0; tile < t1; ++tile) {
            if constexpr (SCORED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) key_pos[i] = next_pos[i];
                positions(tile + 1, next_pos);
            }
            __syncwarp();
            issue(tile + NST - 1);
            cp_async_wait<NST - 1>();
            __syncwarp();
            const int j0 = (tile + skip) * ATT_KEYS + warp * 16;
            if (j0 >= c.s.total) break;
            const uint32_t stage = ring + ((tile - t0) % NST) * (2 * S::SLICE);
            float s[MT][2][4];
            slice_scores<M, C, D, MT>(s, stage, lane, q_fragment);
            bool tail = j0 + 16 > c.s.ctx;  // some row may not see some key
            if constexpr (SCORED) {
                const ScoresView &v = p.sc;
                if (p.parent && v.slopes && !v.slot_pos && tail) {  // a node's position is its depth's
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key_pos[i] >= c.s.ctx && key_pos[i] < c.s.total) key_pos[i] = c.s.ctx + depths[key_pos[i] - c.s.ctx];
                }
                tail |= j0 < c.s.solid;
                if (shaped) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        float x[8];  // key tile, then the fragment's four
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = s[mt][k >> 2][k & 3] * factor[mt][(k & 3) >> 1];
                        if (v.cap2 != 0.0f) {
                            unsigned long long y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = pack2(x[2 * k], x[2 * k + 1]);
                            cap_pairs(v, y);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 z = unpair(y[k]);
                                x[2 * k] = z.x, x[2 * k + 1] = z.y;
                            }
                        }
                        if (v.slopes || moved) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int r = mt * 16 + ((k & 3) >> 1) * 8 + (lane >> 2), far = row_pos[r] - key_pos[2 * (k >> 2) + (k & 1)];
                                if (v.slopes) x[k] = fmaf(-row_slope[r], fabsf(static_cast<float>(far)), x[k]);
                                if (moved && v.window > 0 && far >= v.window) x[k] = -CUDART_INF_F;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[mt][k >> 2][k & 3] = x[k];
                    }
                }
            }
            uint32_t pf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (tail) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const unsigned long long see = sees[mt * 16 + (e >> 1) * 8 + (lane >> 2)];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = j0 + 8 * i + 2 * (lane & 3) + (e & 1);
                            if (SCORED && (j < row_lo[mt * 16 + (e >> 1) * 8 + (lane >> 2)] || see == 0)) s[mt][i][e] = -CUDART_INF_F;
                            if (!(j < c.s.ctx || (j < c.s.total && (see >> (j - c.s.ctx) & 1)))) s[mt][i][e] = -CUDART_INF_F;
                        }
                    }
                }
                // m, the maximum less UP, follows it only where it has grown by more than 2^LAG (or begins): p stays below
                // 2^(UP + LAG), the 32-bit sums lose nothing, and o is seldom rescaled -- with every growth it was in nearly
                // every slice.  (The growth as a difference: a sum may round up to the next score where these are 16 apart,
                // which would then be 2^16, more than an f16 holds.)
                float top[2];
                bool moved = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(fmaxf(s[mt][0][2 * i], s[mt][0][2 * i + 1]), fmaxf(s[mt][1][2 * i], s[mt][1][2 * i + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    top[i] = shaped ? x : x * factor[mt][i];
                    moved |= top[i] - m[mt][i] > UP + Weights<M>::LAG;  // m minus infinity: any score
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float grown = fmaxf(m[mt][i], top[i] - UP);
                        const float a = grown == -CUDART_INF_F ? 0.0f : fast_exp2(m[mt][i] - grown);
                        m[mt][i] = grown;
                        l[mt][i] *= a;
#pragma unroll
                        for (int k = 0; k < D / 8; ++k) {
                            o[mt][k][2 * i] *= a;
                            o[mt][k][2 * i + 1] *= a;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float base = m[mt][i] == -CUDART_INF_F ? 0.0f : m[mt][i], f = shaped ? 1.0f : factor[mt][i];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 2 * i; e < 2 * i + 2; ++e) s[mt][k][e] = fast_exp2(__fmul_rn(s[mt][k][e], f) - base);
                    l[mt][i] += (s[mt][0][2 * i] + s[mt][0][2 * i + 1]) + (s[mt][1][2 * i] + s[mt][1][2 * i + 1]);
                }
                // rounded to the cache's 16-bit type for the product (half a step of it each); l keeps 32 bits
                pf[mt][0] = pack_mma<M>(s[mt][0][0], s[mt][0][1]);
                pf[mt][1] = pack_mma<M>(s[mt][0][2], s[mt][0][3]);
                pf[mt][2] = pack_mma<M>(s[mt][1][0], s[mt][1][1]);
                pf[mt][3] = pack_mma<M>(s[mt][1][2], s[mt][1][3]);
            }
            if (tail) {
                // A key's v may hold infinities or NaN that rows that do not see it must not meet as 0 x inf:
                // such a key is added to the rows that see it here, and its v cleared before the product.
                char *v = smem + S::Q + (stage - smem_u32(smem + S::Q)) + S::SLICE;
                constexpr int CHUNKS = S::ROW_BYTES / 16;
                unsigned odd = 0;
                for (int i = lane; i < 16 * CHUNKS; i += 32) {
                    const int row = i / CHUNKS;
                    if ((SCORED || j0 + row >= c.s.ctx) &&
                        chunk_not_finite<C>(*reinterpret_cast<const uint4 *>(v + chunk_at<S::ROW_BYTES>(row, i % CHUNKS))))
                        odd |= 1u << row;
                }
                odd = __reduce_or_sync(0xffffffffu, odd);
                for (; odd; odd &= odd - 1) {
                    const int row = __ffs(odd) - 1;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // p of (row 8 i + lane / 4, key row): the quad's lane that holds column row % 8
                            const float lo = __shfl_sync(0xffffffffu, row < 8 ? s[mt][0][2 * i] : s[mt][1][2 * i], (lane & ~3) | ((row & 7) >> 1));
                            const float hi = __shfl_sync(0xffffffffu, row < 8 ? s[mt][0][2 * i + 1] : s[mt][1][2 * i + 1], (lane & ~3) | ((row & 7) >> 1));
                            const float w = (row & 1) ? hi : lo;
                            if (w != 0.0f) {
#pragma unroll
                                for (int k = 0; k < D / 8; ++k)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int d = value_column<C>(k, e, lane) * static_cast<int>(sizeof(C));
                                        o[mt][k][2 * i + e] += w * Num<C>::up(*reinterpret_cast<const C *>(
                                                                       v + chunk_at<S::ROW_BYTES>(row, d >> 4) + (d & 15)));
                                    }
                            }
                        }
                    __syncwarp();
                    for (int i = lane; i < CHUNKS; i += 32)
                        *reinterpret_cast<uint4 *>(v + chunk_at<S::ROW_BYTES>(row, i)) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            slice_values<M, C, D, MT>(o, pf, stage + S::SLICE, lane);
        }
        cp_async_wait<0>();

        // the four warps' parts into one
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = l[mt][i];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                const int r = mt * 16 + i * 8 + (lane >> 2);
                if ((lane & 3) == 0) {
                    ms[warp][r] = sees[r] ? m[mt][i] : -CUDART_INF_F;
                    ls[warp][r] = sees[r] ? x : 0.0f;
                }
            }
        if (bad) flag = 1;
        __syncthreads();  // the rings are free
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = mt * 16 + i * 8 + (lane >> 2);
                if (r < live) {
                    float *row = merge + (warp * R + r) * S::PAD;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) row[value_column<C>(k, e, lane)] = o[mt][k][2 * i + e];
                }
            }
        const bool any_bad = flag != 0;
        __syncthreads();
        const bool whole = c.s.total == 0 || (t0 == 0 && t1 == c.tiles);
        const float v_scale = p.c.v_scale ? __ldg(p.c.v_scale + c.h) : 1.0f;
        float *part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (c.first < begin ? 0 : 1)) * PART;

        const AttRows rows{c.b, c.h, row0, live};
        for (int i = tid; i < live * (D / 4); i += ATT_THREADS) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float mr = ms[0][r];
#pragma unroll
            for (int w = 1; w < ATT_WARPS; ++w) mr = fmaxf(mr, ms[w][r]);
            const float base = mr == -CUDART_INF_F ? 0.0f : mr;
            float lr = 0.0f;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) {
                const float a = fast_exp2(ms[w][r] - base);
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * R + r) * S::PAD + d);
                if (ls[w][r] != 0.0f) {  // a warp without keys has nothing to add
                    lr += a * ls[w][r];
                    x.x += a * y.x, x.y += a * y.y, x.z += a * y.z, x.w += a * y.w;
                }
            }
            if (any_bad) mr = CUDART_NAN_F;
            if (whole) {
                write_row<T, D>(p, rows, r, d, x, mr, lr, v_scale);
            } else {
                if (d == 0) {
                    part[r] = mr;
                    part[R + r] = lr;
                }
                *reinterpret_cast<float4 *>(part + 2 * R + r * D + d) = x;
            }
        }
        if (!whole) note_split(p, c, rows, begin, tid);
        if (whole && tid == 0 && p.row_status && c.h == 0 && c.row_tile == 0) p.row_status[c.b] = any_bad ? KV_STATUS_BAD : 0;
        __syncthreads();
    }
}

template <typename T, typename C, int D, int MT, typename P> static cudaError_t launch_rows(const P &p, cudaStream_t st)
{
    using S = AttShape<C, D, MT>;
    auto kernel = attention_kernel<T, C, D, MT, P>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    constexpr int BLOCKS = ATT_SMS * S::BLOCKS_PER_SM;
    e = launch_chained(kernel, dim3(BLOCKS), ATT_THREADS, S::SMEM, st, p);
    return e != cudaSuccess ? e : launch_join(p, std::is_same<T, __half>::value ? SPV_F16 : SPV_BF16, D, S::R, BLOCKS, st);
}
template <typename T, typename C, int D, typename P> static cudaError_t launch_dim(P &p, cudaStream_t st)
{
    if constexpr (sizeof(C) == 1 && D <= 128) {  // 17 to 32 rows at once; at D = 256 their sums would not fit the registers
        if (p.rows > 16) {
            p.w.row_tiles = (p.rows + 31) / 32;
            return launch_rows<T, C, D, 2>(p, st);
        }
    }
    p.w.row_tiles = (p.rows + 15) / 16;
    return launch_rows<T, C, D, 1>(p, st);
}
template <typename T, typename C, typename P> static cudaError_t launch_types(P &p, int D, cudaStream_t st)
{
    if (D == 64) return launch_dim<T, C, 64>(p, st);
    if (D == 128) return launch_dim<T, C, 128>(p, st);
    return launch_dim<T, C, 256>(p, st);
}

}  // namespace spv
