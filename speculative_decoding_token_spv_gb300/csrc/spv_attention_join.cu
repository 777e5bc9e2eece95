// spv_attention_join.cu -- puts together the pieces of the items that several
// blocks of an attention kernel share.
//
// Join blocks (i, 0) and (i, 1) serve the items that main block i has pieces
// of (at most two).  The n blocks of an item share out its rows, so an item in many
// pieces -- few sequences, long caches -- is joined by many blocks; and where
// a block gets fewer rows than it has warps, its warps share out the pieces of
// a row.  M = max m_i, l = sum l_i 2^(m_i - M), o likewise, always in the
// order of the pieces.  All loads come from the L2, about a microsecond away
// for the far half of it: each warp has eight rows under way.  (Joined by the
// last block to finish an item, the attention of 40 rows over 64 sequences of up
// to 8,191 slots took 257 us where it took 245 like this.)
#include "spv_attention.cuh"

namespace spv {

constexpr int JOIN_WARPS = 8;
constexpr int JOIN_AHEAD = 8;

struct JoinShape {
    int part, rows;  // floats of a piece, rows it has room for
};

template <typename T, int D> __global__ void __launch_bounds__(32 * JOIN_WARPS) join_kernel(const AttParams p, const JoinShape js)
{
    constexpr int PER = D / 32;  // columns of a lane: two at D = 64, else four next to one another
    __shared__ float ms[JOIN_WARPS], ls[JOIN_WARPS];
    __shared__ float xs[JOIN_WARPS][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    chain_begin();
    const SplitItem s = p.split[blockIdx.x * 2 + blockIdx.y];
    if (s.n == 0) return;
    const int first = blockIdx.x - s.b0, mine = (s.rows.live - first + s.n - 1) / s.n;  // rows first, first + n, ...
    if (mine <= 0) return;
    int team = 1;  // warps of a row
    while (team * 2 * mine <= JOIN_WARPS && team < s.n) team *= 2;
    const int teams = JOIN_WARPS / team, member = warp % team;
    const int from = s.n * member / team, to = s.n * (member + 1) / team;  // this warp's pieces
    const float v_scale = p.c.v_scale ? __ldg(p.c.v_scale + s.rows.h) : 1.0f;
    for (int k0 = 0; k0 < mine; k0 += teams) {
        const int k = k0 + warp / team, r = first + k * s.n;
        const bool here = k < mine;
        float m = -CUDART_INF_F, l = 0.0f, x[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) x[e] = 0.0f;
        bool nan = false;
        if (here) {
            // the first pieces' rows, on their way before the weights are known
            float y[JOIN_AHEAD][PER];
            auto fetch = [&](int j0) {
#pragma unroll
                for (int j = 0; j < JOIN_AHEAD; ++j) {
#pragma unroll
                    for (int e = 0; e < PER; ++e) y[j][e] = 0.0f;
                    if (j0 + j < to) {
                        const float *o = piece_of(p, s.b0 + j0 + j, s.b0, js.part) + 2 * js.rows + r * D;
                        if (PER == 2) {
                            const float2 z = __ldcg(reinterpret_cast<const float2 *>(o + 2 * lane));
                            y[j][0] = z.x, y[j][1] = z.y;
                        } else {
#pragma unroll
                            for (int e = 0; e < PER; e += 4) {
                                const float4 z = __ldcg(reinterpret_cast<const float4 *>(o + e * 32 + 4 * lane));
                                y[j][e] = z.x, y[j][e + 1] = z.y, y[j][e + 2] = z.z, y[j][e + 3] = z.w;
                            }
                        }
                    }
                }
            };
            fetch(from);
            float pm = -CUDART_INF_F, pl = 0.0f;  // of this lane's piece among 32
            if (from + lane < to) {
                const float *o = piece_of(p, s.b0 + from + lane, s.b0, js.part);
                pm = __ldcg(o + r);
                pl = __ldcg(o + js.rows + r);
            }
            nan = pm != pm;
            m = fmaxf(m, pm);
            for (int i = from + 32 + lane; i < to; i += 32) {
                const float z = __ldcg(piece_of(p, s.b0 + i, s.b0, js.part) + r);
                nan |= z != z;
                m = fmaxf(m, z);
            }
            m = warp_max(m);
            nan = __any_sync(0xffffffffu, nan);
            const float base = m == -CUDART_INF_F ? 0.0f : m;
            for (int i0 = from; i0 < to; i0 += 32) {
                if (i0 > from && i0 + lane < to) {
                    const float *o = piece_of(p, s.b0 + i0 + lane, s.b0, js.part);
                    pm = __ldcg(o + r);
                    pl = __ldcg(o + js.rows + r);
                }
                // not skipped where it is 0: a piece of NaN alone has m = minus infinity
                const float a = i0 + lane < to ? fast_exp2(pm - base) : 0.0f;
                if (i0 + lane < to) l += a * pl;
#pragma unroll
                for (int j0 = 0; j0 < 32; j0 += JOIN_AHEAD) {
                    if (i0 + j0 >= to) break;
                    if (i0 + j0 > from) fetch(i0 + j0);
#pragma unroll
                    for (int j = 0; j < JOIN_AHEAD; ++j) {
                        const float w = __shfl_sync(0xffffffffu, a, j0 + j);
#pragma unroll
                        for (int e = 0; e < PER; ++e) x[e] += w * y[j][e];
                    }
                }
            }
            l = warp_sum(l);
        }
        if (nan) m = CUDART_NAN_F;
        if (team > 1) {
            __syncthreads();
            if (lane == 0) {
                ms[warp] = m;
                ls[warp] = l;
            }
#pragma unroll
            for (int e = 0; e < PER; ++e) xs[warp][PER == 2 ? 2 * lane + e : (e >> 2) * 128 + 4 * lane + (e & 3)] = x[e];
            __syncthreads();
            if (member == 0 && here) {
                float all = -CUDART_INF_F;
                for (int q = 0; q < team; ++q) {
                    nan |= ms[warp + q] != ms[warp + q];
                    all = fmaxf(all, ms[warp + q]);
                }
                const float base = all == -CUDART_INF_F ? 0.0f : all;
                l = 0.0f;
#pragma unroll
                for (int e = 0; e < PER; ++e) x[e] = 0.0f;
                for (int q = 0; q < team; ++q) {
                    if (ls[warp + q] == 0.0f) continue;
                    const float w = fast_exp2(ms[warp + q] - base);
                    l += w * ls[warp + q];
#pragma unroll
                    for (int e = 0; e < PER; ++e)
                        x[e] += w * xs[warp + q][PER == 2 ? 2 * lane + e : (e >> 2) * 128 + 4 * lane + (e & 3)];
                }
                m = nan ? CUDART_NAN_F : all;
            }
        }
        if (here && member == 0) {
            if (PER == 2) {
                const float a = __shfl_down_sync(0xffffffffu, x[0], 1), b = __shfl_down_sync(0xffffffffu, x[1], 1);
                if (lane % 2 == 0) write_row<T, D>(p, s.rows, r, 2 * lane, make_float4(x[0], x[1], a, b), m, l, v_scale);
            } else {
#pragma unroll
                for (int e = 0; e < PER; e += 4)
                    write_row<T, D>(p, s.rows, r, e * 32 + 4 * lane, make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]), m, l, v_scale);
            }
            if (lane == 0 && r == 0 && p.row_status && s.rows.h == 0 && s.rows.row0 == 0)
                p.row_status[s.rows.b] = m == m ? 0 : __ldcg(p.error) ? STATUS_TIMEOUT : KV_STATUS_BAD;
        }
    }
}

template <typename T, int D> static cudaError_t launch(const AttParams &p, const JoinShape &js, int blocks, cudaStream_t st)
{
    return launch_chained(join_kernel<T, D>, dim3(blocks, 2), 32 * JOIN_WARPS, 0, st, p, js);
}

cudaError_t launch_join(const AttParams &p, spv_dtype q, int D, int R, int blocks, cudaStream_t st)
{
    const JoinShape js{R * (D + 2), R};
    if (q == SPV_BF16)
        return D == 64 ? launch<__nv_bfloat16, 64>(p, js, blocks, st) : D == 128 ? launch<__nv_bfloat16, 128>(p, js, blocks, st)
                                                                               : launch<__nv_bfloat16, 256>(p, js, blocks, st);
    return D == 64 ? launch<__half, 64>(p, js, blocks, st) : D == 128 ? launch<__half, 128>(p, js, blocks, st)
                                                                     : launch<__half, 256>(p, js, blocks, st);
}

}  // namespace spv
