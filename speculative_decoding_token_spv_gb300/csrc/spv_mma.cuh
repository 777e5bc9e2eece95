// spv_mma.cuh -- warp-level tensor-core pieces of the attention calls:
// fragments of a paged K or V row slice staged in shared memory, for 16-bit
// and e4m3 caches.
//
// A slice is 16 keys of one head, its rows at D * sizeof(C) bytes with their
// 16-byte chunks permuted so that the eight rows of an 8 x 8 matrix fall on
// different banks.  All products run as m16n8k16 with 32-bit sums.  An e4m3
// cache is multiplied in f16, which holds every e4m3 value; its fragments
// come from 16-bit loads of byte pairs, so the contraction index of a
// 16-element group is permuted (slots 2t, 2t+1, 2t+8, 2t+9 hold elements
// 4t..4t+3), the same way for q, and two adjacent output columns trade places
// in a way that leaves a thread four adjacent outputs.
#pragma once

#include "spv_kv.cuh"
#include "spv_stream.cuh"

namespace spv {

// What the products are computed in.
template <typename T, typename C> struct MmaOf { using type = T; };
template <typename T> struct MmaOf<T, __nv_fp8_e4m3> { using type = __half; };

template <typename M> __device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Two e4m3 values (low, high byte) as two f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(x)));
    return r;
}

template <typename M> __device__ __forceinline__ uint32_t pack_mma(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack_mma<__nv_bfloat16>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack_mma<__half>(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a slice of ROW_BYTES rows.
template <int ROW_BYTES> __device__ __forceinline__ uint32_t chunk_at(int row, int chunk)
{
    if (ROW_BYTES >= 128) return row * ROW_BYTES + ((chunk ^ (row & 7)) << 4);
    return row * ROW_BYTES + ((chunk ^ ((row >> 1) & 3)) << 4);  // 64-byte rows: two share the banks' width
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Sixteen keys of one head on their way to shared memory: where they are.
// Pages of at least 16 slots hold a slice whole (slices start at multiples of
// 16); smaller ones are looked up row by row.
struct SliceSource {
    int page;  // of the whole slice, or of row `lane` (lane < 16); -1: none, or bad
    int keys;  // rows that exist
};
__device__ __forceinline__ SliceSource find_slice(const PagedView &c, const int32_t *table, int j0, int total, int lane,
                                                  bool *bad)
{
    SliceSource s;
    s.keys = min(16, total - j0);
    s.page = -1;
    if (s.keys <= 0) return s;
    if (c.page_shift >= 4) {
        s.page = page_of(c, table, j0);
        *bad |= s.page < 0;
    } else if (lane < s.keys) {
        s.page = page_of(c, table, j0 + lane);
        *bad |= s.page < 0;
    }
    return s;
}

// Starts the copies of a slice's rows (absent ones become zero).  A warp.
template <int ROW_BYTES>
__device__ __forceinline__ void copy_slice(const PagedView &c, const PoolView &pool, const SliceSource &s, int j0, int h,
                                           uint32_t dst, int lane)
{
    constexpr int CHUNKS = ROW_BYTES / 16, STEP = 32 / CHUNKS > 0 ? 32 / CHUNKS : 1;  // rows a warp copies at once
    if (s.keys <= 0) return;
    const int mask = (1 << c.page_shift) - 1;
    if (CHUNKS <= 32) {
        const int chunk = lane % CHUNKS;
        if (c.page_shift >= 4) {
            const char *base = pool.base + (s.page < 0 ? 0 : s.page) * pool.page_stride + h * pool.head_stride + chunk * 16;
            const int in = j0 & mask;
#pragma unroll
            for (int i = 0; i < 16; i += STEP) {
                const int row = i + lane / CHUNKS;
                const bool there = s.page >= 0 && row < s.keys;
                cp_async16_zfill(dst + chunk_at<ROW_BYTES>(row, chunk), there ? base + (in + row) * pool.slot_stride : pool.base,
                                 there ? 16 : 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += STEP) {
                const int row = i + lane / CHUNKS;
                const int page = __shfl_sync(0xffffffffu, s.page, row);
                const bool there = page >= 0;
                cp_async16_zfill(dst + chunk_at<ROW_BYTES>(row, chunk),
                                 there ? pool.base + page * pool.page_stride + ((j0 + row) & mask) * pool.slot_stride +
                                             h * pool.head_stride + chunk * 16
                                       : pool.base,
                                 there ? 16 : 0);
            }
        }
    }
}

// Scores of MT x 16 rows with the 16 keys of a slice: s[mt][key tile][4].
// `qa(mt, ks, a)` gives the q fragment of rows 16 mt.., elements 16 ks...
template <typename M, typename C, int D, int MT, typename QF>
__device__ __forceinline__ void slice_scores(float (&s)[MT][2][4], uint32_t k_slice, int lane, QF &&qa)
{
    constexpr int RB = D * static_cast<int>(sizeof(C));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.0f;
    const int mat = lane >> 3, r8 = lane & 7;
    if (sizeof(C) == 2) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldmatrix4(b, k_slice + chunk_at<RB>((mat >> 1) * 8 + r8, 2 * ks + (mat & 1)));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t a[4];
                qa(mt, ks, a);
                mma16816<M>(s[mt][0], a, b[0], b[1]);
                mma16816<M>(s[mt][1], a, b[2], b[3]);
            }
        }
    } else {
#pragma unroll
        for (int kp = 0; kp < D / 32; ++kp) {
            uint32_t b[4];
            ldmatrix4(b, k_slice + chunk_at<RB>((mat & 1) * 8 + r8, 2 * kp + (mat >> 1)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u0 = e4m3x2_to_f16x2(b[2 * i] & 0xffffu), u1 = e4m3x2_to_f16x2(b[2 * i] >> 16);
                const uint32_t w0 = e4m3x2_to_f16x2(b[2 * i + 1] & 0xffffu), w1 = e4m3x2_to_f16x2(b[2 * i + 1] >> 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t a[4];
                    qa(mt, 2 * kp + i, a);
                    mma16816<M>(s[mt][0], a, u0, u1);
                    mma16816<M>(s[mt][1], a, w0, w1);
                }
            }
        }
    }
}

// o += p v over a slice: p[mt] the probabilities as a fragment.
template <typename M, typename C, int D, int MT>
__device__ __forceinline__ void slice_values(float (&o)[MT][D / 8][4], const uint32_t (&p)[MT][4], uint32_t v_slice, int lane)
{
    constexpr int RB = D * static_cast<int>(sizeof(C));
    const int mat = lane >> 3, r8 = lane & 7;
#pragma unroll
    for (int dt = 0; dt < D / (sizeof(C) == 2 ? 16 : 32); ++dt) {
        uint32_t b[4];
        ldmatrix4_trans(b, v_slice + chunk_at<RB>((mat & 1) * 8 + r8, 2 * dt + (mat >> 1)));
        if (sizeof(C) == 2) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                mma16816<M>(o[mt][2 * dt], p[mt], b[0], b[1]);
                mma16816<M>(o[mt][2 * dt + 1], p[mt], b[2], b[3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u0 = e4m3x2_to_f16x2(b[2 * i] & 0xffffu), u1 = e4m3x2_to_f16x2(b[2 * i] >> 16);
                const uint32_t w0 = e4m3x2_to_f16x2(b[2 * i + 1] & 0xffffu), w1 = e4m3x2_to_f16x2(b[2 * i + 1] >> 16);
                const uint32_t e0 = __byte_perm(u0, u1, 0x5410), e1 = __byte_perm(w0, w1, 0x5410);
                const uint32_t f0 = __byte_perm(u0, u1, 0x7632), f1 = __byte_perm(w0, w1, 0x7632);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma16816<M>(o[mt][4 * dt + 2 * i], p[mt], e0, e1);
                    mma16816<M>(o[mt][4 * dt + 2 * i + 1], p[mt], f0, f1);
                }
            }
        }
    }
}

// Output column of o[.][tile][e] (e = 0, 1 of either row).
template <typename C> __device__ __forceinline__ int value_column(int tile, int e, int lane)
{
    const int t = lane & 3;
    if (sizeof(C) == 2) return tile * 8 + 2 * t + e;
    return (tile >> 1) * 16 + 4 * t + 2 * e + (tile & 1);
}

// Stores 8 elements of q (starting at d, a multiple of 8) of row r, in the
// order that slice_scores multiplies them.
template <typename M, typename C, int D> __device__ __forceinline__ void put_q8(char *qs, int r, int d, const float *x)
{
    if (sizeof(C) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_mma<M>(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint4 *>(qs + chunk_at<D * 2>(r, d >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {  // elements 4t..4t+3 of 16 sit at 2t, 2t+1, 2t+8, 2t+9
        const int c0 = (d >> 4) * 2, t0 = (d & 8) >> 2;  // t = t0, t0 + 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<uint32_t *>(qs + chunk_at<D * 2>(r, c0) + (t0 + i) * 4) = pack_mma<M>(x[4 * i], x[4 * i + 1]);
            *reinterpret_cast<uint32_t *>(qs + chunk_at<D * 2>(r, c0 + 1) + (t0 + i) * 4) = pack_mma<M>(x[4 * i + 2], x[4 * i + 3]);
        }
    }
}

// The q fragment of rows 16 mt.. and elements 16 ks.. from the block's q tile.
template <int D> __device__ __forceinline__ void get_q(uint32_t (&a)[4], uint32_t qs, int mt, int ks, int lane)
{
    const int mat = lane >> 3, r8 = lane & 7;
    ldmatrix4(a, qs + chunk_at<D * 2>(mt * 16 + (mat & 1) * 8 + r8, 2 * ks + (mat >> 1)));
}

}  // namespace spv
