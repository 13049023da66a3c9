// Cached rows of the decode kernels over ranges of tiles (decode_ranges_sm103.cu): for
// each format its tile, and the two products over 16 positions with mma.sync.
//
//   bf16   1,024 bytes a row of one head; operands as stored
//   E4M3   512 bytes; widened exactly to f16
//   4 bits 288 bytes: 256 of E2M1 codes (element 2 i in the low half of byte i), 32
//          E4M3 scales of 16 elements each.  A scale times a code has 6 significant
//          bits and lies between 2^-10 and 2,688: exact in f16.
//
// S^T = K Q^T has the query rows in N and 16 positions in M, a lane holding those at
// order(g) and order(g) + 8 of a block; O^T = V^T P^T has 16 columns in M and the
// positions in K, a lane holding V rows order(2 t), order(2 t + 1) and those + 8.  bf16
// and E4M3 tiles are boxes of 128 bytes x positions under TMA's 128-byte swizzle, 4-bit
// tiles whole rows 288 bytes apart; the order of the positions is the one in which both
// operands' reads touch every bank once.
#pragma once

#include "fa512_device.cuh"
#include "fa512_internal.h"

namespace fa512 {
namespace ranges {

constexpr int D = 512;
constexpr int WARPS = 4;                         // per group: blocks of 16 positions of a tile, or 128 columns of O
constexpr int KSTEPS = D / 16;
constexpr int MTILES = D / WARPS / 16;           // m-tiles of 16 columns a warp
constexpr int CODES = 256;                       // bytes of codes in a 4-bit row

template <int BITS>
struct Format {
    static constexpr int ROW = BITS == 16 ? 1024 : BITS == 8 ? 512 : kFp4RowBytes;   // bytes
    static constexpr int TILE = BITS == 16 ? 16 : BITS == 8 ? 32 : 64;               // positions, 16 to 18 KiB of K or V
    static constexpr int BLOCKS = TILE / 16;
    static constexpr int BOXES = BITS == 4 ? 1 : ROW / 128;                          // TMA boxes of a row
    static constexpr int SLOT = TILE * ROW;
    static constexpr int P_BUFFERS = BITS == 4 ? 2 : 4;                              // tiles whose P may be waiting
    // Position of M row r (0 .. 7) of a block's half
    __device__ static __forceinline__ int order(int r) { return BITS == 4 ? r ^ ((r >> 2) & 1) : r ^ ((r & 1) << 2); }
};

// Row of a block of 16 that lane t's i-th V operand is: the pairs (2 t, 2 t + 1)
// and (2 t + 8, 2 t + 9).
template <int BITS>
__device__ __forceinline__ int v_row(int t, int i) {
    return Format<BITS>::order(2 * t + (i & 1)) + 8 * (i >> 1);
}

// 16-byte piece of row `row` of a box of 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ const uint4* piece(const uint8_t* box, int row, int c) {
    return reinterpret_cast<const uint4*>(box + row * 128 + ((c ^ (row & 7)) << 4));
}

// Four bytes of two codes each -> four f16x2, exactly (low half of the byte first).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 values (low byte first) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
    return h;
}

__device__ __forceinline__ float f16_f32(uint32_t h) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<unsigned short>(h)));
    return f;
}

__device__ __forceinline__ uint32_t prmt(uint32_t x, uint32_t y, uint32_t sel) {
    uint32_t t;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(t) : "r"(x), "r"(y), "r"(sel));
    return t;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Weights of the rows' P: a pair rounded to the type of the product, and times a pair.
template <int BITS>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
    return BITS == 16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
template <int BITS>
__device__ __forceinline__ uint32_t mul_p(uint32_t a, uint32_t b) {
    if constexpr (BITS != 16) return mul_f16x2(a, b);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t LOW_HALVES = 0x0f0f0f0fu;

// 4 bits: S^T of a block of 16 positions, scales applied to the codes; Q fragments in
// shared memory.  b0/b1 of k-step 4 j + s are a row's elements
// 64 j + 16 t + 4 s + {0, 1} / {2, 3}.
template <int NT>
__device__ __forceinline__ void scores_4(const uint8_t* block, int lane, const uint2* s_q, float (&sc)[NT][4]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t *a_row = block + Format<4>::order(g) * Format<4>::ROW, *b_row = a_row + 8 * Format<4>::ROW;
    const uint32_t pick = static_cast<uint32_t>(t) | (static_cast<uint32_t>(4 + t) << 4);
    float acc[NT][2][4];                          // two chains of sums
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][0][e] = acc[n][1][e] = 0.f;
#pragma unroll
    for (int j4 = 0; j4 < 2; ++j4) {
        // the rows' scales of 16 groups; this lane's are every fourth
        const uint4 xa = *reinterpret_cast<const uint4*>(a_row + CODES + 16 * j4);
        const uint4 xb = *reinterpret_cast<const uint4*>(b_row + CODES + 16 * j4);
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
            const uint32_t sa = e4m3x2_f16(prmt(wa[2 * j2], wa[2 * j2 + 1], pick) & 0xffffu);
            const uint32_t sb = e4m3x2_f16(prmt(wb[2 * j2], wb[2 * j2 + 1], pick) & 0xffffu);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 4 * j4 + 2 * j2 + h;
                const uint32_t fa = prmt(sa, sa, h ? 0x3232u : 0x1010u), fb = prmt(sb, sb, h ? 0x3232u : 0x1010u);
                const uint2 ca = *reinterpret_cast<const uint2*>(a_row + 32 * j + 8 * t);
                const uint2 cb = *reinterpret_cast<const uint2*>(b_row + 32 * j + 8 * t);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t ha[4], hb[4];
                    e2m1x8_f16(x ? ca.y : ca.x, ha);
                    e2m1x8_f16(x ? cb.y : cb.x, hb);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int k = 4 * j + 2 * x + s;
                        const uint32_t a0 = mul_f16x2(ha[2 * s], fa), a2 = mul_f16x2(ha[2 * s + 1], fa);
                        const uint32_t a1 = mul_f16x2(hb[2 * s], fb), a3 = mul_f16x2(hb[2 * s + 1], fb);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 q2 = s_q[(n * KSTEPS + k) * 32 + lane];
                            mma_f16(acc[n][k & 1], a0, a1, a2, a3, q2.x, q2.y);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = acc[n][0][e] + acc[n][1][e];
}

// The same for up to 2 rows: column 2 c + r of Q^T holds row r's elements of the
// groups 4 j + c, and zeros.  A lane's sums of step j are those of group 4 j + t.
__device__ __forceinline__ void scores_narrow(const uint8_t* block, int lane, const uint2* s_q, float (&sc)[4]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t *a_row = block + Format<4>::order(g) * Format<4>::ROW, *b_row = a_row + 8 * Format<4>::ROW;
    const uint32_t pick = static_cast<uint32_t>(t) | (static_cast<uint32_t>(4 + t) << 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = 0.f;
#pragma unroll
    for (int j4 = 0; j4 < 2; ++j4) {
        const uint4 xa = *reinterpret_cast<const uint4*>(a_row + CODES + 16 * j4);
        const uint4 xb = *reinterpret_cast<const uint4*>(b_row + CODES + 16 * j4);
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
            const uint32_t sa = e4m3x2_f16(prmt(wa[2 * j2], wa[2 * j2 + 1], pick) & 0xffffu);
            const uint32_t sb = e4m3x2_f16(prmt(wb[2 * j2], wb[2 * j2 + 1], pick) & 0xffffu);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = 4 * j4 + 2 * j2 + h;
                const uint2 ca = *reinterpret_cast<const uint2*>(a_row + 32 * j + 8 * t);
                const uint2 cb = *reinterpret_cast<const uint2*>(b_row + 32 * j + 8 * t);
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t ha[4], hb[4];
                    e2m1x8_f16(x ? ca.y : ca.x, ha);
                    e2m1x8_f16(x ? cb.y : cb.x, hb);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint2 q2 = s_q[(4 * j + 2 * x + s) * 32 + lane];
                        mma_f16(d, ha[2 * s], hb[2 * s], ha[2 * s + 1], hb[2 * s + 1], q2.x, q2.y);
                    }
                }
                const float fa = f16_f32(h ? sa >> 16 : sa), fb = f16_f32(h ? sb >> 16 : sb);
                sc[0] = fmaf(fa, d[0], sc[0]);
                sc[1] = fmaf(fa, d[1], sc[1]);
                sc[2] = fmaf(fb, d[2], sc[2]);
                sc[3] = fmaf(fb, d[3], sc[3]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {                 // the four classes
        sc[e] += __shfl_xor_sync(0xffffffffu, sc[e], 1);
        sc[e] += __shfl_xor_sync(0xffffffffu, sc[e], 2);
    }
}

// O^T of columns 128 warp .. + 127 += V^T P^T over a block, scales applied to the codes;
// m-tile i is columns 16 g + 2 i, 16 g + 2 i + 1 of those.  (Multiplying
// the weights by the scales instead takes 4 multiplications a block for up to 2 rows where
// this takes 32, but the products do not fit f16: 18 binades of scales times the weights'
// own.  It is no faster either, 621 and 626 us for 64 x 28,672 positions.)
template <int NT>
__device__ __forceinline__ void add_values_4(const uint8_t* block, int warp, int lane, const uint32_t (&pb)[NT][2],
                                           float (&o)[NT][MTILES][4]) {
    const int g = lane >> 2, t = lane & 3;
    uint2 c[4];
    uint32_t sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* row = block + v_row<4>(t, i) * Format<4>::ROW;
        c[i] = *reinterpret_cast<const uint2*>(row + 64 * warp + 8 * g);
        sb[i] = row[CODES + 8 * warp + g];
    }
    const uint32_t s01 = e4m3x2_f16(prmt(sb[0], sb[1], 0x0040u)), s23 = e4m3x2_f16(prmt(sb[2], sb[3], 0x0040u));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint32_t w0 = x ? c[0].y : c[0].x, w1 = x ? c[1].y : c[1].x;
        const uint32_t w2 = x ? c[2].y : c[2].x, w3 = x ? c[3].y : c[3].x;
        // bytes of two rows' codes of one column: even columns, odd columns
        uint32_t e01[4], d01[4], e23[4], d23[4];
        e2m1x8_f16((w0 & LOW_HALVES) | ((w1 << 4) & ~LOW_HALVES), e01);
        e2m1x8_f16(((w0 >> 4) & LOW_HALVES) | (w1 & ~LOW_HALVES), d01);
        e2m1x8_f16((w2 & LOW_HALVES) | ((w3 << 4) & ~LOW_HALVES), e23);
        e2m1x8_f16(((w2 >> 4) & LOW_HALVES) | (w3 & ~LOW_HALVES), d23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = mul_f16x2(e01[i], s01), a1 = mul_f16x2(d01[i], s01);
            const uint32_t a2 = mul_f16x2(e23[i], s23), a3 = mul_f16x2(d23[i], s23);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * x + i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
    }
}

// E4M3: the same, from a slot of boxes of TILE rows; the operands' elements as in 4 bits.
template <int NT>
__device__ __forceinline__ void scores_8(const uint8_t* slot, int first, int lane,
                                         const uint2* s_q, float (&sc)[NT][4]) {
    const int g = lane >> 2, t = lane & 3;
    const int row = first + Format<8>::order(g);
    float acc[NT][2][4];                          // two chains of sums
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][0][e] = acc[n][1][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint8_t* box = slot + (j >> 1) * Format<8>::TILE * 128;
        const uint4 a = *piece(box, row, 4 * (j & 1) + t), b = *piece(box, row + 8, 4 * (j & 1) + t);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = 4 * j + s;
            const uint32_t a0 = e4m3x2_f16(wa[s] & 0xffffu), a2 = e4m3x2_f16(wa[s] >> 16);
            const uint32_t a1 = e4m3x2_f16(wb[s] & 0xffffu), a3 = e4m3x2_f16(wb[s] >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 q2 = s_q[(n * KSTEPS + k) * 32 + lane];
                mma_f16(acc[n][k & 1], a0, a1, a2, a3, q2.x, q2.y);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = acc[n][0][e] + acc[n][1][e];
}

// m-tile i is columns 16 g + 2 i, 16 g + 2 i + 1 of the warp's 128, its box.
template <int NT>
__device__ __forceinline__ void add_values_8(const uint8_t* slot, int first, int warp, int lane, const uint32_t (&pb)[NT][2],
                                             float (&o)[NT][MTILES][4]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* box = slot + warp * Format<8>::TILE * 128;
    uint32_t v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 x = *piece(box, first + v_row<8>(t, i), g);
        v[i][0] = x.x;
        v[i][1] = x.y;
        v[i][2] = x.z;
        v[i][3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < MTILES; ++i) {
        // two positions' bytes of one column
        const uint32_t even = i & 1 ? 0x0062u : 0x0040u, odd = i & 1 ? 0x0073u : 0x0051u;
        const uint32_t a0 = e4m3x2_f16(prmt(v[0][i >> 1], v[1][i >> 1], even) & 0xffffu);
        const uint32_t a1 = e4m3x2_f16(prmt(v[0][i >> 1], v[1][i >> 1], odd) & 0xffffu);
        const uint32_t a2 = e4m3x2_f16(prmt(v[2][i >> 1], v[3][i >> 1], even) & 0xffffu);
        const uint32_t a3 = e4m3x2_f16(prmt(v[2][i >> 1], v[3][i >> 1], odd) & 0xffffu);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(o[n][i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
    }
}

// bf16: b0/b1 of k-step 2 j + s are a row's elements 32 j + 8 t + 4 s + {0, 1} / {2, 3}.
template <int NT>
__device__ __forceinline__ void scores_16(const uint8_t* slot, int lane, const uint2* s_q, float (&sc)[NT][4]) {
    const int g = lane >> 2, t = lane & 3;
    const int row = Format<16>::order(g);
    float acc[NT][2][4];                          // two chains of sums
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][0][e] = acc[n][1][e] = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint8_t* box = slot + (j >> 1) * Format<16>::TILE * 128;
        const uint4 a = *piece(box, row, 4 * (j & 1) + t), b = *piece(box, row + 8, 4 * (j & 1) + t);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = 2 * j + s;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 q2 = s_q[(n * KSTEPS + k) * 32 + lane];
                mma_bf16_16816(acc[n][s], {s ? a.z : a.x, s ? b.z : b.x, s ? a.w : a.y, s ? b.w : b.y}, q2.x, q2.y);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = acc[n][0][e] + acc[n][1][e];
}

// m-tile 4 h + i is columns 64 h + 8 g + 2 i, + 1 of the warp's 128, its two boxes.
template <int NT>
__device__ __forceinline__ void add_values_16(const uint8_t* slot, int warp, int lane, const uint32_t (&pb)[NT][2],
                                              float (&o)[NT][MTILES][4]) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t* box = slot + (2 * warp + h) * Format<16>::TILE * 128;
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = *piece(box, v_row<16>(t, i), g);
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = prmt(v[0][i], v[1][i], 0x5410u), a1 = prmt(v[0][i], v[1][i], 0x7632u);
            const uint32_t a2 = prmt(v[2][i], v[3][i], 0x5410u), a3 = prmt(v[2][i], v[3][i], 0x7632u);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_bf16_16816(o[n][4 * h + i], {a0, a1, a2, a3}, pb[n][0], pb[n][1]);
        }
    }
}

}  // namespace ranges
}  // namespace fa512
