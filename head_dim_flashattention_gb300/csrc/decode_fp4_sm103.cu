// Paged split-K decode over a cache held in 4 bits, sm_103a.
//
// A row of one head and position is 288 bytes: 256 bytes of E2M1 codes (element
// 2 i in the low half of byte i) and 32 E4M3 scales, one for 16 elements, so a
// position costs 576 bytes of K and V where bf16 costs 2,048.  An element is
// tensor scale * group scale * code; group scale times code has 6 significant
// bits and lies between 2^-10 and 2,688, so it is exact in f16, and the products
// run on mma.sync with f16 operands and fp32 sums over the cache's exact values.
//
// A CTA of four warps takes one split of the keys of a (sequence, KV head) in
// tiles of 64 positions, K and V rows brought by TMA into two slots each.  For a
// tile, warp w forms S^T = K Q^T of positions 16 w .. 16 w + 15 over the whole
// head dim, with the query rows in N, their softmax against a reference of its
// own, and leaves P^T and the reference in shared memory; after one barrier every
// warp adds V^T P^T of all 64 positions for its 128 columns of O.  So nothing is
// computed twice, and the four warps meet once in 64 positions.  References are
// whole numbers in log2 units: what brings two of them together is a power of
// two, exact in f16.
//
// K pairs are neighbouring codes of a row, as stored.  A V pair is the codes of
// one column in two rows: a shift and a bit select turn two rows' words into
// bytes that hold such pairs.  Within a group of 8 positions a lane's rows are
// taken in the order 0 1 2 3 5 4 7 6, with which both operands' shared-memory
// reads (rows 288 bytes apart) touch every bank once.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_list.cuh"

namespace fa512 {
namespace fp4 {

constexpr int D = 512;
constexpr int ROW = kFp4RowBytes;
constexpr int CODES = 256;                       // bytes of codes in a row
constexpr int TILE = 64;                         // positions per tile
constexpr int WARPS = 4;                         // 16 positions of a tile and 128 columns of O each
constexpr int THREADS = WARPS * 32;
constexpr int SLOT = TILE * ROW;                 // 18,432 bytes
constexpr int KSTEPS = D / 16;
constexpr int MTILES = D / WARPS / 16;           // m-tiles of 16 columns a warp
constexpr int META = 4;                          // tiles whose positions are kept

__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

template <int NT>
struct Smem {
    static constexpr int k = 0;                              // 2 slots
    static constexpr int v = 2 * SLOT;                       // 2 slots
    static constexpr int p = 4 * SLOT;                       // [parity][block][nt][lane] uint2
    static constexpr int q = p + 2 * WARPS * NT * 32 * 8;    // NT = 2: [nt][kstep][lane] uint2
    static constexpr int ref = q + (NT == 2 ? NT * KSTEPS * 32 * 8 : 0);   // [parity][block][8 NT] float
    static constexpr int lsum = ref + 2 * WARPS * 8 * NT * 4;              // [warp][8 NT] float
    static constexpr int base = lsum + WARPS * 8 * NT * 4;                 // [META][4] first position of 16
    static constexpr int row = base + META * 16;                           // [META][4] first row of a run
    static constexpr int bar = row + META * 16;                            // K slots, V slots
    static constexpr int total = bar + 4 * 8;
};
static_assert(3 * (Smem<1>::total + 1024) <= 228 * 1024, "three CTAs fit an SM's shared memory");
static_assert(2 * (Smem<2>::total + 1024) <= 228 * 1024, "two CTAs fit an SM's shared memory");

__device__ __forceinline__ int turned(int r) { return r ^ ((r >> 2) & 1); }

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

// NT: 1 for up to 8 query rows (q_len * G) of a KV head, whose fragments stay in
// registers, 2 for up to 16, whose fragments are read from shared memory.
template <int NT, bool LIST>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(NT))
decode_fp4_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const DecodeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using Smem = fp4::Smem<NT>;
    extern __shared__ __align__(128) uint8_t fp4_smem[];
    uint8_t* smem = fp4_smem;
    uint2* s_p = reinterpret_cast<uint2*>(smem + Smem::p);
    uint2* s_q = reinterpret_cast<uint2*>(smem + Smem::q);
    float* s_ref = reinterpret_cast<float*>(smem + Smem::ref);
    float* s_l = reinterpret_cast<float*>(smem + Smem::lsum);
    int* s_base = reinterpret_cast<int*>(smem + Smem::base);
    int* s_row = reinterpret_cast<int*>(smem + Smem::row);
    uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + Smem::bar);
    uint64_t* bar_v = bar_k + 2;

    const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;       // mma fragment coordinates
    const int G = p.group, R = p.q_len * G;      // query rows: (token, head) -> token * G + head
    const int ps = p.page_size;

    int len = p.kv_lens[b];
    if (len < 0 || len > p.len_cap) {
        if (threadIdx.x == 0 && split == 0 && kvh == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        len = len < 0 ? 0 : p.len_cap;
    }
    // union of the rows' bands (the row of token t sees [pos - window + 1, pos])
    const int hi = len;
    const int w_lo = len - p.q_len + 1 - p.window;
    const int lo = (p.window > 0 && w_lo > 0) ? w_lo : 0;
    // the split's positions: absolute, or counted along the list of pages
    const int32_t* list = LIST ? list_of(p, b, kvh) : nullptr;
    int v0, v1;
    if constexpr (LIST) {
        const long long first = static_cast<long long>(split) * p.tiles_per_split * TILE;
        const int all = p.n_listed * ps;
        v0 = static_cast<int>(min(first, static_cast<long long>(all)));
        v1 = static_cast<int>(min(first + static_cast<long long>(p.tiles_per_split) * TILE, static_cast<long long>(all)));
        v1 = list_end(p, list, v0, v1);
    } else {
        const long long first = static_cast<long long>(lo / TILE + static_cast<long long>(split) * p.tiles_per_split) * TILE;
        v0 = static_cast<int>(min(first, static_cast<long long>(hi)));
        v1 = static_cast<int>(min(first + static_cast<long long>(p.tiles_per_split) * TILE, static_cast<long long>(hi)));
    }
    const int n_tiles = v1 > v0 ? (v1 - v0 + TILE - 1) / TILE : 0;
    const int held = (len + ps - 1) / ps;        // pages of the sequence

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_k[i], 1);
            mbar_init(&bar_v[i], 1);
        }
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    __syncthreads();

    // ---- loads, by warp 0.  A run is box_rows positions of one page; lane l
    // keeps the first row and position of runs run0 + l (cur) and run0 + 32 + l.
    const int box = p.box_rows, runs_per_tile = TILE / box, blocks_per_run = box / 16;
    const int n_runs = n_tiles * runs_per_tile;
    int run0 = 0, row_cur = -1, base_cur = -1, row_nxt = -1, base_nxt = -1;
    auto look_up = [&](int r, int& row, int& base) {
        row = base = -1;
        if (r >= n_runs) return;
        const int v = v0 + r * box;
        int lp = v / ps, at = v;
        if constexpr (LIST) {
            if (v >= v1) return;
            const int off = v - lp * ps;
            lp = list_page(p, list, lp, held);
            if (lp < 0) return;
            at = lp * ps + off;
        }
        if (at >= hi || at + box <= lo) return;
        const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
        if (page < 0 || page >= p.num_pages) {
            report_error(p.err, FA512_DEVICE_ERR_INDEX);
            return;
        }
        row = page * ps + (at - lp * ps);
        base = at;
    };
    // K rows of tile i into their slot; what the V load and the masks need is kept
    auto load_k = [&](int i) {
        if (i >= n_tiles) return;
        const int r = i * runs_per_tile;
        if (r >= run0 + 32) {
            run0 += 32;
            row_cur = row_nxt;
            base_cur = base_nxt;
            look_up(run0 + 32 + lane, row_nxt, base_nxt);
        }
        const int l = (r - run0) + lane / blocks_per_run;      // lanes 0 .. 3: their 16 positions' run
        const int base = __shfl_sync(0xffffffffu, base_cur, l & 31);
        const int slot = (i & (META - 1)) * 4;
        if (lane < 4) s_base[slot + lane] = base < 0 ? -1 : base + 16 * (lane % blocks_per_run);
        const int run_row = __shfl_sync(0xffffffffu, row_cur, (r - run0 + lane) & 31);
        const unsigned some = __ballot_sync(0xffffffffu, lane < runs_per_tile && run_row >= 0);
        if (lane < runs_per_tile) s_row[slot + lane] = run_row;
        __syncwarp();
        uint64_t* bar = &bar_k[i & 1];
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(some) * box * ROW);
        __syncwarp();
        if (lane < runs_per_tile && run_row >= 0)
            tma_load_3d(smem + Smem::k + (i & 1) * SLOT + lane * box * ROW, &tmk, bar, 0, kvh, run_row);
    };
    auto load_v = [&](int i) {
        if (i >= n_tiles) return;
        const int run_row = lane < runs_per_tile ? s_row[(i & (META - 1)) * 4 + lane] : -1;
        const unsigned some = __ballot_sync(0xffffffffu, run_row >= 0);
        uint64_t* bar = &bar_v[i & 1];
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(some) * box * ROW);
        __syncwarp();
        if (run_row >= 0)
            tma_load_3d(smem + Smem::v + (i & 1) * SLOT + lane * box * ROW, &tmv, bar, 0, kvh, run_row);
    };
    if (warp == 0) {
        look_up(lane, row_cur, base_cur);
        look_up(32 + lane, row_nxt, base_nxt);
        load_k(0);
        load_v(0);
        load_k(1);
        load_v(1);
    }

    // ---- Q^T fragments: b0/b1 of k-step 4 j + s hold row g's elements 64 j + 16
    // t + 4 s + {0, 1} / {2, 3}, in f16 after a power-of-two scale per row that
    // keeps its largest element below 2^15 (exact for elements down to 2^-39 of
    // that; a score is unscaled before the softmax)
    uint32_t qb[NT == 1 ? KSTEPS : 1][2];
    float rs[NT][2];                              // 1 / scale of rows 8 n + 2 t, 8 n + 2 t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // NT = 2: each warp holds a quarter of the k-steps, all of them the maxima
        const int r = 8 * n + g;
        const bool row_ok = r < R;
        const size_t qrow = (static_cast<size_t>(b) * p.q_len + (row_ok ? r / G : 0)) * p.n_q_heads + kvh * G +
                            (row_ok ? r % G : 0);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + qrow * D);
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint4 a = row_ok ? src[8 * j + 2 * t + e] : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
                if constexpr (NT == 1) {
                    qb[4 * j + 2 * e][0] = a.x;
                    qb[4 * j + 2 * e][1] = a.y;
                    qb[4 * j + 2 * e + 1][0] = a.z;
                    qb[4 * j + 2 * e + 1][1] = a.w;
                }
            }
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // 2^(14 - E), E = exponent of the maximum (0 or not finite: 1)
        const int E = (__float_as_uint(most) >> 23) & 0xff;
        const int biased = min(127 + 14 + 127 - E, 254);
        const float scale = (most > 0.f && E < 255) ? __uint_as_float(static_cast<uint32_t>(biased) << 23) : 1.f;
        auto to_f16 = [&](uint32_t w) {
            return pack_f16x2(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xffff0000u) * scale);
        };
        if constexpr (NT == 1) {
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
                qb[k][0] = to_f16(qb[k][0]);
                qb[k][1] = to_f16(qb[k][1]);
            }
        } else {
#pragma unroll
            for (int j = 2 * warp; j < 2 * warp + 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 a = row_ok ? src[8 * j + 2 * t + e] : make_uint4(0u, 0u, 0u, 0u);
                    s_q[(n * KSTEPS + 4 * j + 2 * e) * 32 + lane] = make_uint2(to_f16(a.x), to_f16(a.y));
                    s_q[(n * KSTEPS + 4 * j + 2 * e + 1) * 32 + lane] = make_uint2(to_f16(a.z), to_f16(a.w));
                }
        }
        rs[n][0] = 1.f / __shfl_sync(0xffffffffu, scale, 4 * (2 * t));
        rs[n][1] = 1.f / __shfl_sync(0xffffffffu, scale, 4 * (2 * t + 1));
    }
    if constexpr (NT == 2) __syncthreads();

    // positions of rows 8 n + 2 t + i (-1: padding row, sees nothing); a row sees
    // the keys whose distance to it is in [0, reach)
    int qpos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * n + 2 * t + i;
            qpos[n][i] = r < R ? len - p.q_len + r / G : -1;
        }
    const unsigned reach = p.window > 0 ? static_cast<unsigned>(p.window) : 0x7fffffffu;

    float m[NT][2], mg[NT], l[NT][2];             // references of rows 2 t + i and g; this lane's part of the sums
    float o[NT][MTILES][4];                       // O^T: m-tile i = columns 16 g + 2 i, 16 g + 2 i + 1 of this warp's 128
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = mg[n] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MTILES; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }
    auto finite_ref = [](float x) { return x == -INFINITY ? 0.f : x; };   // nothing seen yet: 2^(-inf - 0) = 0

    const int ra = turned(g);                     // this lane's rows of 16 positions: ra, ra + 8
    bool ok = true;
    int done = 0;
    for (int it = 0; it < n_tiles; ++it) {
        const int par = it & 1, phase = (it >> 1) & 1;
        const int* base4 = s_base + (it & (META - 1)) * 4;
        if (!mbar_wait(&bar_k[par], phase, p.err)) ok = false;

        // ---- S^T of this warp's 16 positions, softmax against their own maximum
        {
            const int base = base4[warp];
            float sc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
            if (base >= 0) {
                const uint8_t* a_row = smem + Smem::k + par * SLOT + (16 * warp + ra) * ROW;
                const uint8_t* b_row = a_row + 8 * ROW;
                uint32_t wa[8], wb[8];            // the rows' scales
                {
                    const uint4 x = *reinterpret_cast<const uint4*>(a_row + CODES);
                    const uint4 y = *reinterpret_cast<const uint4*>(a_row + CODES + 16);
                    const uint4 z = *reinterpret_cast<const uint4*>(b_row + CODES);
                    const uint4 w = *reinterpret_cast<const uint4*>(b_row + CODES + 16);
                    wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w; wa[4] = y.x; wa[5] = y.y; wa[6] = y.z; wa[7] = y.w;
                    wb[0] = z.x; wb[1] = z.y; wb[2] = z.z; wb[3] = z.w; wb[4] = w.x; wb[5] = w.y; wb[6] = w.z; wb[7] = w.w;
                }
                const uint32_t pick = static_cast<uint32_t>(t) | (static_cast<uint32_t>(4 + t) << 4);
                float other[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) other[n][0] = other[n][1] = other[n][2] = other[n][3] = 0.f;
#pragma unroll
                for (int j2 = 0; j2 < 4; ++j2) {
                    const uint32_t sa = e4m3x2_f16(prmt(wa[2 * j2], wa[2 * j2 + 1], pick) & 0xffffu);
                    const uint32_t sb = e4m3x2_f16(prmt(wb[2 * j2], wb[2 * j2 + 1], pick) & 0xffffu);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = 2 * j2 + h;
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
                                    uint32_t b0, b1;
                                    if constexpr (NT == 1) {
                                        b0 = qb[k][0];
                                        b1 = qb[k][1];
                                    } else {
                                        const uint2 q2 = s_q[(n * KSTEPS + k) * 32 + lane];
                                        b0 = q2.x;
                                        b1 = q2.y;
                                    }
                                    mma_f16(h ? other[n] : sc[n], a0, a1, a2, a3, b0, b1);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] += other[n][e];
            }
            const int kp = base + ra;
            float* ref = s_ref + (par * WARPS + warp) * 8 * NT;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float sv[2][2], cm[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool va = base >= 0 && static_cast<unsigned>(qpos[n][i] - kp) < reach;
                    const bool vb = base >= 0 && static_cast<unsigned>(qpos[n][i] - kp - 8) < reach;
                    sv[i][0] = va ? sc[n][i] * rs[n][i] * p.scale_log2 : -INFINITY;
                    sv[i][1] = vb ? sc[n][2 + i] * rs[n][i] * p.scale_log2 : -INFINITY;
                    cm[i] = fmaxf(sv[i][0], sv[i][1]);
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    const float x0 = __shfl_xor_sync(0xffffffffu, cm[0], off);
                    const float x1 = __shfl_xor_sync(0xffffffffu, cm[1], off);
                    cm[0] = fmaxf(cm[0], x0);
                    cm[1] = fmaxf(cm[1], x1);
                }
                float pr[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    cm[i] = ceilf(cm[i]);
                    const float sh = finite_ref(cm[i]);
                    pr[i][0] = fast_exp2(sv[i][0] - sh);
                    pr[i][1] = fast_exp2(sv[i][1] - sh);
                }
                // P rounds to f16 (2^-12 of a weight, 2^-25 of the largest one's
                // block); the sums keep the fp32 values
                const uint32_t b0 = transpose8x8(pack_f16x2(pr[0][0], pr[1][0]));
                const uint32_t b1 = transpose8x8(pack_f16x2(pr[0][1], pr[1][1]));
                s_p[((par * WARPS + warp) * NT + n) * 32 + lane] = make_uint2(b0, b1);
                if (g == 0) *reinterpret_cast<float2*>(ref + 8 * n + 2 * t) = make_float2(cm[0], cm[1]);
                // this lane's part of the sums, until all references are known
                sc[n][0] = pr[0][0] + pr[0][1];
                sc[n][1] = pr[1][0] + pr[1][1];
                sc[n][2] = cm[0];
                sc[n][3] = cm[1];
            }
            if (__syncthreads_or(!ok)) {
                ok = false;
                break;
            }
            if (warp == 0) {
                load_k(it + 2);                   // K of this tile is read, V of the last one too
                if (it > 0) load_v(it + 1);
            }
            // ---- one reference for the tile
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float* all = s_ref + par * WARPS * 8 * NT + 8 * n;
                float mn[2] = {m[n][0], m[n][1]};
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float2 x = *reinterpret_cast<const float2*>(all + w * 8 * NT + 2 * t);
                    mn[0] = fmaxf(mn[0], x.x);
                    mn[1] = fmaxf(mn[1], x.y);
                }
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sh = finite_ref(mn[i]);
                    al[i] = fast_exp2(m[n][i] - sh);
                    l[n][i] = l[n][i] * al[i] + sc[n][i] * fast_exp2(sc[n][2 + i] - sh);
                    m[n][i] = mn[i];
                }
                if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
                    for (int i = 0; i < MTILES; ++i) {
                        o[n][i][0] *= al[0];
                        o[n][i][1] *= al[1];
                        o[n][i][2] *= al[0];
                        o[n][i][3] *= al[1];
                    }
                }
#pragma unroll
                for (int w = 0; w < WARPS; ++w) mg[n] = fmaxf(mg[n], all[w * 8 * NT + g]);
            }
        }
        if (!mbar_wait(&bar_v[par], phase, p.err)) ok = false;

        // ---- O^T += V^T P^T for this warp's columns, 16 positions at a time
        const uint8_t* vst = smem + Smem::v + par * SLOT;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int base = base4[w];
            if (base < 0) continue;
            uint32_t pb[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float f = fast_exp2(s_ref[(par * WARPS + w) * 8 * NT + 8 * n + g] - finite_ref(mg[n]));
                const uint32_t f2 = pack_f16x2(f, f);
                const uint2 x = s_p[((par * WARPS + w) * NT + n) * 32 + lane];
                pb[n][0] = mul_f16x2(x.x, f2);
                pb[n][1] = mul_f16x2(x.y, f2);
            }
            // rows of the pairs (2 t, 2 t + 1) and (2 t + 8, 2 t + 9); a position that no
            // row sees gets the scale 0 (its bytes may be anything: codes are finite)
            uint2 c[4];
            uint32_t sb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = turned(2 * t + (i & 1)) + 8 * (i >> 1);
                const uint8_t* row = vst + (16 * w + r) * ROW;
                c[i] = *reinterpret_cast<const uint2*>(row + 64 * warp + 8 * g);
                const uint32_t s = row[CODES + 8 * warp + g];
                sb[i] = base + r < hi && base + r >= lo ? s : 0u;
            }
            const uint32_t s01 = e4m3x2_f16(sb[0] | (sb[1] << 8)), s23 = e4m3x2_f16(sb[2] | (sb[3] << 8));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t w0 = x ? c[0].y : c[0].x, w1 = x ? c[1].y : c[1].x;
                const uint32_t w2 = x ? c[2].y : c[2].x, w3 = x ? c[3].y : c[3].x;
                // bytes of two rows' codes of one column: even columns, odd columns
                constexpr uint32_t LOW = 0x0f0f0f0fu;
                uint32_t e01[4], d01[4], e23[4], d23[4];
                e2m1x8_f16((w0 & LOW) | ((w1 << 4) & ~LOW), e01);
                e2m1x8_f16(((w0 >> 4) & LOW) | (w1 & ~LOW), d01);
                e2m1x8_f16((w2 & LOW) | ((w3 << 4) & ~LOW), e23);
                e2m1x8_f16(((w2 >> 4) & LOW) | (w3 & ~LOW), d23);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = mul_f16x2(e01[i], s01), a1 = mul_f16x2(d01[i], s01);
                    const uint32_t a2 = mul_f16x2(e23[i], s23), a3 = mul_f16x2(d23[i], s23);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * x + i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                }
            }
        }
        done = it + 1;
    }
    // A wait that ran out: bounded waits for the copies in flight, so that none
    // lands after this CTA has gone.  `done` tiles were gone through; the V wait of
    // the last one may be the one that ran out.
    if (__syncthreads_or(!ok)) {
        ok = false;
        if (threadIdx.x == 0)
            for (int i = max(done - 1, 0); i < n_tiles && i < done + 2; ++i) {
                if (i >= done) mbar_wait(&bar_k[i & 1], (i >> 1) & 1, p.err);
                mbar_wait(&bar_v[i & 1], (i >> 1) & 1, p.err);
            }
    }

    // ---- this split's partial, unnormalised and times v_scale
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], off);
            if (g == 0) s_l[warp * 8 * NT + 8 * n + 2 * t + i] = l[n][i];
        }
    __syncthreads();
    const size_t S = static_cast<size_t>(p.num_splits);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * n + 2 * t + i;
            if (r >= R) continue;
            const size_t hq = (static_cast<size_t>(b) * p.q_len + r / G) * p.n_q_heads + kvh * G + r % G;
            float4* dst = reinterpret_cast<float4*>(p.ws_o + (hq * S + split) * D + 128 * warp + 16 * g);
            const float f = ok ? p.o_scale : 0.f;
#pragma unroll
            for (int j = 0; j < MTILES / 2; ++j)
                dst[j] = make_float4(o[n][2 * j][i] * f, o[n][2 * j][2 + i] * f, o[n][2 * j + 1][i] * f,
                                     o[n][2 * j + 1][2 + i] * f);
            if (warp == 0 && g == 0) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) sum += s_l[w * 8 * NT + r];
                float ref = m[n][i];
                if (sum != sum && ref == -INFINITY) ref = 0.f;   // only scores of NaN: not an empty split
                p.ws_ml[(hq * S + split) * 2 + 0] = ok ? ref : -INFINITY;
                p.ws_ml[(hq * S + split) * 2 + 1] = ok && ref != -INFINITY ? sum : 0.f;
            }
        }
}

template <int NT, bool LIST>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(decode_fp4_kernel<NT, LIST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Smem<NT>::total);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.num_splits, p.n_kv_heads, p.batch);
    decode_fp4_kernel<NT, LIST><<<grid, THREADS, Smem<NT>::total, stream>>>(tmk, tmv, p);
    return cudaGetLastError();
}

}  // namespace fp4

int decode_fp4_tile_positions() { return fp4::TILE; }
int decode_fp4_ctas_per_sm(int rows) { return fp4::ctas_per_sm(rows <= 8 ? 1 : 2); }

cudaError_t launch_decode_fp4(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p,
                              cudaStream_t stream) {
    const bool two = p.q_len * p.group > 8;
    const cudaError_t e = p.listed ? (two ? fp4::launch<2, true>(tmk, tmv, p, stream) : fp4::launch<1, true>(tmk, tmv, p, stream))
                                   : (two ? fp4::launch<2, false>(tmk, tmv, p, stream) : fp4::launch<1, false>(tmk, tmv, p, stream));
    return e != cudaSuccess ? e : launch_decode_merge(p, stream);
}

}  // namespace fa512
