// Which pages of a long cache a decode step reads, sm_103a: the bounds of each
// page's keys, and for each (sequence, KV head) the pages whose bounds allow the
// largest products with its queries.
//
//   bounds  lo[d], hi[d] = smallest and largest element d of a page's keys, which
//           bf16 holds exactly whatever the cache's format
//   score   of a page = max over the KV head's query rows of
//           sum_d max(q_d lo_d, q_d hi_d), no smaller than any q.k of the page
//   chosen  the n pages of largest score, equal ones by their number, the first
//           and last ones always
//
// The products of two bf16 values are exact in fp32, and the order in which a
// score's sum is taken is fixed (channels c and c + 256, then the eight of c / 8
// by halves, then the 32 groups by halves), so the choice is the same on every
// card and for every launch shape.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fa512_device.cuh"
#include "fa512_internal.h"

namespace fa512 {
namespace select {

constexpr int D = 512;

// ------------------------------------------------------------------- bounds
//
// A block takes one touched page of one KV head; a thread 8 elements of a row (16
// of a coded one, in 4 bits those of one scale), the rows dealt to 4 groups of
// threads, 16 of them in flight, whose results meet in shared memory.  NaN elements
// make both bounds NaN.  The blocks of a page's heads, whose rows lie side by side, come
// one after another.  What it takes is the two look-ups before a block's first row, anew
// for the second wave of blocks (of 2,024 with work 1,216 are resident), and, in 4 bits,
// the arithmetic (24 conversions and comparisons for 16 elements): 8 sequences
// of up to 4,096 new tokens, 4 heads, 4 bits: 37 MB in 13.0 us from memory (six blocks an
// SM instead of eight: 13.9, five 14.2; E4M3 15.2 with seven, 15.9 with six, 15.7 with
// eight); one token of 16 sequences, bf16, 2.3 us.
__host__ __device__ constexpr int bounds_threads(int bits) { return bits == 16 ? 256 : 128; }

struct MinMax {
    uint32_t lo, hi;
};
template <bool F16>
__device__ __forceinline__ void widen_to(MinMax& m, uint32_t x) {
    if constexpr (F16) {
        asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(m.lo) : "r"(x));
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m.hi) : "r"(x));
    } else {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(m.lo) : "r"(x));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m.hi) : "r"(x));
    }
}

// f16x2 (a value of an 8-bit or 4-bit cache) -> bf16x2, exactly
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
    float a, b;
    asm("cvt.f32.f16 %0, %1;" : "=f"(a) : "h"(static_cast<unsigned short>(h & 0xffffu)));
    asm("cvt.f32.f16 %0, %1;" : "=f"(b) : "h"(static_cast<unsigned short>(h >> 16)));
    return pack_bf16x2(a, b);
}

template <int BITS>
__global__ void __launch_bounds__(bounds_threads(BITS), BITS == 16 ? 2 : BITS == 8 ? 7 : 8) bounds_kernel(const BoundsParams p) {
    constexpr int ROW = BITS == 16 ? 2 * D : BITS == 8 ? D : kFp4RowBytes;
    constexpr int PAIRS = BITS == 16 ? 4 : 8;       // x 2 elements of a thread
    constexpr int LANES = D / (2 * PAIRS);          // threads of a row: 64, 32
    constexpr int GROUPS = bounds_threads(BITS) / LANES;
    constexpr bool F16 = BITS != 16;
    __shared__ uint32_t s_lo[GROUPS - 1][D / 2], s_hi[GROUPS - 1][D / 2];
    const int b = blockIdx.y, h = blockIdx.x % p.n_kv_heads, nth = blockIdx.x / p.n_kv_heads;   // nth touched page
    const int len = p.kv_lens[b];
    const int n_new = p.q_lens ? p.q_lens[b] : p.q_len;
    if (n_new < 0 || n_new > p.q_len || len < n_new ||
        len > static_cast<long long>(p.max_pages_per_seq) * p.page_size) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int lp = (len - n_new) / p.page_size + nth;
    if (n_new == 0 || lp > (len - 1) / p.page_size) return;
    const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
    if (page < 0 || page >= p.num_pages) {
        if (h == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int live = min(p.page_size, len - lp * p.page_size);
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const unsigned step = static_cast<unsigned>(p.n_kv_heads) * ROW;  // bytes from a row to the next
    const uint8_t* src = p.k_pages + (static_cast<size_t>(page) * p.page_size * p.n_kv_heads + h) * ROW + (BITS == 4 ? 8 : 16) * u;
    const uint8_t* scales = src + 256 - 7 * u;
    MinMax m[PAIRS];
    const uint32_t inf = F16 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) m[i] = {inf, inf | 0x80008000u};
    constexpr int RUN = 16;                         // rows in flight of a thread
    for (int r0 = grp; r0 < live; r0 += RUN * GROUPS) {
        uint4 x[RUN];
        uint8_t scale[RUN];
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
            // (a row past the end is the last one again)
            const size_t at = static_cast<size_t>(static_cast<unsigned>(min(r0 + k * GROUPS, live - 1))) * step;
            if constexpr (BITS == 4) {
                const uint2 y = *reinterpret_cast<const uint2*>(src + at);
                x[k] = make_uint4(y.x, y.y, 0u, 0u);
                scale[k] = scales[at];
            } else {
                x[k] = *reinterpret_cast<const uint4*>(src + at);
            }
        }
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            if constexpr (BITS == 16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) widen_to<F16>(m[i], w[i]);
            } else if constexpr (BITS == 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t y;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)))));
                    widen_to<F16>(m[i], y);
                }
            } else {
                uint32_t s;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"(static_cast<unsigned short>(scale[k] * 0x101u)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t y[4];
                    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
                        : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                        : "r"(w[i]));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[j]) : "r"(s));
                        widen_to<F16>(m[4 * i + j], y[j]);
                    }
                }
            }
        }
    }
    if (grp > 0)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            s_lo[grp - 1][u * PAIRS + i] = m[i].lo;
            s_hi[grp - 1][u * PAIRS + i] = m[i].hi;
        }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
#pragma unroll
        for (int q = 0; q < GROUPS - 1; ++q) {
            const uint32_t lo = s_lo[q][u * PAIRS + i], hi = s_hi[q][u * PAIRS + i];
            if constexpr (F16) {
                asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(m[i].lo) : "r"(lo));
                asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m[i].hi) : "r"(hi));
            } else {
                asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(m[i].lo) : "r"(lo));
                asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m[i].hi) : "r"(hi));
            }
        }
        if constexpr (F16) {
            m[i].lo = f16x2_to_bf16x2(m[i].lo);
            m[i].hi = f16x2_to_bf16x2(m[i].hi);
        }
    }
    uint4* dst = reinterpret_cast<uint4*>(p.bounds + (static_cast<size_t>(page) * p.n_kv_heads + h) * 2 * D) + u * (PAIRS / 4);
#pragma unroll
    for (int i = 0; i < PAIRS; i += 4) {
        dst[i / 4] = make_uint4(m[i].lo, m[i + 1].lo, m[i + 2].lo, m[i + 3].lo);
        dst[D / 8 + i / 4] = make_uint4(m[i].hi, m[i + 1].hi, m[i + 2].hi, m[i + 3].hi);
    }
}

// ------------------------------------------------------------------- scores
//
// The bounds of a warp's pages come through a ring of its own in shared memory, a
// page (2 KiB) a stage; it scores two at a time.  Lane l holds channels 8 l .. 8 l +
// 7 and 256 + 8 l .. of them, goes through the query rows (in shared memory, as fp32)
// and keeps each page's largest score.  max(q lo, q hi) is max(q, 0) hi + min(q, 0)
// lo, of which one term is 0: two packed multiply-adds a pair of channels, and each
// sum below rounds once.
constexpr int SCORE_WARPS = 4;
constexpr int SCORE_PAGES = 2;
constexpr int SCORE_STAGES = 4;                      // pages in the ring, a multiple of SCORE_PAGES
// Blocks to spread the pages over, 12 for each SM of a GB300 (a third of them, or twice as
// many: 43 us a selection instead of 40).
constexpr int SCORE_BLOCKS = 12 * 152;
constexpr int PAGE_BYTES = 2 * D * 2;                // a page's bounds
// shared memory: the warps' rings, then the query rows as fp32
constexpr int score_smem(int rows) { return SCORE_WARPS * SCORE_STAGES * PAGE_BYTES + rows * D * 4; }

// Unsigned integers in the order of the scores, -0 and 0 equal.  Largest of all are the
// pages that are always chosen, then those with a NaN or infinite score: the formula
// above turns every bound that is not finite into one of the two.  (A NaN in a query
// makes all scores NaN, so the pages are chosen by their number.)
constexpr uint32_t KEY_ALWAYS = 0xffffffffu, KEY_NOT_FINITE = 0xfffffffeu;
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x || x == INFINITY) return KEY_NOT_FINITE;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int length_of(const SelectParams& p, int b, bool record) {
    int len = p.kv_lens[b];
    if (len < 0 || len > p.len_cap) {
        if (record) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        len = len < 0 ? 0 : p.len_cap;
    }
    return len;
}

__device__ __forceinline__ void unpack8(const uint4 x, float2 (&f)[4]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// max(q, 0) and min(q, 0), NaN of NaN
__device__ __forceinline__ float above_0(float q) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(q));
    return r;
}
__device__ __forceinline__ float below_0(float q) {
    float r;
    asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(q));
    return r;
}

// Sums over the lanes of N values at once, each by halves (lanes 16 apart, then 8, ...):
// lane l gets value l / (32 / N)'s.
template <int N>
__device__ __forceinline__ float sum_of(float (&v)[N], int lane) {
    int off = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n >>= 1, off >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) {                // values i and i + n
            const float other = __shfl_xor_sync(0xffffffffu, lane & off ? v[i] : v[i + n], off);
            v[i] = (lane & off ? v[i + n] : v[i]) + other;
        }
#pragma unroll
    for (; off >= 1; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}

// ROWS: query rows at a time, 2 for up to 2 rows (64 sequences of up to 448 pages, 4 heads:
// 38 us a selection, with 4 at a time 46), else 4 (8 rows: 69, with 2 72).
template <int ROWS>
__global__ void __launch_bounds__(SCORE_WARPS * 32) score_kernel(const SelectParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint8_t score_raw[];
    const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = score_raw + warp * SCORE_STAGES * PAGE_BYTES;
    // [row][half of the channels][4 of 8][lane]
    float4* s_q = reinterpret_cast<float4*>(score_raw + SCORE_WARPS * SCORE_STAGES * PAGE_BYTES);
    const int len = length_of(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int held = static_cast<int>((static_cast<unsigned>(len) + p.page_size - 1) / p.page_size);
    const int step = gridDim.x * SCORE_WARPS * SCORE_PAGES;
    if (blockIdx.x * SCORE_WARPS * SCORE_PAGES >= held || held <= p.n_select) return;   // all pages are chosen
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    // the i-th page of this warp; of its pool page: -1 none (always chosen, or past the
    // end), -2 outside the pool
    auto number = [&](int i) {
        return (blockIdx.x * SCORE_WARPS + warp) * SCORE_PAGES + (i / SCORE_PAGES) * step + i % SCORE_PAGES;
    };
    auto page_of = [&](int i) {
        const int lp = number(i);
        if (lp >= held || lp < p.n_first || lp >= held - p.n_last) return -1;
        const int page = table[lp];
        return page < 0 || page >= p.num_pages ? -2 : page;
    };
    // lane l keeps the pool pages of the 32 of this warp's pages from `batch` on
    int batch = 0, mine = page_of(lane);
    const uint8_t* head = reinterpret_cast<const uint8_t*>(p.bounds) + static_cast<size_t>(h) * PAGE_BYTES + lane * 16;
    const unsigned apart = static_cast<unsigned>(p.n_kv_heads) * PAGE_BYTES;   // from a page to the next
    auto load = [&](int i, int stage) {
        if (i >= batch + 32) {
            batch += 32;
            mine = page_of(batch + lane);
        }
        const int page = __shfl_sync(0xffffffffu, mine, i & 31);
        if (page >= 0) {
            const uint8_t* src = head + static_cast<size_t>(static_cast<unsigned>(page)) * apart;
            const uint32_t dst = smem_u32(ring + stage * PAGE_BYTES + lane * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * j), "l"(src + 512 * j) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return page;
    };
    int pages[SCORE_STAGES];                         // of the stages, the next one to be scored first
#pragma unroll
    for (int i = 0; i < SCORE_STAGES; ++i) pages[i] = load(i, i);

    const int R = p.q_len * p.group;
    const int r0 = max(0, p.q_len - len) * p.group;  // rows of tokens before the sequence's first position see nothing
    for (int i = threadIdx.x; i < (R - r0) * 64; i += SCORE_WARPS * 32) {
        const int r = r0 + i / 64, c = i % 64;
        const size_t row = (static_cast<size_t>(b) * p.q_len + r / p.group) * p.n_q_heads + h * p.group + r % p.group;
        float2 f[4];
        unpack8(reinterpret_cast<const uint4*>(p.q + row * D)[c], f);
        float4* dst = s_q + ((r * 2 + (c >> 5)) * 2) * 32 + (c & 31);
        dst[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        dst[32] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
    __syncthreads();
    uint32_t* keys = p.keys + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.max_pages;
    int at = 0;                                      // stage of page i
    for (int i = 0; number(i) < held; i += SCORE_PAGES, at = at + SCORE_PAGES < SCORE_STAGES ? at + SCORE_PAGES : 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(SCORE_STAGES - SCORE_PAGES) : "memory");
        __syncwarp();
        float2 lo[SCORE_PAGES][8], hi[SCORE_PAGES][8];
#pragma unroll
        for (int k = 0; k < SCORE_PAGES; ++k) {
            const uint4* src = reinterpret_cast<const uint4*>(ring + (at + k) * PAGE_BYTES) + lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 f[4];
                unpack8(src[32 * j], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) lo[k][4 * j + e] = f[e];
                unpack8(src[64 + 32 * j], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) hi[k][4 * j + e] = f[e];
            }
        }
        int now[SCORE_PAGES];
#pragma unroll
        for (int k = 0; k < SCORE_PAGES; ++k) now[k] = pages[k];
        __syncwarp();                                // the stages are read
#pragma unroll
        for (int k = 0; k < SCORE_STAGES - SCORE_PAGES; ++k) pages[k] = pages[k + SCORE_PAGES];
#pragma unroll
        for (int k = 0; k < SCORE_PAGES; ++k) pages[SCORE_STAGES - SCORE_PAGES + k] = load(i + SCORE_STAGES + k, at + k);

        // ROWS rows at a time (the last one again where they run out): lane l gets the sum of
        // row l / (16 / ROWS) % ROWS of them and page l / 16
        float best = -INFINITY;
        bool nan = false;
        for (int r = r0; r < R; r += ROWS) {
            float v[SCORE_PAGES * ROWS];
#pragma unroll
            for (int e2 = 0; e2 < ROWS; ++e2) {
                const float4* q = s_q + min(r + e2, R - 1) * 128 + lane;
                float2 x[SCORE_PAGES][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 q4 = q[(2 * j + (e >> 1)) * 32];
                        const float2 qe = e & 1 ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
                        const float2 up = make_float2(above_0(qe.x), above_0(qe.y));
                        const float2 down = make_float2(below_0(qe.x), below_0(qe.y));
#pragma unroll
                        for (int k = 0; k < SCORE_PAGES; ++k) {
                            x[k][e] = ffma2(down, lo[k][4 * j + e], j ? x[k][e] : make_float2(0.f, 0.f));
                            x[k][e] = ffma2(up, hi[k][4 * j + e], x[k][e]);
                        }
                    }
#pragma unroll
                for (int k = 0; k < SCORE_PAGES; ++k) {
                    // the eight of this lane: 0 + 4, 1 + 5, ..., then halves of those
                    const float2 d = fadd2(fadd2(x[k][0], x[k][2]), fadd2(x[k][1], x[k][3]));
                    v[ROWS * k + e2] = d.x + d.y;
                }
            }
            const float s = sum_of(v, lane);
            nan |= s != s;
            best = fmaxf(best, s);
        }
#pragma unroll
        for (int off = 8; off >= 16 / ROWS; off >>= 1) {
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
            nan |= __shfl_xor_sync(0xffffffffu, nan ? 1 : 0, off) != 0;
        }
        const int k = lane >> 4, lp = number(i + k);
        if ((lane & 15) == 0 && lp < held) {
            const int page = k ? now[1] : now[0];
            if (page == -2) report_error(p.err, FA512_DEVICE_ERR_INDEX);
            // (outside the pool: lowest)
            keys[lp] = page == -2 ? 0u : page == -1 ? KEY_ALWAYS : nan ? KEY_NOT_FINITE : key_of(best);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------- choice
//
// A block per (sequence, KV head) finds the last key that is chosen by its digits, eight
// bits at a time from the highest in which two keys differ, a histogram each, until all
// of a digit's keys are chosen (two digits for a few hundred scores of about a size);
// then each warp writes the chosen pages of its part of the sequence, in rising order.
// What takes the time is the way from one step to the next: 64 sequences of up to 448
// pages, 4 heads, take 5 us, four digits of all 32 bits took 8.  The first SHARED keys
// wait in shared memory, the rest is read again for each digit.  (A warp with 32 keys a
// lane in registers, searching bit by bit, takes twice as long: its code runs once, and
// fetching it is what that takes.)
constexpr int CHOOSE_THREADS = 256;
constexpr int CHOOSE_WARPS = CHOOSE_THREADS / 32;
constexpr int SHARED = 4096;
constexpr int DIGITS = 4;

__global__ void __launch_bounds__(CHOOSE_THREADS) choose_kernel(const SelectParams p) {
    __shared__ uint32_t s_keys[SHARED];
    __shared__ __align__(16) int s_hist[DIGITS][256];
    __shared__ uint32_t s_most[CHOOSE_WARPS], s_least[CHOOSE_WARPS];
    __shared__ int s_above[CHOOSE_WARPS], s_equal[CHOOSE_WARPS];
    __shared__ int s_digit, s_left, s_count;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // also where no scores were needed: for whatever ran before
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t* keys = p.keys + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.max_pages;
    // (the first keys are on their way before the length is known)
    const uint32_t key0 = tid < p.max_pages ? keys[tid] : 0u;
    const uint32_t key1 = tid + CHOOSE_THREADS < p.max_pages ? keys[tid + CHOOSE_THREADS] : 0u;
    const int len = length_of(p, b, false);
    const int held = static_cast<int>((static_cast<unsigned>(len) + p.page_size - 1) / p.page_size);
    int32_t* out = p.selected + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.n_select;
    if (held <= p.n_select) {
        for (int i = tid; i < p.n_select; i += CHOOSE_THREADS) out[i] = i < held ? i : -1;
        return;
    }
#pragma unroll
    for (int i = 0; i < DIGITS; ++i) s_hist[i][tid] = 0;
    static_assert(CHOOSE_THREADS == 256, "a thread a digit");
    // the largest and the smallest key but for the pages that are always chosen
    uint32_t most = 0u, least = KEY_ALWAYS;
    for (int i = tid; i < held; i += CHOOSE_THREADS) {
        const uint32_t k = i == tid ? key0 : i == tid + CHOOSE_THREADS ? key1 : keys[i];
        if (i < SHARED) s_keys[i] = k;
        if (k != KEY_ALWAYS) {
            most = max(most, k);
            least = min(least, k);
        }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
        s_most[warp] = most;
        s_least[warp] = least;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < CHOOSE_WARPS; ++w) {
        most = max(most, s_most[w]);
        least = min(least, s_least[w]);
    }
    auto key_at = [&](int i) { return i < SHARED ? s_keys[i] : keys[i]; };
    // `left` to take among the keys whose bits from `shift` on are `prefix`, all of the larger ones
    int left = p.n_select - p.n_first - p.n_last, shift = 0;
    uint32_t prefix = KEY_ALWAYS;
    if (left > 0) {
        int known = 32 - __clz(most ^ least);            // the bits from here on are all keys'
        prefix = known < 32 ? most >> known : 0u;
        for (int d = 0;; ++d) {
            shift = max(0, known - 8);
            for (int i = tid; i < held; i += CHOOSE_THREADS) {
                const uint32_t k = key_at(i);
                if (k != KEY_ALWAYS && (known == 32 || k >> known == prefix)) atomicAdd(&s_hist[d][(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {                             // lane l: digits 255 - 8 l downwards
                const int4* hist = reinterpret_cast<const int4*>(&s_hist[d][248 - 8 * lane]);
                const int4 lo = hist[0], hi = hist[1];
                const int n[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
                int sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += n[e];
                int before = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += y;
                }
                before -= sum;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (before < left && before + n[e] >= left) {
                        s_digit = 255 - 8 * lane - e;
                        s_left = left - before;
                        s_count = n[e];
                    }
                    before += n[e];
                }
            }
            __syncthreads();
            // (where the digit has bits that were known, they are the prefix's)
            const int bits = known - shift;
            prefix = (prefix << bits) | (static_cast<uint32_t>(s_digit) & ((1u << bits) - 1u));
            left = s_left;
            known = shift;
            if (s_count == left || shift == 0) break;
        }
    }
    // a warp's part of the pages: counted, then written behind the parts before it
    const int part = (held + CHOOSE_THREADS - 1) / CHOOSE_THREADS * 32, end = min(held, (warp + 1) * part);
    auto look = [&](int i, bool* equal) {
        const uint32_t k = i < end ? key_at(i) : 0u;
        *equal = i < end && k != KEY_ALWAYS && k >> shift == prefix;
        return i < end && (k == KEY_ALWAYS || k >> shift > prefix);
    };
    int above = 0, equal = 0;
    for (int i = warp * part; i < end; i += 32) {
        bool eq;
        const bool gt = look(i + lane, &eq);
        above += __popc(__ballot_sync(0xffffffffu, gt));
        equal += __popc(__ballot_sync(0xffffffffu, eq));
    }
    if (lane == 0) {
        s_above[warp] = above;
        s_equal[warp] = equal;
    }
    __syncthreads();
    above = equal = 0;
#pragma unroll
    for (int w = 0; w < CHOOSE_WARPS; ++w) {
        above += w < warp ? s_above[w] : 0;
        equal += w < warp ? s_equal[w] : 0;
    }
    for (int i = warp * part; i < end; i += 32) {
        bool eq;
        const bool gt = look(i + lane, &eq);
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq), lower = (1u << lane) - 1u;
        const int g0 = above + __popc(mg & lower), e0 = equal + __popc(me & lower);
        if (gt || (eq && e0 < left)) out[g0 + min(e0, left)] = i + lane;
        above += __popc(mg);
        equal += __popc(me);
    }
}

}  // namespace select

cudaError_t launch_page_bounds(const BoundsParams& p, int element_bits, cudaStream_t stream) {
    using namespace select;
    const int touched = min((p.q_len - 1) / p.page_size + ((p.q_len - 1) % p.page_size != 0) + 1, p.max_pages_per_seq);
    const dim3 grid(static_cast<unsigned>(touched) * static_cast<unsigned>(p.n_kv_heads), p.batch);
    if (element_bits == 16) bounds_kernel<16><<<grid, bounds_threads(16), 0, stream>>>(p);
    else if (element_bits == 8) bounds_kernel<8><<<grid, bounds_threads(8), 0, stream>>>(p);
    else bounds_kernel<4><<<grid, bounds_threads(4), 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_select_pages(const SelectParams& p, cudaStream_t stream) {
    using namespace select;
    if (p.max_pages > p.n_select) {
        // three rounds of four blocks on each SM, and none with less than a round of pages
        const int rounds = (p.max_pages + SCORE_WARPS * SCORE_PAGES - 1) / (SCORE_WARPS * SCORE_PAGES);
        const long long items = static_cast<long long>(p.n_kv_heads) * p.batch, want = (SCORE_BLOCKS + items - 1) / items;
        const dim3 grid(static_cast<unsigned>(want < rounds ? want : rounds), p.n_kv_heads, p.batch);
        const int smem = score_smem(p.q_len * p.group);
        auto kernel = p.q_len * p.group <= 2 ? score_kernel<2> : score_kernel<4>;
        const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, score_smem(16));
        if (set != cudaSuccess) return set;
        kernel<<<grid, SCORE_WARPS * 32, smem, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(p.n_kv_heads, p.batch);
    cfg.blockDim = dim3(CHOOSE_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, choose_kernel, p);
}

}  // namespace fa512
