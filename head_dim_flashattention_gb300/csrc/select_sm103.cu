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
// of a coded one, in 4 bits those of one scale), the rows dealt to 4 or 8 groups of
// threads whose results meet in shared memory.  NaN elements make both bounds NaN.
constexpr int BOUNDS_THREADS = 256;

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
__global__ void __launch_bounds__(BOUNDS_THREADS) bounds_kernel(const BoundsParams p) {
    constexpr int ROW = BITS == 16 ? 2 * D : BITS == 8 ? D : kFp4RowBytes;
    constexpr int PAIRS = BITS == 16 ? 4 : 8;       // x 2 elements of a thread
    constexpr int LANES = D / (2 * PAIRS);          // threads of a row: 64, 32
    constexpr int GROUPS = BOUNDS_THREADS / LANES;
    constexpr bool F16 = BITS != 16;
    __shared__ uint32_t s_lo[GROUPS - 1][D / 2], s_hi[GROUPS - 1][D / 2];
    const int b = blockIdx.z, h = blockIdx.y;
    const int len = p.kv_lens[b];
    const int n_new = p.q_lens ? p.q_lens[b] : p.q_len;
    if (n_new < 0 || n_new > p.q_len || len < n_new ||
        len > static_cast<long long>(p.max_pages_per_seq) * p.page_size) {
        if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int lp = (len - n_new) / p.page_size + blockIdx.x;
    if (n_new == 0 || lp > (len - 1) / p.page_size) return;
    const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
    if (page < 0 || page >= p.num_pages) {
        if (h == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int live = min(p.page_size, len - lp * p.page_size);
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const size_t step = static_cast<size_t>(p.n_kv_heads) * ROW;      // bytes from a row to the next
    const uint8_t* src = p.k_pages + (static_cast<size_t>(page) * p.page_size * p.n_kv_heads + h) * ROW;
    MinMax m[PAIRS];
    const uint32_t inf = F16 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) m[i] = {inf, inf | 0x80008000u};
    constexpr int RUN = 8;                          // rows in flight
    for (int r0 = grp; r0 < live; r0 += RUN * GROUPS) {
        uint4 x[RUN];
        uint8_t scale[RUN];
#pragma unroll
        for (int k = 0; k < RUN; ++k) {
            // (a row past the end is the first one again)
            const int r = r0 + k * GROUPS < live ? r0 + k * GROUPS : r0;
            const uint8_t* row = src + r * step;
            if constexpr (BITS == 4) {
                const uint2 y = *reinterpret_cast<const uint2*>(row + 8 * u);
                x[k] = make_uint4(y.x, y.y, 0u, 0u);
                scale[k] = row[256 + u];
            } else {
                x[k] = *reinterpret_cast<const uint4*>(row + 16 * u);
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
// A warp scores two pages at a time, the bounds of its next two on their way: lane
// l holds channels 8 l .. 8 l + 7 and 256 + 8 l .. of them, goes through the query
// rows (in shared memory, as fp32) and keeps each page's largest score.  max(q lo,
// q hi) is max(q, 0) hi + min(q, 0) lo, of which one term is 0: two packed
// multiply-adds a pair of channels, and each sum below rounds once.
constexpr int SCORE_WARPS = 4;
constexpr int SCORE_PAGES = 2;
constexpr int SCORE_BLOCKS = 6 * 152;                // blocks to spread the pages over
constexpr int SCORE_ROWS = 16;                       // most query rows of a KV head

// Unsigned integers in the order of the scores, -0 and 0 equal.  Largest of all,
// with the pages that are always chosen, are those with a NaN or infinite score:
// the formula above turns every bound that is not finite into one of the two.
constexpr uint32_t KEY_MOST = 0xffffffffu;
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x || x == INFINITY) return KEY_MOST;
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

__global__ void __launch_bounds__(SCORE_WARPS * 32) score_kernel(const SelectParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float4 s_q[SCORE_ROWS][2][2][32];     // [row][half of the channels][4 of 8][lane]
    const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int held = (len + p.page_size - 1) / p.page_size;
    const int step = gridDim.x * SCORE_WARPS * SCORE_PAGES;
    if (blockIdx.x * SCORE_WARPS * SCORE_PAGES >= held || held <= p.n_select) return;   // all pages are chosen
    const int R = p.q_len * p.group;
    const int r0 = max(0, p.q_len - len) * p.group;  // rows of tokens before the sequence's first position see nothing
    for (int i = threadIdx.x; i < (R - r0) * 64; i += SCORE_WARPS * 32) {
        const int r = r0 + i / 64, c = i % 64;
        const size_t row = (static_cast<size_t>(b) * p.q_len + r / p.group) * p.n_q_heads + h * p.group + r % p.group;
        float2 f[4];
        unpack8(reinterpret_cast<const uint4*>(p.q + row * D)[c], f);
        s_q[r][c >> 5][0][c & 31] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        s_q[r][c >> 5][1][c & 31] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
    __syncthreads();
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    uint32_t* keys = p.keys + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.max_pages;
    // the page of lp: -1 none (always chosen, or past the end), -2 outside the pool
    auto page_of = [&](int lp) {
        if (lp >= held || lp < p.n_first || lp >= held - p.n_last) return -1;
        const int page = table[lp];
        return page < 0 || page >= p.num_pages ? -2 : page;
    };
    uint4 raw[SCORE_PAGES][4];
    int page[SCORE_PAGES], page_next[SCORE_PAGES];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < SCORE_PAGES; ++i) {
            const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<size_t>(max(page[i], 0)) * p.n_kv_heads + h) * 2 * D);
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[i][j] = page[i] >= 0 ? src[32 * j + lane] : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int lp0 = (blockIdx.x * SCORE_WARPS + warp) * SCORE_PAGES;
#pragma unroll
    for (int i = 0; i < SCORE_PAGES; ++i) page[i] = page_of(lp0 + i);
    load();
#pragma unroll
    for (int i = 0; i < SCORE_PAGES; ++i) page_next[i] = page_of(lp0 + step + i);
    for (; lp0 < held; lp0 += step) {
        float2 lo[SCORE_PAGES][8], hi[SCORE_PAGES][8];
        float best[SCORE_PAGES];
        int now[SCORE_PAGES];
#pragma unroll
        for (int i = 0; i < SCORE_PAGES; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float2 f[4];
                unpack8(raw[i][j], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) lo[i][4 * j + e] = f[e];
                unpack8(raw[i][2 + j], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) hi[i][4 * j + e] = f[e];
            }
            best[i] = -INFINITY;
            now[i] = page[i];
            page[i] = page_next[i];
        }
        if (lp0 + step < held) load();
#pragma unroll
        for (int i = 0; i < SCORE_PAGES; ++i) page_next[i] = page_of(lp0 + 2 * step + i);
        bool nan[SCORE_PAGES] = {};
        for (int r = r0; r < R; ++r) {
            float2 x[SCORE_PAGES][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 q4 = s_q[r][j][e >> 1][lane];
                    const float2 q = e & 1 ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
                    const float2 up = make_float2(fmaxf(q.x, 0.f), fmaxf(q.y, 0.f));
                    const float2 down = make_float2(fminf(q.x, 0.f), fminf(q.y, 0.f));
#pragma unroll
                    for (int i = 0; i < SCORE_PAGES; ++i) {
                        x[i][e] = ffma2(down, lo[i][4 * j + e], j ? x[i][e] : make_float2(0.f, 0.f));
                        x[i][e] = ffma2(up, hi[i][4 * j + e], x[i][e]);
                    }
                }
#pragma unroll
            for (int i = 0; i < SCORE_PAGES; ++i) {
                // the eight of this lane: 0 + 4, 1 + 5, ..., then halves of those
                const float2 a = fadd2(x[i][0], x[i][2]), c = fadd2(x[i][1], x[i][3]);
                const float2 d = fadd2(a, c);
                float s = d.x + d.y;
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                nan[i] |= s != s;
                best[i] = fmaxf(best[i], s);
            }
        }
        if (lane < SCORE_PAGES && lp0 + lane < held) {
            uint32_t key = 0;
#pragma unroll
            for (int i = 0; i < SCORE_PAGES; ++i)
                if (lane == i) {
                    if (now[i] == -2) report_error(p.err, FA512_DEVICE_ERR_INDEX);
                    key = now[i] == -1 || nan[i] ? KEY_MOST : now[i] >= 0 ? key_of(best[i]) : 0u;   // outside: lowest
                }
            keys[lp0 + lane] = key;
        }
    }
}

// ------------------------------------------------------------------- choice
//
// A block per (sequence, KV head) finds the n-th largest key by its four bytes
// from the top, a histogram of 256 each, then writes the pages above it, and the
// lowest of those equal to it, in rising order.
constexpr int CHOOSE_THREADS = 256;

__global__ void __launch_bounds__(CHOOSE_THREADS) choose_kernel(const SelectParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int hist[256], s_warp[2][CHOOSE_THREADS / 32];
    __shared__ int s_digit, s_left;
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = length_of(p, b, false);
    const int held = (len + p.page_size - 1) / p.page_size;
    int32_t* out = p.selected + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.n_select;
    if (held <= p.n_select) {
        for (int i = tid; i < p.n_select; i += CHOOSE_THREADS) out[i] = i < held ? i : -1;
        return;
    }
    const uint32_t* keys = p.keys + (static_cast<size_t>(b) * p.n_kv_heads + h) * p.max_pages;
    uint32_t prefix = 0;
    int left = p.n_select;                           // to take among the keys that begin with the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < held; i += CHOOSE_THREADS) {
            const uint32_t k = keys[i];
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        // how many lie above each digit: a scan from the top
        const int mine = hist[255 - tid];
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_warp[0][warp] = sum;
        __syncthreads();
        int before = sum - mine;
        for (int w = 0; w < warp; ++w) before += s_warp[0][w];
        if (before < left && before + mine >= left) {
            s_digit = 255 - tid;
            s_left = left - before;
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(s_digit);
        left = s_left;
        __syncthreads();
    }
    int above = 0, equal = 0;                        // chosen before this run of pages: above the n-th key, equal to it
    for (int i0 = 0; i0 < held; i0 += CHOOSE_THREADS) {
        const int i = i0 + tid;
        const uint32_t k = i < held ? keys[i] : 0u;
        const bool gt = i < held && k > prefix, eq = i < held && k == prefix;
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_warp[0][warp] = __popc(mg);
            s_warp[1][warp] = __popc(me);
        }
        __syncthreads();
        int g0 = above, e0 = equal;
        for (int w = 0; w < CHOOSE_THREADS / 32; ++w) {
            if (w < warp) {
                g0 += s_warp[0][w];
                e0 += s_warp[1][w];
            }
            above += s_warp[0][w];
            equal += s_warp[1][w];
        }
        const unsigned lower = (1u << lane) - 1u;
        g0 += __popc(mg & lower);
        e0 += __popc(me & lower);
        if (gt || (eq && e0 < left)) out[g0 + min(e0, left)] = i;
        __syncthreads();
    }
}

}  // namespace select

cudaError_t launch_page_bounds(const BoundsParams& p, int element_bits, cudaStream_t stream) {
    using namespace select;
    const int touched = min((p.q_len - 1) / p.page_size + ((p.q_len - 1) % p.page_size != 0) + 1, p.max_pages_per_seq);
    const dim3 grid(touched, p.n_kv_heads, p.batch);
    if (element_bits == 16) bounds_kernel<16><<<grid, BOUNDS_THREADS, 0, stream>>>(p);
    else if (element_bits == 8) bounds_kernel<8><<<grid, BOUNDS_THREADS, 0, stream>>>(p);
    else bounds_kernel<4><<<grid, BOUNDS_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_select_pages(const SelectParams& p, cudaStream_t stream) {
    using namespace select;
    if (p.max_pages > p.n_select) {
        // enough blocks for six on each SM, and none with less than a round of pages
        const int rounds = (p.max_pages + SCORE_WARPS * SCORE_PAGES - 1) / (SCORE_WARPS * SCORE_PAGES);
        const long long items = static_cast<long long>(p.n_kv_heads) * p.batch, want = (SCORE_BLOCKS + items - 1) / items;
        const dim3 grid(static_cast<unsigned>(want < rounds ? want : rounds), p.n_kv_heads, p.batch);
        score_kernel<<<grid, SCORE_WARPS * 32, 0, stream>>>(p);
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
