// The paged cache around the attention kernels, sm_103a: appending rows
// (bf16, or rounded to E4M3), moving accepted rows together, and planning,
// sharing, copying and freeing pages by reference counts.
//
// All of it moves data: the floor of each kernel is its bytes at the copy
// rate, and for the small calls of a decode step the launch and a chain of
// dependent loads (length, page-table entry, row).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <mutex>

#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_pair.cuh"

namespace fa512 {
namespace cache {

constexpr int D = 512;

// ------------------------------------------------------------------- append
//
// A thread moves 16 stored bytes (8 bf16 elements, or 16 elements rounded to
// E4M3) of the key row and of the value row of up to APPEND_RUN places of its
// sequence (blockIdx.y), all its loads before the first store.
// Bound: bytes (8 sequences of up to 4,096 new tokens, 4 heads, into E4M3: 394
// MB in 58.9 us, 6.7 TB/s); one token of 16 sequences takes 2.4 us, the chain
// of three dependent loads.  The division by a scale that is no power of two
// costs more issue slots than the bytes take (83.0 us); a power of two (whose
// reciprocal is exact) multiplies, which gives the same quotients.
constexpr int APPEND_THREADS = 256;
constexpr int APPEND_RUN = 2;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// 16 bf16 elements -> the 16 E4M3 bytes of x / scale (the nearest fp32
// quotient, then the nearest code, ties to even).  POW2: `by` is 1 / scale.
template <bool POW2>
__device__ __forceinline__ uint4 quantise16(const uint4 a, const uint4 b, float by) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        x[2 * i] = POW2 ? lo * by : __fdiv_rn(lo, by);
        x[2 * i + 1] = POW2 ? hi * by : __fdiv_rn(hi, by);
    }
    return make_uint4(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]),
                      e4m3x4(x[8], x[9], x[10], x[11]), e4m3x4(x[12], x[13], x[14], x[15]));
}

// MODE 0: bf16, 1: E4M3, 2: E4M3 with scales that are powers of two
template <int MODE>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams p) {
    constexpr int UNIT = MODE ? 16 : 8;                   // elements of a place
    constexpr int V = UNIT / 8;                           // 16-byte loads of one
    const int b = blockIdx.y;
    const int units = p.n_kv_heads * (D / UNIT);          // per token
    int n_new = p.q_lens ? p.q_lens[b] : p.q_len;
    const int len = p.kv_lens[b];
    if (n_new < 0 || n_new > p.q_len) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        n_new = 0;                                        // no telling where its tokens belong
    }
    uint4 k[APPEND_RUN][V], v[APPEND_RUN][V];
    size_t at[APPEND_RUN];
    bool there[APPEND_RUN];
#pragma unroll
    for (int r = 0; r < APPEND_RUN; ++r) {
        const unsigned idx = (blockIdx.x * APPEND_RUN + r) * APPEND_THREADS + threadIdx.x;
        const int t = static_cast<int>(idx / static_cast<unsigned>(units));
        const int u = static_cast<int>(idx % static_cast<unsigned>(units));
        const long long pos = static_cast<long long>(len) - n_new + t;
        there[r] = t < n_new;
        if (there[r] && (pos < 0 || pos >= static_cast<long long>(p.max_pages_per_seq) * p.page_size)) {
            if (u == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
            there[r] = false;
        }
        if (!there[r]) continue;
        const int lp = static_cast<int>(pos) / p.page_size;
        const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
        const uint4* ks = reinterpret_cast<const uint4*>(p.k_new + b * p.k_batch_stride + t * p.k_token_stride) + V * u;
        const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + b * p.v_batch_stride + t * p.v_token_stride) + V * u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            k[r][i] = ks[i];
            v[r][i] = vs[i];
        }
        if (page < 0 || page >= p.num_pages) {
            if (u == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
            there[r] = false;
        }
        at[r] = (static_cast<size_t>(page) * p.page_size + static_cast<int>(pos) % p.page_size) * units + u;
    }
#pragma unroll
    for (int r = 0; r < APPEND_RUN; ++r) {
        if (!there[r]) continue;
        uint4 *kd = static_cast<uint4*>(p.k_pages) + at[r], *vd = static_cast<uint4*>(p.v_pages) + at[r];
        if constexpr (MODE == 0) {
            *kd = k[r][0];
            *vd = v[r][0];
        } else {
            *kd = quantise16<MODE == 2>(k[r][0], k[r][V - 1], p.k_scale);
            *vd = quantise16<MODE == 2>(v[r][0], v[r][V - 1], p.v_scale);
        }
    }
}

// ----------------------------------------------------------- append, 4 bits
//
// A row of a head is 288 bytes: 256 bytes of E2M1 codes (element 2 i in the
// low half of byte i), then 32 E4M3 scales, one for 16 elements.  With y = x /
// tensor scale (the nearest fp32 quotient) a group's scale is the E4M3 value
// nearest to max |y| / 6, and a code the E2M1 value nearest to the fp32
// quotient y / scale, ties to even; both saturate.  A group that holds NaN gets
// the NaN scale and codes 0; a scale that rounds to 0 makes the codes 0.
//
// A warp rounds one row of K and of V, a group of 16 elements a lane.  Bound: bytes (8
// sequences of up to 4,096 new tokens, 4 heads: 335 MB in 55 us, 6.1 TB/s); the 33
// divisions of a group cost more issue slots than that takes (147 us), so tensor
// scales that are both powers of two have a path without them (to_4bit_pow2).  One token
// of 16 sequences takes 2.1 us.
__device__ __forceinline__ uint32_t e2m1x8(const float (&z)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    return r;
}

// E4M3 nearest to x: its byte, and its value.
__device__ __forceinline__ float to_e4m3(float x, uint8_t* byte) {
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(x));
    uint32_t s2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(s8));
    float s;
    asm("cvt.f32.f16 %0, %1;" : "=f"(s) : "h"(static_cast<unsigned short>(s2 & 0xffffu)));
    *byte = static_cast<uint8_t>(s8 & 0xff);
    return s;
}

// 16 bf16 elements -> codes and the scale byte
__device__ __forceinline__ uint2 to_4bit(const uint4 a, const uint4 b, float tensor_scale, uint8_t* scale_byte) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float y[16], most = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[2 * i] = __fdiv_rn(__uint_as_float(w[i] << 16), tensor_scale);
        y[2 * i + 1] = __fdiv_rn(__uint_as_float(w[i] & 0xffff0000u), tensor_scale);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        most = fmaxf(most, fabsf(y[i]));
        nan |= y[i] != y[i];
    }
    const float s = to_e4m3(__fdiv_rn(most, 6.f), scale_byte);
    float z[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i >> 3][i & 7] = s > 0.f ? __fdiv_rn(y[i], s) : 0.f;
    if (!nan) return make_uint2(e2m1x8(z[0]), e2m1x8(z[1]));
    *scale_byte = 0x7f;
    return make_uint2(0u, 0u);
}

// The same for a tensor scale whose reciprocal `by` is a power of two, without a
// division.  Then y has 8 significant bits.
//   Scale: max |y| / 6, where it is no midpoint of two E4M3 values (5 bits), differs
//   from all of them by 2^-11 of it or more; the product with the rounded 1/6, off by
//   2^-23 of it, rounded to 16 bits hits the midpoints exactly and crosses none.
//   Codes: y / s, where it is no midpoint of two E2M1 values, lies 2^-11 or more from
//   all of them (the lowest bit of a y above s / 8 is at least 2^-11 s, and a midpoint
//   times s, which has 4 bits, is a multiple of it).  x times by / s, off by 2^-22 of
//   it, plus 1.5 * 2^11 rounds to a multiple of 2^-12: midpoints come out exactly, and
//   nothing crosses one.
__device__ __forceinline__ uint2 to_4bit_pow2(const uint4 a, const uint4 b, float by, uint8_t* scale_byte) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t top = 0;                                     // largest magnitudes of the halves, NaN where there is one
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[i] & 0x7fff7fffu));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"((top << 16) | (top >> 16)));
    const float most = __uint_as_float(top & 0xffff0000u);
    const bool nan = most != most;
    const float sixth = most * by * (1.f / 6.f);
    const float s = to_e4m3(nan ? 0.f : __uint_as_float((__float_as_uint(sixth) + 0x80u) & ~0xffu), scale_byte);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // 0 < s: 2^-9 at least
    r *= by;
    constexpr float SNAP = 1.5f * 2048.f;
    float z[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        const float q = __fadd_rn(__fmaf_rn(x, r, SNAP), -SNAP);
        // its sign also where it came to 0
        z[i >> 3][i & 7] = __uint_as_float((__float_as_uint(q) & 0x7fffffffu) | (__float_as_uint(x) & 0x80000000u));
    }
    if (nan) *scale_byte = 0x7f;
    const uint2 codes = make_uint2(e2m1x8(z[0]), e2m1x8(z[1]));
    return s > 0.f ? codes : make_uint2(0u, 0u);
}

template <bool POW2>
__global__ void __launch_bounds__(APPEND_THREADS) append_fp4_kernel(const AppendParams p) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    int n_new = p.q_lens ? p.q_lens[b] : p.q_len;
    const int len = p.kv_lens[b];
    if (n_new < 0 || n_new > p.q_len) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        n_new = 0;                                        // no telling where its tokens belong
    }
    const unsigned row = blockIdx.x * (APPEND_THREADS / 32) + (threadIdx.x >> 5);
    const int t = static_cast<int>(row / static_cast<unsigned>(p.n_kv_heads));
    const int h = static_cast<int>(row - static_cast<unsigned>(t) * static_cast<unsigned>(p.n_kv_heads));
    if (t >= n_new) return;
    const long long pos = static_cast<long long>(len) - n_new + t;
    if (pos < 0 || pos >= static_cast<long long>(p.max_pages_per_seq) * p.page_size) {
        if (lane == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + (static_cast<int>(pos) >> p.page_shift)];
    const uint4* ks = reinterpret_cast<const uint4*>(p.k_new + b * p.k_batch_stride + t * p.k_token_stride) + h * 64 + 2 * lane;
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + b * p.v_batch_stride + t * p.v_token_stride) + h * 64 + 2 * lane;
    const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const size_t at = ((static_cast<size_t>(page) * p.page_size + (static_cast<int>(pos) & (p.page_size - 1))) * p.n_kv_heads + h) *
                      kFp4RowBytes;
    uint8_t *kd = static_cast<uint8_t*>(p.k_pages) + at, *vd = static_cast<uint8_t*>(p.v_pages) + at;
    uint8_t s;
    *reinterpret_cast<uint2*>(kd + 8 * lane) = POW2 ? to_4bit_pow2(k0, k1, p.k_scale, &s) : to_4bit(k0, k1, p.k_scale, &s);
    kd[256 + lane] = s;
    *reinterpret_cast<uint2*>(vd + 8 * lane) = POW2 ? to_4bit_pow2(v0, v1, p.v_scale, &s) : to_4bit(v0, v1, p.v_scale, &s);
    vd[256 + lane] = s;
}

// ------------------------------------------------------------------ compact
//
// accepted[i] >= i, rising: a row only ever moves down.  A thread owns one
// 16-byte column of the rows of one sequence, layer and tensor and moves its
// rows in rising order.  The write of row i cannot hit the source of a later
// row (accepted[i'] >= i' > i), and it can only hit a source of an earlier
// row, which this thread has read already; so loading a batch of sources
// ahead and storing afterwards is safe, and no two threads touch one byte.
// Bound: bytes, in rows of 1 KiB a head (64 sequences, 8 layers, ragged trees of
// 64: 21.4 us); small calls the loads in a row (16 sequences, one layer: 3.2 us).
constexpr int COMPACT_THREADS = 256;
constexpr int COMPACT_BATCH = 8;        // rows in flight per thread
constexpr int COMPACT_MAX = 1024;

__global__ void __launch_bounds__(COMPACT_THREADS) compact_kernel(const CompactParams p) {
    __shared__ int src[COMPACT_MAX], dst[COMPACT_MAX];   // row numbers in the pool, -1: not moved
    const int b = blockIdx.y, tid = threadIdx.x;
    const int len = p.kv_lens[b];
    const int cnt = p.q_lens ? p.q_lens[b] : p.q_len;
    const int n = p.n_accepted[b];
    const int start = len - cnt;
    bool ok = cnt >= 0 && cnt <= p.q_len && n >= 0 && n <= cnt && n <= p.max_accepted && start >= 0 &&
              len <= static_cast<long long>(p.max_pages_per_seq) * p.page_size;
    bool pages_ok = true;
    if (ok) {
        const int* acc = p.accepted + static_cast<size_t>(b) * p.max_accepted;
        const int* pt = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
        for (int i = tid; i < n; i += COMPACT_THREADS) {
            const int a = acc[i];
            const int before = i ? acc[i - 1] : -1;
            int s = -1, d = -1;
            if (a <= before || a < 0 || a >= cnt) {
                ok = false;
            } else if (a != i) {
                const int sp = start + a, dp = start + i;
                const int s_page = pt[sp / p.page_size], d_page = pt[dp / p.page_size];
                if (s_page < 0 || s_page >= p.num_pages || d_page < 0 || d_page >= p.num_pages) {
                    pages_ok = false;
                } else {
                    s = s_page * p.page_size + sp % p.page_size;
                    d = d_page * p.page_size + dp % p.page_size;
                }
            }
            src[i] = s;
            dst[i] = d;
        }
    }
    ok = __syncthreads_and(ok);
    if (blockIdx.x == 0) {
        if (!pages_ok || (!ok && tid == 0)) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        if (tid == 0) p.new_kv_lens[b] = ok ? start + n : len;
    }
    if (!ok) return;
    const int units = p.row_bytes / 16;
    const long long idx = static_cast<long long>(blockIdx.x) * COMPACT_THREADS + tid;
    const long long line = idx / units;                   // (layer, K or V)
    if (line >= 2LL * p.n_layers) return;
    const int u = static_cast<int>(idx - line * units);
    uint4* base = reinterpret_cast<uint4*>((line & 1) ? p.v_pages : p.k_pages) +
                  static_cast<size_t>(line >> 1) * p.num_pages * p.page_size * units + u;
    for (int i0 = 0; i0 < n; i0 += COMPACT_BATCH) {
        uint4 x[COMPACT_BATCH];
#pragma unroll
        for (int j = 0; j < COMPACT_BATCH; ++j)
            if (i0 + j < n && src[i0 + j] >= 0) x[j] = base[static_cast<size_t>(src[i0 + j]) * units];
#pragma unroll
        for (int j = 0; j < COMPACT_BATCH; ++j)
            if (i0 + j < n && src[i0 + j] >= 0) base[static_cast<size_t>(dst[i0 + j]) * units] = x[j];
    }
}

// -------------------------------------------------------- fork and resize
//
// One cluster of blocks plans the pages, so that its phases are separated by
// the cluster's barrier and not by launches: (A) copy the reference counts
// and find how many fresh pages each sequence needs (fork: the first child of
// every parent), with a scan over the sequences; (B) write the new tables and
// move the counts by integer atomics (their order does not matter); (C) mark
// the free pages of the block's part of the pool in a bit map, learn the
// other blocks' counts through distributed shared memory, and deal the free
// pages, lowest first, to the needs in order: the page of rank r goes to the
// sequence whose scan interval holds r.
//
// Bound: chains of dependent loads, not bytes (2.3 MB for 512 sequences of
// 448 pages and a pool of 178,000 pages), so every pass keeps 8 loads a
// thread in flight and nothing is looked up twice: lengths, parents and needs
// stay in shared memory.  Those 512 sequences take 18.2 us with 16 blocks (27.5
// with 8, 109 with one); 16 sequences 6.9 us, of which the launch of a cluster and
// its barriers are most.
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_MAX_BATCH = 8192;
constexpr int PLAN_CLUSTER = 16;         // blocks, at most (8 where a cluster of 16 does not fit)
constexpr int PLAN_RUN = 8;              // loads in flight per thread
constexpr int PLAN_CHUNK = PLAN_THREADS; // words (of 32 pages) of the bit map

// Shared memory: fixed part, then the arrays of the call's sizes.
struct PlanSmem {
    int warp_sum[PLAN_WARPS];
    int counts[PLAN_CLUSTER];            // free pages of each block's part
    uint32_t bits[PLAN_CHUNK];           // free pages of a chunk
    int rank[PLAN_CHUNK];                // free pages before each word of it
};
inline size_t plan_smem_bytes(int n_new, int batch, bool fork) {
    return sizeof(PlanSmem) + 4 * (3 * static_cast<size_t>(n_new) + 1 + (fork ? 2 * static_cast<size_t>(batch) : 0));
}

// Exclusive scan of one value per thread; *total gets the block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                    // the last scan's readers are done
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    const int w = warp_sum[lane];       // 32 warps
    int ws = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o) ws += y;
    }
    *total = __shfl_sync(0xffffffffu, ws, 31);
    const int before = __shfl_sync(0xffffffffu, ws - w, warp);
    return before + x - v;
}

// Pages of a length, clipped to the table (recorded when it was outside).
__device__ __forceinline__ int pages_of(int n, const PagePlanParams& p) {
    const long long cap = static_cast<long long>(p.max_pages_per_seq) * p.page_size;
    if (n < 0 || n > cap) {
        report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return n < 0 ? 0 : p.max_pages_per_seq;
    }
    return static_cast<int>((static_cast<long long>(n) + p.page_size - 1) / p.page_size);
}

// Walks the first held(b) entries of `rows` table rows in runs of 32 x
// PLAN_RUN entries, a warp each: f(row, entry, page) with page = the entry's
// page, -1 where the row does not hold the entry or (recorded) where it lies
// outside the pool.
template <class Held, class Row, class F>
__device__ __forceinline__ void walk_tables(const PagePlanParams& p, int rows, Held held, Row row_of, F f) {
    const int lane = threadIdx.x & 31;
    const int width = p.max_pages_per_seq;
    constexpr int RUN = 32 * PLAN_RUN;
    const int runs = (width + RUN - 1) / RUN;
    const long long all = static_cast<long long>(rows) * runs;
    const int step = gridDim.x * PLAN_WARPS;
    for (long long u = blockIdx.x * PLAN_WARPS + (threadIdx.x >> 5); u < all; u += step) {
        const int b = static_cast<int>(u / runs), i0 = static_cast<int>(u - static_cast<long long>(b) * runs) * RUN + lane;
        const int n = held(b);
        const int32_t* row = p.page_table + static_cast<size_t>(row_of(b)) * width;
        int page[PLAN_RUN];
#pragma unroll
        for (int k = 0; k < PLAN_RUN; ++k) page[k] = i0 + 32 * k < n ? row[i0 + 32 * k] : -1;
#pragma unroll
        for (int k = 0; k < PLAN_RUN; ++k) {
            const int i = i0 + 32 * k;
            if (i >= width) break;
            if (i < n && (page[k] < 0 || page[k] >= p.num_pages)) {
                report_error(p.err, FA512_DEVICE_ERR_INDEX);
                page[k] = -1;
            }
            f(b, i, page[k]);
        }
    }
}

template <bool FORK>
__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(const PagePlanParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint8_t raw[];
    PlanSmem& s = *reinterpret_cast<PlanSmem*>(raw);
    int* s_off = reinterpret_cast<int*>(raw + sizeof(PlanSmem));   // fresh pages needed before sequence b
    int* s_from = s_off + p.n_new + 1;                             // fork: parent or -1; resize: pages held now
    int* s_held = s_from + p.n_new;                                // pages held by the new table
    int* s_first = s_held + p.n_new;                               // fork: first child of each parent
    int* s_len = s_first + p.batch;                                // fork: its length; ~length: its partly filled page is none
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, blocks = gridDim.x;               // the grid is one cluster
    const int gtid = rank * PLAN_THREADS + tid, all = blocks * PLAN_THREADS;
    const int width = p.max_pages_per_seq, ps = p.page_size;

    // ---- A: counts; needs
    if (p.new_refs != p.page_refs) {
        int done = 0;
        if (((reinterpret_cast<uintptr_t>(p.new_refs) | reinterpret_cast<uintptr_t>(p.page_refs)) & 15) == 0) {
            const int4* src = reinterpret_cast<const int4*>(p.page_refs);
            int4* dst = reinterpret_cast<int4*>(p.new_refs);
            const int quads = p.num_pages / 4;
            for (int i0 = gtid; i0 < quads; i0 += 4 * all) {
                int4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * all < quads) x[k] = src[i0 + k * all];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * all < quads) dst[i0 + k * all] = x[k];
            }
            done = quads * 4;
        }
        for (int i = done + gtid; i < p.num_pages; i += all) p.new_refs[i] = p.page_refs[i];
    }
    if constexpr (FORK) {
        // from the last thread down: the first ones copy a small pool's counts
        // meanwhile (4 sequences 9.5 -> 9.1 us)
        for (int a = PLAN_THREADS - 1 - tid; a < p.batch; a += PLAN_THREADS) {
            s_first[a] = INT_MAX;
            int n = p.kv_lens[a];
            n = n < 0 ? 0 : static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(width) * ps));
            if (n % ps != 0) {
                const int page = p.page_table[static_cast<size_t>(a) * width + n / ps];
                if (page < 0 || page >= p.num_pages) n = ~n;       // recorded in B
            }
            s_len[a] = n;
        }
        __syncthreads();
        for (int c = tid; c < p.n_new; c += PLAN_THREADS) {
            int a = p.parents[c];
            if (a < 0 || a >= p.batch) {
                if (rank == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
                a = -1;
            } else {
                atomicMin(&s_first[a], c);
            }
            s_from[c] = a;
        }
        __syncthreads();
    }
    int total = 0;
    for (int b0 = 0; b0 < p.n_new; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        int need = 0;
        if (b < p.n_new) {
            if constexpr (FORK) {
                const int a = s_from[b];
                int n = a >= 0 ? s_len[a] : 0;
                const bool copies = n >= 0 && n % ps != 0 && s_first[a] != b;
                need = copies ? 1 : 0;
                n = n < 0 ? ~n : n;
                s_held[b] = static_cast<int>((static_cast<long long>(n) + ps - 1) / ps);
                if (rank == 0) p.new_lens[b] = n;
            } else {
                s_from[b] = pages_of(p.kv_lens[b], p);
                s_held[b] = pages_of(p.next_lens[b], p);
                need = max(0, s_held[b] - s_from[b]);
            }
        }
        int sum;
        const int before = block_scan(need, s.warp_sum, &sum);
        if (b < p.n_new) s_off[b] = total + before;
        total += sum;
    }
    if (tid == 0) s_off[p.n_new] = total;
    cluster_sync_all();

    // ---- B: tables and counts
    if constexpr (FORK) {
        // a fresh last page is not the parent's: the table gets it in C
        walk_tables(
            p, p.n_new, [&](int c) { return s_held[c] - (s_off[c + 1] - s_off[c]); },
            [&](int c) { return max(s_from[c], 0); },
            [&](int c, int i, int page) {
                if (page >= 0) atomicAdd(&p.new_refs[page], 1);
                p.new_table[static_cast<size_t>(c) * width + i] = page;
            });
        walk_tables(
            p, p.batch, [&](int a) { return pages_of(p.kv_lens[a], p); }, [](int a) { return a; },
            [&](int, int, int page) {
                if (page >= 0) atomicAdd(&p.new_refs[page], -1);
            });
    } else {
        walk_tables(
            p, p.n_new, [&](int b) { return s_from[b]; }, [](int b) { return b; },
            [&](int b, int i, int page) {
                if (i >= s_held[b] && page >= 0) {
                    atomicAdd(&p.new_refs[page], -1);
                    page = -1;
                }
                p.new_table[static_cast<size_t>(b) * width + i] = page;
            });
    }
    if (total == 0) return;              // the same in every block: no fresh page to deal
    cluster_sync_all();

    // ---- C: free pages of this block's part, in chunks of the bit map
    const int words = (p.num_pages + 31) / 32;
    const int part = (words + blocks - 1) / blocks;
    const int lo = min(words, rank * part), hi = min(words, lo + part);
    auto mark = [&](int c0) -> int {     // fills s.bits with the words from c0 on; their number
        const int n = min(PLAN_CHUNK, hi - c0);
        for (int w0 = warp; w0 < n; w0 += PLAN_WARPS * PLAN_RUN) {
            int refs[PLAN_RUN];
#pragma unroll
            for (int k = 0; k < PLAN_RUN; ++k) {
                const int w = w0 + k * PLAN_WARPS, page = (c0 + w) * 32 + lane;
                refs[k] = w < n && page < p.num_pages ? __ldcg(&p.new_refs[page]) : 1;
            }
#pragma unroll
            for (int k = 0; k < PLAN_RUN; ++k) {
                const int w = w0 + k * PLAN_WARPS;
                const uint32_t free_bits = __ballot_sync(0xffffffffu, refs[k] == 0);
                if (lane == 0 && w < n) s.bits[w] = free_bits;
            }
        }
        __syncthreads();
        return n;
    };
    int part_free = 0;
    for (int c0 = lo; c0 < hi; c0 += PLAN_CHUNK) {
        const int n = mark(c0);
        int sum;
        block_scan(tid < n ? __popc(s.bits[tid]) : 0, s.warp_sum, &sum);
        part_free += sum;
        if (c0 + PLAN_CHUNK < hi) __syncthreads();
    }
    if (tid < blocks)
        pair::st_cluster_u32(map_to_cta(smem_u32(&s.counts[rank]), tid), static_cast<uint32_t>(part_free));
    cluster_sync_all();
    int base = 0, free_pages = 0;
    for (int r = 0; r < blocks; ++r) {
        if (r < rank) base += s.counts[r];
        free_pages += s.counts[r];
    }
    if (total > free_pages && rank == 0 && tid == 0) report_error(p.err, FA512_DEVICE_ERR_PAGES);
    const int top = 1 << (31 - __clz(p.n_new));                    // highest power of two up to n_new
    for (int c0 = lo; c0 < hi && base < total; c0 += PLAN_CHUNK) {
        const int n = hi - lo > PLAN_CHUNK ? mark(c0) : hi - lo;   // one chunk: its bits are still there
        int sum;
        const int before = block_scan(tid < n ? __popc(s.bits[tid]) : 0, s.warp_sum, &sum);
        if (tid < n) s.rank[tid] = base + before;
        __syncthreads();
        // four words a warp at a time, so that their searches overlap
        constexpr int DEAL = 4;
        for (int w0 = warp; w0 < n && s.rank[w0] < total; w0 += DEAL * PLAN_WARPS) {
            int r[DEAL], at[DEAL];
#pragma unroll
            for (int k = 0; k < DEAL; ++k) {
                const int w = w0 + k * PLAN_WARPS;
                const uint32_t free_bits = w < n ? s.bits[w] : 0u;
                r[k] = (free_bits >> lane) & 1u ? s.rank[w] + __popc(free_bits & ((1u << lane) - 1u)) : total;
                at[k] = 0;
            }
            // the last b with off[b] <= r
            for (int step = top; step > 0; step >>= 1)
#pragma unroll
                for (int k = 0; k < DEAL; ++k)
                    if (at[k] + step < p.n_new && s_off[at[k] + step] <= r[k]) at[k] += step;
#pragma unroll
            for (int k = 0; k < DEAL; ++k)
                if (r[k] < total) {
                    const int b = at[k], page = (c0 + w0 + k * PLAN_WARPS) * 32 + lane;
                    const int entry = FORK ? s_held[b] - 1 : s_from[b] + r[k] - s_off[b];
                    p.new_table[static_cast<size_t>(b) * width + entry] = page;
                    p.new_refs[page] = 1;
                }
        }
        base += sum;
        __syncthreads();
    }
}

// Fork: the filled rows of the last pages that children got fresh, one block
// per 32 KiB of one layer's K or V page.
constexpr int COPY_THREADS = 256;
constexpr int COPY_UNITS = 8;           // 16-byte units per thread

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const PagePlanParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.y;
    const int a = p.parents[c];
    if (a < 0 || a >= p.batch) return;
    const int n = p.new_lens[c], rem = n % p.page_size;
    const int units = p.row_bytes / 16;
    const long long live = static_cast<long long>(rem) * units;
    const long long u0 = static_cast<long long>(blockIdx.x) * (COPY_THREADS * COPY_UNITS) + threadIdx.x;
    if (u0 - threadIdx.x >= live) return;
    const int i = n / p.page_size;
    const int src = p.page_table[static_cast<size_t>(a) * p.max_pages_per_seq + i];
    const int dst = p.new_table[static_cast<size_t>(c) * p.max_pages_per_seq + i];
    if (dst < 0 || dst == src || src < 0 || src >= p.num_pages) return;
    const long long page_units = static_cast<long long>(p.page_size) * units;
    const int layer = blockIdx.z >> 1;
    uint4* base = reinterpret_cast<uint4*>((blockIdx.z & 1) ? p.v_pages : p.k_pages) +
                  static_cast<size_t>(layer) * p.num_pages * page_units;
    const uint4* from = base + src * page_units;
    uint4* to = base + dst * page_units;
    uint4 x[COPY_UNITS];
#pragma unroll
    for (int j = 0; j < COPY_UNITS; ++j)
        if (u0 + j * COPY_THREADS < live) x[j] = from[u0 + j * COPY_THREADS];
#pragma unroll
    for (int j = 0; j < COPY_UNITS; ++j)
        if (u0 + j * COPY_THREADS < live) to[u0 + j * COPY_THREADS] = x[j];
}

}  // namespace cache

cudaError_t launch_cache_append(const AppendParams& p, int element_bits, cudaStream_t stream) {
    using namespace cache;
    // scales that are powers of two with a normal reciprocal
    auto pow2 = [](float x) {
        int e;
        return frexpf(x, &e) == 0.5f && e > -100 && e < 100;
    };
    const bool both = element_bits != 16 && pow2(p.k_scale) && pow2(p.v_scale);
    AppendParams by = p;                                  // reciprocals in the place of the scales
    by.k_scale = 1.f / p.k_scale;
    by.v_scale = 1.f / p.v_scale;
    if (element_bits == 4) {
        const long long rows = static_cast<long long>(p.q_len) * p.n_kv_heads;
        constexpr int ROWS = APPEND_THREADS / 32;
        const dim3 grid(static_cast<unsigned>((rows + ROWS - 1) / ROWS), p.batch);
        if (both) append_fp4_kernel<true><<<grid, APPEND_THREADS, 0, stream>>>(by);
        else append_fp4_kernel<false><<<grid, APPEND_THREADS, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const bool fp8 = element_bits == 8;
    const long long units = static_cast<long long>(p.q_len) * p.n_kv_heads * (fp8 ? D / 16 : D / 8);
    constexpr int BLOCK = APPEND_THREADS * APPEND_RUN;
    const dim3 grid(static_cast<unsigned>((units + BLOCK - 1) / BLOCK), p.batch);
    if (!fp8) append_kernel<0><<<grid, APPEND_THREADS, 0, stream>>>(p);
    else if (both) append_kernel<2><<<grid, APPEND_THREADS, 0, stream>>>(by);
    else append_kernel<1><<<grid, APPEND_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

int compact_max_accepted() { return cache::COMPACT_MAX; }

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream) {
    using namespace cache;
    // a cache without layers has new lengths all the same
    const long long units = 2LL * (p.n_layers > 0 ? p.n_layers : 1) * (p.row_bytes / 16);
    const dim3 grid(static_cast<unsigned>((units + COMPACT_THREADS - 1) / COMPACT_THREADS), p.batch);
    compact_kernel<<<grid, COMPACT_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

int page_plan_max_batch() { return cache::PLAN_MAX_BATCH; }

// Most blocks of the plan's cluster on the current device, asked once per
// device (0: a query failed); it also opts the kernels into their shared
// memory and into clusters above the portable 8 there.
static int plan_blocks() {
    using namespace cache;
    static std::mutex mu;
    static int known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] != 0) return known[dev];
    const int smem = static_cast<int>(plan_smem_bytes(PLAN_MAX_BATCH, PLAN_MAX_BATCH, true));
    int fits = PLAN_CLUSTER;
    for (auto kernel : {page_plan_kernel<true>, page_plan_kernel<false>}) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3(PLAN_CLUSTER);
        cfg.blockDim = dim3(PLAN_THREADS);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = PLAN_CLUSTER;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            fits = 8;
        }
    }
    return known[dev] = fits;
}

cudaError_t launch_page_plan(const PagePlanParams& p, bool fork, cudaStream_t stream) {
    using namespace cache;
    auto kernel = fork ? page_plan_kernel<true> : page_plan_kernel<false>;
    const size_t smem = plan_smem_bytes(p.n_new, p.batch, fork);
    const int most = plan_blocks();
    if (most < 1) return cudaErrorLaunchOutOfResources;
    cudaError_t e;
    // a block for every 4,096 table entries and counts (4 per thread): 4 sequences
    // fork in 9.1 us with the blocks they need, in 9.4 with 8
    const long long work = static_cast<long long>(p.n_new + (fork ? p.batch : 0)) * p.max_pages_per_seq + p.num_pages;
    const int blocks = static_cast<int>(work >= most * 4096LL ? most : work / 4096 + 1);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(PLAN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess || !fork || p.n_new == 0 || p.n_layers == 0) return e;
    // the copies wait for the plan, scheduled while it runs
    const long long units = static_cast<long long>(p.page_size - 1) * (p.row_bytes / 16);
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>((units + COPY_THREADS * COPY_UNITS - 1) / (COPY_THREADS * COPY_UNITS)),
                       p.n_new, 2 * p.n_layers);
    cfg.blockDim = dim3(COPY_THREADS);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_copy_kernel, p);
}

}  // namespace fa512
