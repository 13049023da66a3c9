// Drafted tokens (a tree of them, or a plain run) over a paged cache, head
// dim 512, sm_103a.
//
// With start = len - cnt the last cnt cached positions are the tokens' own.
// Token t sees a key j < start always and a key start + c if its mask has bit
// c (no mask: c <= t); with a window, only keys whose place is above the
// token's place - window or below n_sinks, where the place of a cached key is
// its position and that of token t is start + (tokens it sees) - 1.
//
// A CTA takes 64 rows ((token, query head) pairs) of one KV head and one
// split of their key tiles of 128, and computes both products transposed on
// tcgen05: S^T = K Q^T (M = 128 keys, N = 64 rows, K = 512) and
// O^T += V^T P^T (four M = 128 blocks of the head dim, N = 64 rows, K = 128
// keys).  So the whole fp32 O of 64 rows takes 256 TMEM columns and leaves
// room for two S^T buffers, and the operands that are streamed, K and V, are
// read once from shared memory as they arrive:
//   K rows are the K-major A operand, V rows the MN-major A operand (its M
//   dimension, the head dim, is the contiguous one), Q stays in shared memory
//   as the K-major B operand, and P^T is written by the softmax threads as
//   an MN-major B operand: a thread holds one key, so its 64 (32) values are
//   contiguous.
// Per 128 keys the CTA streams 256 KiB (bf16): ~5.9 us at an SM's share of
// the measured HBM rate, against ~1.6 us of tensor work: HBM-bound for up to
// 64 rows; more rows share the keys through L2.
//
// The row maxima lie across lanes here, so they are not reduced every tile:
// each thread compares its scores with the reference its rows hold, and only
// when some score is above it by 2^THR (a vote at the tile's one barrier) do
// the four warps of a column half reduce the maxima and rescale O.  The row
// sums stay per-thread partials until the end.
//
// FP8 E4M3 cache: the bytes are MMA operands as stored (kind::f8f6f4).  Each
// query row is scaled by a power of two so that its largest element is in
// [128, 256) and written as the sum of two E4M3 terms (exact for elements
// above 2^-10 of the largest, off by at most 2^-18 of it below), and P as the
// sum of three E5M2 terms (relative error 2^-9, down to 2^-28 of the
// reference), so every product keeps at least the accuracy of the bf16 path
// without widening a byte of the cache.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_pair.cuh"

namespace fa512 {
namespace tree {

using pair::elect_one;
using pair::wait_or_abort;

constexpr int D = 512;
constexpr int MAX_NODES = 256;
constexpr int ROWS = 64;                 // rows of a CTA: N of both products
constexpr int TILE = 128;                // keys per tile: M of S^T
constexpr int SLOT = 16384;              // 128 keys x 128 bytes of the head dim
constexpr int NS = 8;                    // ring slots
constexpr int SOFTMAX_WARPS = 8;         // (TMEM lane quadrant, half of the rows)
constexpr int THREADS = 64 + SOFTMAX_WARPS * 32;
constexpr int HALF = ROWS / 2;

template <bool FP8>
struct Cfg {
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int CHUNKS = D * EB / 128;          // slots of a K (V) tile: 8 or 4
    static constexpr int Q_CHUNK = ROWS * 128;           // one 128-byte column chunk of Q
    static constexpr int Q_TERM = CHUNKS * Q_CHUNK;      // 64 or 32 KiB; FP8 holds two terms
    static constexpr int Q_TERMS = FP8 ? 2 : 1;
    static constexpr int P_LINE = ROWS * EB;             // bytes of a key's row values
    static constexpr int P_TERM = TILE * P_LINE;
    static constexpr int P_TERMS = FP8 ? 3 : 1;
    static constexpr float THR = FP8 ? 4.f : 8.f;        // log2 of the growth that rescales
    static constexpr float P_SCALE = FP8 ? 2048.f : 1.f; // keeps E5M2 terms of small p normal
    // shared memory, from a 1 KiB aligned base
    static constexpr int ring = 0;
    static constexpr int q = NS * SLOT;
    static constexpr int p = q + Q_TERMS * Q_TERM;
    static constexpr int mask = p + P_TERMS * P_TERM;    // [ROWS tokens][words]
    static constexpr int depth = mask + ROWS * (MAX_NODES / 32) * 4;
    static constexpr int red = depth + MAX_NODES * 4;    // [4][ROWS] float
    static constexpr int mult = red + 4 * ROWS * 4;      // [ROWS] float: score -> log2 units
    static constexpr int place = mult + ROWS * 4;        // [ROWS] int
    static constexpr int tok = place + ROWS * 4;         // [ROWS] int, -1: not a row
    static constexpr int bars = tok + ROWS * 4;
    static constexpr int FULL = 0, EMPTY = NS, S_FULL = 2 * NS, S_FREE = S_FULL + 2, P_FULL = S_FREE + 2,
                         PV_DONE = P_FULL + 1, DRAIN = PV_DONE + 1, N_BARS = DRAIN + 1;
    static constexpr int misc = bars + N_BARS * 8;       // tmem address, abort flag
    static constexpr int total = misc + 16;
};
static_assert(Cfg<false>::total + 1024 <= 232448 && Cfg<true>::total + 1024 <= 232448, "shared memory of an SM");

constexpr uint32_t TM_O = 0, TM_S = 256, TM_COLS = 512;

// D[tmem] (+)= A[smem] * B[smem]^T, 8-bit floating-point operands.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptors: M = 128, N = ROWS, fp32 accumulator.
constexpr uint32_t SHAPE = (1u << 4) | (static_cast<uint32_t>(ROWS >> 3) << 17) | (128u >> 4 << 24);
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;
constexpr uint32_t IDESC_QK16 = SHAPE | (1u << 7) | (1u << 10);                   // bf16 x bf16, both K-major
constexpr uint32_t IDESC_PV16 = IDESC_QK16 | A_MN | B_MN;
constexpr uint32_t IDESC_QK8 = SHAPE;                                             // e4m3 x e4m3
constexpr uint32_t IDESC_PV8 = SHAPE | (1u << 10) | A_MN | B_MN;                  // e4m3 x e5m2

// The same descriptor with 64-byte swizzle (rows of 64 bytes, 8-row atoms of 512 B).
__device__ __forceinline__ uint64_t make_sdesc_sw64(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    return (make_sdesc_sw128(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61)) | (4ull << 61);
}

// Named barrier over `count` threads that also ORs a predicate across them.
__device__ __forceinline__ bool bar_or(int id, int count, bool pred) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "barrier.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"(count), "r"(pred ? 1u : 0u) : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Reduces 32 values per lane over the warp's 32 lanes at once: lane i gets
// the reduction of everyone's v[i] (31 shuffles: halves swap the values that
// the other half keeps).
template <class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[32], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    return v[0];
}

// What a CTA knows of its sequence and rows.
struct Band {
    int len, cnt, start;        // cached positions, tokens, first token's position
    int lo, hi;                 // keys that some row may see: [lo, hi) and the sinks below n_sinks
    int sink_end;               // min(n_sinks, hi) with a window, else 0
    int sink_tiles, lo_tile;    // tile i of the band is tile i < sink_tiles ? i : lo_tile + i - sink_tiles
    int place_max;
    int first, n_tiles;         // this split's tiles
    __device__ __forceinline__ int key0(int i) const {
        const int g = first + i;
        return (g < sink_tiles ? g : lo_tile + g - sink_tiles) * TILE;
    }
};

// E4M3 pair of two fp32 values (low byte first) and the pair's values.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float& vlo, float& vhi) {
    uint16_t e;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(hi), "f"(lo));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(e));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(vlo), "=f"(vhi) : "r"(h2));
    return e;
}
__device__ __forceinline__ uint32_t e5m2_pair(float lo, float hi, float& vlo, float& vhi) {
    uint16_t e;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(e) : "f"(hi), "f"(lo));
    uint32_t h2;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(e));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(vlo), "=f"(vhi) : "r"(h2));
    return e;
}

template <bool FP8>
__global__ void __launch_bounds__(THREADS, 1)
tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
            const __grid_constant__ TreeParams p) {
    using C = Cfg<FP8>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    int* s_depth = reinterpret_cast<int*>(smem + C::depth);
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + C::mask);
    float* s_red = reinterpret_cast<float*>(smem + C::red);
    float* s_mult = reinterpret_cast<float*>(smem + C::mult);
    int* s_place = reinterpret_cast<int*>(smem + C::place);
    int* s_tok = reinterpret_cast<int*>(smem + C::tok);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row_tiles = (p.q_len * p.group + ROWS - 1) / ROWS;
    const int rt = blockIdx.x % row_tiles, split = blockIdx.x / row_tiles;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int G = p.group, W = p.mask_words;
    const int row0 = rt * ROWS;
    const int tok0 = row0 / G;                                   // first token of this row tile
    const int tok_last = min((row0 + ROWS - 1) / G, p.q_len - 1);

    // ---- lengths, masks and places
    Band bd;
    bd.len = p.kv_lens[b];
    bd.cnt = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bd.len < 0 || bd.len > p.len_cap || bd.cnt < 0 || bd.cnt > p.q_len) {
        if (tid == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        bd.len = max(0, min(bd.len, p.len_cap));
        bd.cnt = max(0, min(bd.cnt, p.q_len));
    }
    bd.start = bd.len - bd.cnt;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[C::FULL + i], 1);
            mbar_init(&bars[C::EMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[C::S_FULL + i], 1);
            mbar_init(&bars[C::S_FREE + i], SOFTMAX_WARPS);
        }
        mbar_init(&bars[C::P_FULL], SOFTMAX_WARPS);
        mbar_init(&bars[C::PV_DONE], 1);
        mbar_init(&bars[C::DRAIN], 1);
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
    }
    if (p.tree_mask) {
        // bits at and behind cnt name no token
        auto word = [&](int t, int w) -> uint32_t {
            const int left = bd.cnt - 32 * w;
            const uint32_t m = static_cast<uint32_t>(p.tree_mask[(static_cast<size_t>(b) * p.q_len + t) * W + w]);
            return left >= 32 ? m : left <= 0 ? 0u : m & ((1u << left) - 1u);
        };
        for (int t = tid; t < bd.cnt; t += THREADS) {
            int n = 0;
            for (int w = 0; w < W; ++w) n += __popc(word(t, w));
            s_depth[t] = n - 1;
        }
        const int toks = tok_last - tok0 + 1;
        for (int i = tid; i < toks * W; i += THREADS) {
            const int t = tok0 + i / W, w = i % W;
            s_mask[i] = t < bd.cnt ? word(t, w) : 0u;
        }
    }
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    {
        // places of the rows (every warp the same; warp 2 keeps them for the softmax)
        int pmin = INT_MAX, pmax = INT_MIN;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row0 + lane + 32 * i, t = r / G;
            const bool real = t < bd.cnt && bd.start + t >= 0;
            const int place = real ? bd.start + (p.tree_mask ? s_depth[t] : t) : 0;
            if (real) {
                pmin = min(pmin, place);
                pmax = max(pmax, place);
            }
            if (warp == 2) {
                s_place[lane + 32 * i] = place;
                s_tok[lane + 32 * i] = real ? t : -1;
            }
        }
        pmin = __reduce_min_sync(0xffffffffu, pmin);
        pmax = __reduce_max_sync(0xffffffffu, pmax);
        bd.place_max = pmax;
        bd.hi = pmax == INT_MIN ? 0 : p.tree_mask ? bd.len : min(bd.len, bd.start + min(tok_last, bd.cnt - 1) + 1);
        bd.lo = 0;
        bd.sink_end = 0;
        if (p.window > 0 && bd.hi > 0) {
            // a mask may name any token, so the tokens' own keys are always walked then
            bd.lo = max(0, p.tree_mask ? min(bd.start, pmin - p.window + 1) : pmin - p.window + 1);
            bd.sink_end = min(p.n_sinks, bd.hi);
        }
        bd.lo_tile = bd.lo / TILE;
        bd.sink_tiles = min((bd.sink_end + TILE - 1) / TILE, bd.lo_tile);
        const int all = bd.sink_tiles + (bd.hi + TILE - 1) / TILE - bd.lo_tile;
        const int per = (all + p.num_splits - 1) / p.num_splits;
        bd.first = split * per;
        bd.n_tiles = max(0, min(per, all - bd.first));
        if (bd.hi <= 0) bd.n_tiles = 0;
    }
    const int n = bd.n_tiles;
    // ring position of the first slot of K(t) and V(t): K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1)
    auto k_seq = [&](int t) { return (t == 0 ? 0 : 2 * t - 1) * C::CHUNKS; };
    auto v_seq = [&](int t) { return (t < n - 1 ? 2 * t + 2 : 2 * n - 1) * C::CHUNKS; };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // lane i < boxes brings the i-th run of box_rows positions of each slot
        const int box_rows = min(p.page_size, TILE), boxes = TILE / box_rows;
        auto row_of = [&](int t) -> int {
            const int oob = p.num_pages * p.page_size;       // past the pool: filled with zeros
            if (t >= n || lane >= boxes) return oob;
            const int pos = bd.key0(t) + lane * box_rows;
            const bool live = pos < bd.hi && (pos + box_rows > bd.lo || pos < bd.sink_end);
            if (!live) return oob;
            const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + pos / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                report_error(p.err, FA512_DEVICE_ERR_INDEX);
                return oob;
            }
            return page * p.page_size + pos % p.page_size;
        };
        int seq = 0;
        bool ok = true;
        auto load_tile = [&](const CUtensorMap* tm, int row) {
            for (int c = 0; c < C::CHUNKS && ok; ++c, ++seq) {
                const int s = seq % NS;
                if (seq >= NS &&
                    !__all_sync(0xffffffffu, wait_or_abort(&bars[C::EMPTY + s], ((seq / NS) & 1) ^ 1, p.err, abort))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&bars[C::FULL + s], SLOT);
                __syncwarp();
                if (lane < boxes)
                    tma_load_3d(smem + C::ring + s * SLOT + lane * box_rows * 128, tm, &bars[C::FULL + s],
                                c * (128 / C::EB), kvh, row);
            }
        };
        int cur = row_of(0), next = row_of(1);
        if (n > 0) load_tile(&tmk, cur);
        for (int t = 0; t < n && ok; ++t) {
            const int after = row_of(t + 2);                 // a tile ahead of its use
            if (t + 1 < n) load_tile(&tmk, next);
            if (ok) load_tile(&tmv, cur);
            cur = next;
            next = after;
        }
        // after an abort: no copy may land once this CTA has gone
        if (!ok)
            for (int i = max(0, seq - NS); i < seq; ++i)
                (void)mbar_wait(&bars[C::FULL + i % NS], (i / NS) & 1, p.err);
    } else {
        // ---- Q: 64 rows as K-major B operand, zeros where there is no row
        const int wid = warp - 1;                            // 0..8
        constexpr int QW = THREADS / 32 - 1;
        constexpr int PER = (ROWS + QW - 1) / QW;            // rows of a warp
        uint4 x[PER][2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = wid + i * QW, t = (row0 + r) / G;
            const bool real = r < ROWS && t < bd.cnt;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + ((static_cast<size_t>(b) * p.q_len + (real ? t : 0)) * p.n_q_heads + kvh * G +
                       (real ? (row0 + r) % G : 0)) * D) + 2 * lane;
            x[i][0] = real ? src[0] : make_uint4(0u, 0u, 0u, 0u);
            x[i][1] = real ? src[1] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = wid + i * QW;
            if (r >= ROWS) break;
            if constexpr (!FP8) {
                // this lane's 32 bytes: chunk lane / 4, pieces 2 (lane % 4) and + 1
                uint8_t* line = smem + C::q + (lane >> 2) * C::Q_CHUNK + r * 128;
                const int c = 2 * (lane & 3);
                *reinterpret_cast<uint4*>(line + ((c ^ (r & 7)) << 4)) = x[i][0];
                *reinterpret_cast<uint4*>(line + (((c + 1) ^ (r & 7)) << 4)) = x[i][1];
                if (lane == 0) s_mult[r] = p.scale_log2;
            } else {
                const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                                       x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                             fabsf(__uint_as_float(w[j] & 0xffff0000u))));
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                // 2^(7 - exponent of amax): the largest element comes to [128, 256)
                const int E = (__float_as_uint(amax) >> 23) & 0xff;
                const int biased = min(7 + 2 * 127 - E, 254);
                const float qs = (amax > 0.f && E < 255) ? __uint_as_float(static_cast<uint32_t>(biased) << 23) : 1.f;
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    hi[j] = lo[j] = 0u;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float a = __uint_as_float(w[2 * j + k] << 16) * qs;
                        const float c = __uint_as_float(w[2 * j + k] & 0xffff0000u) * qs;
                        float va, vc, ra, rc;
                        hi[j] |= e4m3_pair(a, c, va, vc) << (16 * k);
                        lo[j] |= e4m3_pair(a - va, c - vc, ra, rc) << (16 * k);
                    }
                }
                // this lane's 16 bytes: chunk lane / 8, piece lane % 8
                uint8_t* line = smem + C::q + (lane >> 3) * C::Q_CHUNK + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4*>(line) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(line + C::Q_TERM) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (lane == 0) s_mult[r] = p.scale_log2 / qs;
            }
        }
        fence_proxy_async_smem();
        bar_sync(3, THREADS - 32);

        if (warp == 1) {
            // -------------------------------------------------------------- MMA issue
            // the whole warp walks the tiles and waits; one elected lane issues
            const uint32_t ring = smem_u32(smem + C::ring);
            const uint64_t qd = make_sdesc_sw128(smem_u32(smem + C::q), 16, 1024);
            bool ok = true;
            auto wait = [&](int bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait_or_abort(&bars[bar], parity, p.err, abort));
            };
            auto issue_qk = [&](int t) -> bool {
                if (t >= 2 && !wait(C::S_FREE + (t & 1), ((t >> 1) & 1) ^ 1)) return false;
                const uint32_t sb = tmem + TM_S + static_cast<uint32_t>(t & 1) * ROWS;
                const int seq0 = k_seq(t);
                for (int c = 0; c < C::CHUNKS; ++c) {
                    const int s = (seq0 + c) % NS;
                    if (!wait(C::FULL + s, ((seq0 + c) / NS) & 1)) return false;
                    tc_fence_after_sync();
                    const uint64_t kd = make_sdesc_sw128(ring + s * SLOT, 16, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {            // 32 bytes of the head dim at a time
                            const uint64_t off = static_cast<uint64_t>(2 * k);
                            if constexpr (FP8) {
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    tc_mma_f8(sb, kd + off,
                                              qd + off + static_cast<uint64_t>((e * C::Q_TERM + c * C::Q_CHUNK) >> 4),
                                              IDESC_QK8, (c | k | e) ? 1u : 0u);
                            } else {
                                tc_mma_ss(sb, kd + off, qd + off + static_cast<uint64_t>((c * C::Q_CHUNK) >> 4),
                                          IDESC_QK16, (c | k) ? 1u : 0u);
                            }
                        }
                        tc_commit(&bars[C::EMPTY + s]);
                        if (c == C::CHUNKS - 1) tc_commit(&bars[C::S_FULL + (t & 1)]);
                    }
                    __syncwarp();
                }
                return true;
            };
            auto issue_pv = [&](int t) -> bool {
                if (!wait(C::P_FULL, t & 1)) return false;
                const uint64_t pd = FP8 ? make_sdesc_sw64(smem_u32(smem + C::p), 16, 512)
                                        : make_sdesc_sw128(smem_u32(smem + C::p), 16, 1024);
                const int seq0 = v_seq(t);
                constexpr int PER_M = C::CHUNKS / 4;             // slots of 128 head-dim elements
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    const int s = (seq0 + m * PER_M) % NS;       // two neighbours in the ring (bf16)
#pragma unroll
                    for (int j = 0; j < PER_M; ++j)
                        if (!wait(C::FULL + s + j, ((seq0 + m * PER_M) / NS) & 1)) return false;
                    tc_fence_after_sync();
                    const uint64_t vd = make_sdesc_sw128(ring + s * SLOT, SLOT, 1024);
                    const uint32_t ob = tmem + TM_O + static_cast<uint32_t>(m * ROWS);
                    if (elect_one()) {
                        if constexpr (FP8) {
#pragma unroll
                            for (int k = 0; k < TILE / 32; ++k)
#pragma unroll
                                for (int e = 0; e < C::P_TERMS; ++e)
                                    tc_mma_f8(ob, vd + static_cast<uint64_t>((k * 32 * 128) >> 4),
                                              pd + static_cast<uint64_t>((e * C::P_TERM + k * 32 * C::P_LINE) >> 4),
                                              IDESC_PV8, (t | k | e) ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int k = 0; k < TILE / 16; ++k)
                                tc_mma_ss(ob, vd + static_cast<uint64_t>((k * 16 * 128) >> 4),
                                          pd + static_cast<uint64_t>((k * 16 * C::P_LINE) >> 4), IDESC_PV16,
                                          (t | k) ? 1u : 0u);
                        }
#pragma unroll
                        for (int j = 0; j < PER_M; ++j) tc_commit(&bars[C::EMPTY + s + j]);
                        if (m == 3) tc_commit(&bars[C::PV_DONE]);
                    }
                    __syncwarp();
                }
                return true;
            };
            if (n > 0) ok = issue_qk(0);
            for (int t = 0; t < n && ok; ++t) {
                if (t + 1 < n) ok = issue_qk(t + 1);
                if (ok) ok = issue_pv(t);
            }
            if (elect_one()) tc_commit(&bars[C::DRAIN]);
            __syncwarp();
            (void)mbar_wait(&bars[C::DRAIN], 0, p.err);
        } else {
            // ---------------------------------------------------------------- softmax
            const int quad = warp & 3, half = warp >= 6 ? 1 : 0;
            const int bar = 1 + half;                        // the half's four warps
            const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
            const int kk = quad * 32 + lane;                 // this thread's key of a tile
            const int col0 = half * HALF;                    // its rows
            float m[HALF], l[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            bool ok = true;
            for (int t = 0; t < n; ++t) {
                const int key0 = bd.key0(t), key = key0 + kk;
                ok = ok && wait_or_abort(&bars[C::S_FULL + (t & 1)], (t >> 1) & 1, p.err, abort);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after_sync();
                float x[HALF];
                {
                    uint32_t raw[32];
                    tmem_ld32(tmem + lanes + TM_S + static_cast<uint32_t>((t & 1) * ROWS + col0), raw);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < HALF; ++i) x[i] = __uint_as_float(raw[i]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::S_FREE + (t & 1)]);
#pragma unroll
                for (int i = 0; i < HALF; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&s_mult[col0 + i]);
                    x[i] *= f.x;
                    x[i + 1] *= f.y;
                    x[i + 2] *= f.z;
                    x[i + 3] *= f.w;
                }
                // a tile of cached keys inside every row's window needs no mask
                const bool whole = key0 + TILE <= bd.start &&
                                   (p.window <= 0 || key0 > bd.place_max - p.window || key0 + TILE <= bd.sink_end);
                // keys that no row sees: their V rows may hold anything
                bool live = true;
                if (!whole) {
                    live = key < bd.hi && (key >= bd.lo || key < bd.sink_end);
                    const int c = key - bd.start;
                    const int kp = c < 0 || !p.tree_mask ? key : bd.start + s_depth[min(c, MAX_NODES - 1)];
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        const int tk = s_tok[col0 + i], pl = s_place[col0 + i];
                        bool see = live && tk >= 0;
                        if (see && c >= 0)
                            see = p.tree_mask ? (s_mask[(tk - tok0) * W + (c >> 5)] >> (c & 31)) & 1u : c <= tk;
                        if (p.window > 0) see = see && (kp > pl - p.window || kp < p.n_sinks);
                        x[i] = see ? x[i] : -INFINITY;
                    }
                }
                bool over = !ok;
#pragma unroll
                for (int i = 0; i < HALF; ++i) over = over || x[i] > m[i] + C::THR;
                bool pv_waited = t == 0;
                if (bar_or(bar, 128, over)) {
                    if (!(ok = pair::bar_and(bar, 128, ok))) break;
                    float v[HALF];
#pragma unroll
                    for (int i = 0; i < HALF; ++i) v[i] = x[i];
                    const float mx = reduce_columns(v, [](float a, float c) { return fmaxf(a, c); });
                    s_red[quad * ROWS + col0 + lane] = mx;
                    bar_sync(bar, 128);
                    const float top = fmaxf(fmaxf(s_red[col0 + lane], s_red[ROWS + col0 + lane]),
                                            fmaxf(s_red[2 * ROWS + col0 + lane], s_red[3 * ROWS + col0 + lane]));
                    float mine = 1.f;                        // lane i: the factor of row col0 + i
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        const float mn = fmaxf(m[i], __shfl_sync(0xffffffffu, top, i));
                        const float a = mn == -INFINITY ? 1.f : fast_exp2(m[i] - mn);
                        l[i] *= a;
                        m[i] = mn;
                        mine = lane == i ? a : mine;
                    }
                    if (t > 0) {
                        // O is at rest once P V of the last tile has completed
                        ok = wait_or_abort(&bars[C::PV_DONE], (t - 1) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, ok);
                        pv_waited = true;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int o = 0; o < 4; ++o) {
                            const uint32_t ta = tmem + lanes + TM_O + static_cast<uint32_t>(o * ROWS + col0);
                            uint32_t r[32];
                            tmem_ld32(ta, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < HALF; ++i) 
                                r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xffffffffu, mine, i));
                            tmem_st32(ta, r);
                        }
                        tmem_st_wait();
                    }
                    bar_sync(bar, 128);                      // s_red is free again
                }
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    x[i] = fast_exp2(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
                    l[i] += x[i];
                }
                // P's buffer is free, and V of this tile will be read, after P V of the last tile
                if (!pv_waited) {
                    ok = wait_or_abort(&bars[C::PV_DONE], (t - 1) & 1, p.err, abort);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if constexpr (FP8) {
                    uint8_t* line = smem + C::p + kk * C::P_LINE;
#pragma unroll
                    for (int c = 0; c < HALF / 16; ++c) {
                        uint32_t w[3][4] = {};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float a = x[16 * c + 2 * j] * C::P_SCALE, d = x[16 * c + 2 * j + 1] * C::P_SCALE;
#pragma unroll
                            for (int e = 0; e < 3; ++e) {
                                float va, vd;
                                w[e][j >> 1] |= e5m2_pair(a, d, va, vd) << (16 * (j & 1));
                                a -= va;
                                d -= vd;
                            }
                        }
                        const int piece = ((col0 / 16 + c) ^ ((kk >> 1) & 3)) << 4;
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            *reinterpret_cast<uint4*>(line + e * C::P_TERM + piece) =
                                make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                    }
                } else {
                    uint8_t* line = smem + C::p + kk * C::P_LINE;
#pragma unroll
                    for (int c = 0; c < HALF / 8; ++c)
                        *reinterpret_cast<uint4*>(line + (((col0 / 8 + c) ^ (kk & 7)) << 4)) =
                            make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                                       pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
                }
                // P = 0 must not meet stale or poisoned V rows: each half's
                // threads clear their key's row in half of the tile's slots.
                // Before V(t) a slot held K(t + 1): S^T of that tile says that
                // it has been read, so the wait for V(t) is one phase ahead
                // at most.
                if (!whole && pair::bar_and(bar, 128, live) == false) {
                    if (t + 1 < n) {
                        const bool got = wait_or_abort(&bars[C::S_FULL + ((t + 1) & 1)], ((t + 1) >> 1) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                    }
                    const int seq0 = v_seq(t) + half * (C::CHUNKS / 2);
#pragma unroll 1
                    for (int j = 0; j < C::CHUNKS / 2; ++j) {
                        const int s = (seq0 + j) % NS;
                        const bool got = wait_or_abort(&bars[C::FULL + s], ((seq0 + j) / NS) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                        if (got && !live) {
                            uint4* line = reinterpret_cast<uint4*>(smem + C::ring + s * SLOT + kk * 128);
#pragma unroll
                            for (int e = 0; e < 8; ++e) line[e] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::P_FULL]);
            }
            if (n > 0 && ok)
                ok = wait_or_abort(&bars[C::PV_DONE], (n - 1) & 1, p.err, abort);
            ok = pair::bar_and(bar, 128, ok);
            tc_fence_after_sync();
            // ---- row sums: lanes, then the four quadrants' warps
            const float part = reduce_columns(l, [](float a, float c) { return a + c; });
            s_red[quad * ROWS + col0 + lane] = part;
            bar_sync(bar, 128);
            const float sum = (s_red[col0 + lane] + s_red[ROWS + col0 + lane]) +
                              (s_red[2 * ROWS + col0 + lane] + s_red[3 * ROWS + col0 + lane]);
            float top = -INFINITY;                           // lane i: row col0 + i
#pragma unroll
            for (int i = 0; i < HALF; ++i) top = lane == i ? m[i] : top;
            const int my_row = row0 + col0 + lane, my_tok = my_row / G;
            const bool mine = my_tok < p.q_len;
            const bool some = ok && s_tok[col0 + lane] >= 0 && top != -INFINITY;
            const size_t my_out = (static_cast<size_t>(b) * p.q_len + my_tok) * p.n_q_heads + kvh * G + my_row % G;
            const size_t S = static_cast<size_t>(p.num_splits);
            // O / sum where this is the whole row, else the unnormalised partial
            const float unit = p.o_scale * (1.f / C::P_SCALE);
            const float factor = !some ? 0.f : p.num_splits == 1 ? unit / sum : unit;
            if (quad == 0 && mine) {
                if (p.num_splits == 1) {
                    if (p.lse) p.lse[my_out] = some ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
                } else {
                    p.ws_ml[(my_out * S + split) * 2] = some ? top : -INFINITY;
                    p.ws_ml[(my_out * S + split) * 2 + 1] = some ? sum : 0.f;
                }
            }
#pragma unroll 1
            for (int o = 0; o < 4; ++o) {
                uint32_t r[32];
                if (n > 0) {
                    tmem_ld32(tmem + lanes + TM_O + static_cast<uint32_t>(o * ROWS + col0), r);
                    tmem_ld_wait();
                }
                const int d = o * 128 + kk;
#pragma unroll
                for (int i = 0; i < HALF; ++i) {
                    const float f = __shfl_sync(0xffffffffu, factor, i);
                    const size_t row = __shfl_sync(0xffffffffu, my_out, i);
                    const bool there = __shfl_sync(0xffffffffu, mine ? 1 : 0, i);
                    if (!there) continue;
                    const float val = f != 0.f ? __uint_as_float(r[i]) * f : 0.f;
                    if (p.num_splits == 1)
                        p.out[row * D + d] = __float2bfloat16_rn(val);
                    else
                        p.ws_o[(row * S + split) * D + d] = val;
                }
            }
            tc_fence_before_sync();
        }
    }
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, TM_COLS);
}

template <bool FP8>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    const int smem = Cfg<FP8>::total + 1024;
    cudaError_t e = cudaFuncSetAttribute(tree_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int row_tiles = (p.q_len * p.group + ROWS - 1) / ROWS;
    const dim3 grid(row_tiles * p.num_splits, p.n_kv_heads, p.batch);
    tree_kernel<FP8><<<grid, THREADS, smem, stream>>>(tmk, tmv, p);
    return cudaGetLastError();
}

}  // namespace tree

int tree_max_nodes() { return tree::MAX_NODES; }
int tree_rows() { return tree::ROWS; }
int tree_tile() { return tree::TILE; }

cudaError_t launch_decode_tree(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                               cudaStream_t stream) {
    const cudaError_t e = fp8 ? tree::launch<true>(tmk, tmv, p, stream) : tree::launch<false>(tmk, tmv, p, stream);
    if (e != cudaSuccess || p.num_splits == 1) return e;
    DecodeParams m;
    memset(&m, 0, sizeof m);
    m.ws_o = p.ws_o;
    m.ws_ml = p.ws_ml;
    m.out = p.out;
    m.lse = p.lse;
    m.batch = p.batch;
    m.q_len = p.q_len;
    m.n_q_heads = p.n_q_heads;
    m.num_splits = p.num_splits;
    return launch_decode_merge(m, stream);
}

}  // namespace fa512
