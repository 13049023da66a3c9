// Paged decode over ranges of key tiles, sm_103a: caches held in 4 bits, and selected
// pages of a cache in any format.
//
// The key tiles of all sequences stand in a row and are dealt in ranges of equal length
// to groups of CTAs, one CTA for each KV head, two CTAs to an SM for the whole launch;
// what a CTA has of a sequence is a segment, with an (O, m, l) partial of its own.  (The
// heads of a position lie side by side: read at about the same time they share the
// memory's lines.  Ranges that did not keep the heads together took 997 us instead of
// 741 for 64 sequences of 28,672 positions in 4 bits.)  With a list of pages the tiles
// are counted along it.  Ranges are long enough that no sequence is left in more than
// num_splits segments, the places that its partials have: the host's choice of those is
// for lengths between half of max_kv_len and all of it.
//
// K and V rows come by TMA, two warps' work, into rings of slots that run on across
// segments.  Four warps form S^T = K Q^T, a block of 16 positions at a time over the
// whole head dim with the query rows in N, and their softmax against a reference of
// their own, and leave P^T and the reference in shared memory; four other warps add
// V^T P^T of all blocks of the tile, 128 columns of O each.  Nothing is computed twice,
// and the groups only meet at barriers in shared memory with tiles of slack, so that
// both products of different tiles overlap.  (64 sequences of 28,672 positions in 4
// bits: one group of warps that did both in turn 846 us, two groups 775, the group
// scales in free columns for 2 rows 707, loads on warps of their own 649, references
// that seldom change 641, Q in shared memory and registers where they are needed 622,
// values' scales back on their codes 622 to 627: 6.8 TB/s.  9 to 16 rows spill a few
// registers: 64 x 8,192, 16 heads over 1, 83 us for 45 us of bytes; 32 over 4 with 2
// tokens 278 for 178.)  References are whole numbers in log2 units: what brings two of them
// together is a power of two, exact in f16 and bf16.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "decode_ranges.cuh"
#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_list.cuh"

namespace fa512 {
namespace ranges {

constexpr int THREADS = 3 * WARPS * 32;          // K group, V group, loads
constexpr int CTAS_PER_SM = 2;
constexpr int META = 16;                         // tiles and segments whose notes are kept

template <int BITS, int NT>
struct Smem {
    using F = Format<BITS>;
    // Slots of K, and of V.  Three, more loads in flight, are slower but for bf16 (E4M3, 48
    // sequences, 32 pages of 64, 2 heads: 45.9 us, with two 43.6; 64 x 64 pages of 64: E4M3
    // 165 and 166, bf16 307 and 310).  In 4 bits they took 654 us instead of 645 for 64 x
    // 28,672 positions when Q still left room for them.
    static constexpr int slots = NT == 1 && BITS == 16 ? 3 : 2;
    // A K warp takes every turns-th tile.  K's `full` barriers go by tiles, not slots, so
    // that each is one warp's own, which then sees all of its phases: the first common
    // multiple of both counts.
    static constexpr int turns = WARPS / F::BLOCKS;
    static constexpr int k_bars = slots % turns == 0 ? slots : turns == 2 || slots % 2 ? slots * turns : slots * turns / 2;
    static_assert(k_bars % slots == 0 && k_bars % turns == 0, "a common multiple");
    static constexpr int k = 0;
    static constexpr int v = slots * F::SLOT;
    static constexpr int p = 2 * slots * F::SLOT;            // [buffer][block][nt][lane] uint2
    static constexpr int q = p + F::P_BUFFERS * F::BLOCKS * NT * 32 * 8;    // [nt][kstep][lane] uint2
    static constexpr int ref = q + NT * KSTEPS * 32 * 8;    // [buffer][block][8 NT] float
    static constexpr int sums = ref + F::P_BUFFERS * F::BLOCKS * 8 * NT * 4;   // [parity][warp][8 NT] float2: reference, sum
    static constexpr int base = sums + 2 * WARPS * 8 * NT * 8;              // [META][BLOCKS] first position of 16
    static constexpr int seg = base + META * F::BLOCKS * 4;                 // [META] Segment
    static constexpr int total_tiles = seg + META * 16;
    static constexpr int bar = total_tiles + 8;
    // barriers: K and V slots full and empty, P buffers full and empty
    static constexpr int total = bar + (k_bars + 3 * slots + 2 * F::P_BUFFERS) * 8;
    static_assert(CTAS_PER_SM * (total + 1024) <= 228 * 1024, "the CTAs fit an SM's shared memory");
};

// A reference to subtract: 0 while nothing was seen, so that 2^(-inf - 0) = 0.
__device__ __forceinline__ float finite_ref(float x) { return x == -INFINITY ? 0.f : x; }

struct Item {
    int len;                                      // live positions
    int lo;                                       // first position that some row sees
    int tiles;                                    // LIST: along the list of pages
    int held;                                     // pages
};
template <int BITS, bool LIST>
__device__ __forceinline__ Item item_with(const DecodeParams& p, int len) {
    Item x;
    x.len = min(max(len, 0), p.len_cap);
    // union of the rows' bands (the row of token t sees [pos - window + 1, pos])
    const int w_lo = x.len - p.q_len + 1 - p.window;
    x.lo = p.window > 0 && w_lo > 0 ? w_lo : 0;
    x.held = static_cast<int>((static_cast<unsigned>(x.len) + p.page_size - 1) >> p.page_shift);
    const int end = LIST ? min(p.n_listed, x.held) << p.page_shift : x.len;
    constexpr int TILE = Format<BITS>::TILE;
    x.tiles = (end + TILE - 1) / TILE - x.lo / TILE;
    return x;
}
template <int BITS, bool LIST>
__device__ __forceinline__ Item item_of(const DecodeParams& p, int b) {
    return item_with<BITS, LIST>(p, p.kv_lens[b]);
}

// What the loading warp notes of a segment.
struct Segment {
    int b, len;                                   // sequence, live positions
    int run;                                      // tiles
    int index;                                    // of the sequence's segments, + LAST for its last one
    static constexpr int LAST = 1 << 30;
};

// A CTA's way through its range of tiles.
template <int BITS, bool LIST>
struct Walk {
    int b;                                        // sequence
    Item item;
    int tile;                                     // its next tile
    int start;                                    // tiles of the sequences before it
    int left;                                     // tiles of the range that are left
    __device__ __forceinline__ int run() const { return min(item.tiles - tile, left); }   // those of this sequence
    __device__ __forceinline__ void next(const DecodeParams& p, int n) {
        tile += n;
        left -= n;
        while (left > 0 && tile == item.tiles) {
            start += item.tiles;
            tile = 0;
            item = item_of<BITS, LIST>(p, ++b);
        }
    }
};

// Where the `index`-th of `groups` ranges begins, and the length of the ranges.
// num_splits = 1: ranges of whole sequences.  All lanes of a warp together.
template <int BITS, bool LIST>
__device__ __forceinline__ Walk<BITS, LIST> first_of_range(const DecodeParams& p, int index, int groups, int* range) {
    const int lane = threadIdx.x & 31;
    Walk<BITS, LIST> w;
    w.b = w.tile = w.start = w.left = 0;
    *range = 0x7fffffff;
    if (p.num_splits == 1) {
        const int per = (p.batch + groups - 1) / groups;
        const int begin = min(p.batch, index * per), end = min(p.batch, begin + per);
        if (begin == end) return w;
        int left = 0;
        for (int b = begin + lane; b < end; b += 32) left += item_of<BITS, LIST>(p, b).tiles;
        w.left = __reduce_add_sync(0xffffffffu, left);
        w.b = begin;
        w.item = item_of<BITS, LIST>(p, begin);
        w.next(p, 0);                             // past sequences without a tile
        return w;
    }
    int total = 0, len = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        len = b0 + lane < p.batch ? p.kv_lens[b0 + lane] : 0;
        total += __reduce_add_sync(0xffffffffu, item_with<BITS, LIST>(p, len).tiles);
    }
    const int r = max((total + groups - 1) / groups, p.tiles_per_split);
    const long long at = static_cast<long long>(index) * r;
    if (at >= total) return w;
    *range = r;
    w.left = min(r, total - static_cast<int>(at));
    // the sequence that the range begins in
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        if (p.batch > 32) len = b0 + lane < p.batch ? p.kv_lens[b0 + lane] : 0;
        const int n = item_with<BITS, LIST>(p, len).tiles;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned here = __ballot_sync(0xffffffffu, w.start + sum > static_cast<int>(at));
        if (here) {
            const int l = __ffs(here) - 1;
            w.b = b0 + l;
            w.start += __shfl_sync(0xffffffffu, sum - n, l);
            w.item = item_with<BITS, LIST>(p, __shfl_sync(0xffffffffu, len, l));
            break;
        }
        w.start += __shfl_sync(0xffffffffu, sum, 31);
    }
    w.tile = static_cast<int>(at) - w.start;
    return w;
}

// ROWS: the most query rows (q_len * G) of a KV head, in NT n-tiles of 8.
//
// Up to 2 rows leave six of the eight columns of an n-tile free, and the keys' group
// scales move there (NARROW): column 2 c + r belongs to row r and scale class c.
//   S^T: lane t holds K codes of groups 4 j + t, so with Q zero outside class t a
//        lane's sums of step j are those of its own group, and take its scale in
//        fp32: 32 multiply-adds a tile where scaling the codes takes 128.
//   O^T: the weights of row r stand in all columns 2 c + r, so that every lane has O,
//        of which it writes a quarter.
template <int BITS, int ROWS, bool LIST>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM)
decode_ranges_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const DecodeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int NT = ROWS > 8 ? 2 : 1;
    constexpr bool NARROW = ROWS == 2;
    static_assert(!NARROW || BITS == 4, "only group scales take free columns");
    using F = Format<BITS>;
    constexpr int TILE = F::TILE, BLOCKS = F::BLOCKS, P_BUFFERS = F::P_BUFFERS;
    using Smem = ranges::Smem<BITS, NT>;
    constexpr int SLOTS = Smem::slots, TURNS = Smem::turns, K_BARS = Smem::k_bars;
    static_assert(P_BUFFERS % TURNS == 0, "a P buffer is one K warp's own");
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {                // the swizzle goes by addresses
        if (threadIdx.x == 0) report_error(p.err, FA512_DEVICE_ERR_LAYOUT);
        return;
    }
    uint2* s_p = reinterpret_cast<uint2*>(smem + Smem::p);
    uint16_t* s_p2 = reinterpret_cast<uint16_t*>(smem + Smem::p);   // NARROW: [buffer][block][row][16]
    uint2* s_q = reinterpret_cast<uint2*>(smem + Smem::q);
    float* s_ref = reinterpret_cast<float*>(smem + Smem::ref);
    float2* s_sums = reinterpret_cast<float2*>(smem + Smem::sums);
    int* s_base = reinterpret_cast<int*>(smem + Smem::base);
    Segment* s_seg = reinterpret_cast<Segment*>(smem + Smem::seg);
    int* s_total = reinterpret_cast<int*>(smem + Smem::total_tiles);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Smem::bar);
    uint64_t *k_empty = k_full + K_BARS, *v_full = k_empty + SLOTS, *v_empty = v_full + SLOTS, *p_full = v_empty + SLOTS,
             *p_empty = p_full + P_BUFFERS;

    const int lane = threadIdx.x & 31;
    const int warp = (threadIdx.x >> 5) & (WARPS - 1);   // within its group
    const int role = threadIdx.x / (WARPS * 32); // 0 K group, 1 V group, 2 loads
    const int g = lane >> 2, t = lane & 3;       // mma fragment coordinates
    const int G = p.group, R = p.q_len * G;      // query rows: (token, head) -> token * G + head
    const int ps = p.page_size;
    const int S = p.num_splits;
    const int kvh = blockIdx.x % p.n_kv_heads, index = blockIdx.x / p.n_kv_heads;
    auto row_index = [&](int b, int r) {
        return (static_cast<size_t>(b) * p.q_len + r / G) * p.n_q_heads + kvh * G + r % G;
    };

    auto done_with = [&](uint64_t* bar) {        // this warp has read what the barrier guards
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // Every wait of a warp that follows another role's phase of a barrier guards what
    // that role cannot pass before this warp has arrived, so a phase is never missed.
    auto wait = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, p.err)) != 0; };
    bool ok = true;                              // the same in all lanes of a warp
    int loaded = 0;                              // tiles whose load this warp has issued

    // The launch's 80 registers a thread are dealt anew: a share for each role, the K
    // group's and the V group's no less than 80, the loads' no more, as the instructions
    // that take and give them ask.  (64 x 28,672 positions in 4 bits, K, V and loads: 128,
    // 80, 32 with Q in registers 641 us; with Q in shared memory 104, 96, 40 630; 88, 104,
    // 48 623; 88, 88, 64 630.)
    constexpr int LAUNCH_REGS = 80, K_REGS = 88, V_REGS = 104, LOAD_REGS = 48;
    static_assert(K_REGS + V_REGS + LOAD_REGS <= 3 * LAUNCH_REGS, "no more than the launch has");
    static_assert(K_REGS >= LAUNCH_REGS && V_REGS >= LAUNCH_REGS && LOAD_REGS <= LAUNCH_REGS, "taken, taken, given");
    if (role == 0) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(K_REGS));
        // ---- Q^T fragments, bf16 as stored, else in f16 after a power-of-two scale per row
        // that keeps its largest element below 2^15 (exact down to 2^-32 of that, where all 8
        // bits of an element still fit, and off by at most 2^-40 of it below; a score is
        // unscaled before the softmax)
        float rs[NT][2];                          // 1 / scale of rows row_of(n, 0), row_of(n, 1)
        auto load_q = [&](int b) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // each warp writes a quarter of the k-steps, all of them find the maxima
                const int r = NARROW ? g & 1 : 8 * n + g;
                const bool row_ok = r < R;
                const uint4* src = reinterpret_cast<const uint4*>(p.q + row_index(b, row_ok ? r : 0) * D);
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 a = row_ok ? src[BITS == 16 ? 8 * j + 4 * e + t : 8 * j + 2 * t + e] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
                    }
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // 2^(14 - E), E = exponent of the maximum (0 or not finite: 1)
                const int E = (__float_as_uint(most) >> 23) & 0xff;
                const int biased = min(127 + 14 + 127 - E, 254);
                const float scale = (BITS != 16 && most > 0.f && E < 255) ? __uint_as_float(static_cast<uint32_t>(biased) << 23) : 1.f;
                auto to_f16 = [&](uint32_t w) {
                    if constexpr (BITS == 16) return w;
                    else return pack_f16x2(__uint_as_float(w << 16) * scale, __uint_as_float(w & 0xffff0000u) * scale);
                };
                const bool mine = row_ok && (!NARROW || g >> 1 == t);
#pragma unroll
                for (int j = 2 * warp; j < 2 * warp + 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 a = mine ? src[BITS == 16 ? 8 * j + 4 * e + t : 8 * j + 2 * t + e] : make_uint4(0u, 0u, 0u, 0u);
                        s_q[(n * KSTEPS + 4 * j + 2 * e) * 32 + lane] = make_uint2(to_f16(a.x), to_f16(a.y));
                        s_q[(n * KSTEPS + 4 * j + 2 * e + 1) * 32 + lane] = make_uint2(to_f16(a.z), to_f16(a.w));
                    }
                rs[n][0] = 1.f / __shfl_sync(0xffffffffu, scale, NARROW ? 0 : 4 * (2 * t));
                rs[n][1] = 1.f / __shfl_sync(0xffffffffu, scale, NARROW ? 4 : 4 * (2 * t + 1));
            }
        };
        auto k_warps = [&]() {                    // the group meets, and agrees on whether to go on
            uint32_t bad;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                         "bar.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(bad)
                         : "r"(ok ? 0u : 1u), "n"(WARPS * 32)
                         : "memory");
            ok = bad == 0;
        };
        // this lane's rows: i (NARROW) or 8 n + 2 t + i
        auto row_of = [&](int n, int i) { return NARROW ? i : 8 * n + 2 * t + i; };
        const unsigned reach = p.window > 0 ? static_cast<unsigned>(p.window) : 0x7fffffffu;
        const int ra = F::order(g);               // this lane's rows of 16 positions: ra, ra + 8
        const int block = warp % BLOCKS, turn = warp / BLOCKS;   // which of a tile, and of which tiles
        int range;
        const int first_b = first_of_range<BITS, LIST>(p, index, gridDim.x / p.n_kv_heads, &range).b;
        load_q(first_b);                          // (of sequence 0 where the range is empty)
        __syncthreads();                          // barriers, the first tiles' notes, the queries
        const int total = *s_total;

        int it = 0;                               // tiles of the range gone through
        for (int segment = 0; it < total && ok; ++segment) {
            if (segment > 0) {
                load_q(s_seg[segment % META].b);
                k_warps();
            }
            const Segment seg = s_seg[segment % META];
            // positions of the rows (-1: padding row, sees nothing); a row sees the keys
            // whose distance to it is in [0, reach)
            int qpos[NT][2];
            float m[NT][2], l[NT][2];             // this warp's running reference and sum (a lane's part) of those rows
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = row_of(n, i);
                    qpos[n][i] = r < R ? seg.len - p.q_len + r / G : -1;
                    m[n][i] = -INFINITY;
                    l[n][i] = 0.f;
                }
            const int end = it + seg.run;
            for (; it < end; ++it) {
                if (it % TURNS != turn) continue;
                const int slot = it % SLOTS, buffer = it % P_BUFFERS;
                if (!wait(&k_full[it % K_BARS], it / K_BARS)) {
                    ok = false;
                    break;
                }
                const int base = s_base[(it % META) * BLOCKS + block];
                // (an unloaded block's rows are stale: its scores are masked)
                float sc[NT][4];
                const uint8_t* rows = smem + Smem::k + slot * F::SLOT;
                if constexpr (NARROW) scores_narrow(rows + 16 * block * F::ROW, lane, s_q, sc[0]);
                else if constexpr (BITS == 4) scores_4<NT>(rows + 16 * block * F::ROW, lane, s_q, sc);
                else if constexpr (BITS == 8) scores_8<NT>(rows, 16 * block, lane, s_q, sc);
                else scores_16<NT>(rows, lane, s_q, sc);
                done_with(&k_empty[slot]);
                // ---- softmax against this warp's reference, which rises where a weight would pass
                // 2^7, to the block's maximum rounded up to a whole number, less 3: few blocks raise it
                const int kp = base + ra;
                uint2 frag[NT];
                float sv[NT][2][2];
                bool above = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool va = base >= 0 && static_cast<unsigned>(qpos[n][i] - kp) < reach;
                        const bool vb = base >= 0 && static_cast<unsigned>(qpos[n][i] - kp - 8) < reach;
                        sv[n][i][0] = va ? sc[n][i] * rs[n][i] * p.scale_log2 : -INFINITY;
                        sv[n][i][1] = vb ? sc[n][2 + i] * rs[n][i] * p.scale_log2 : -INFINITY;
                        above |= fmaxf(sv[n][i][0], sv[n][i][1]) - m[n][i] > 7.f;   // (a sum with m may round)
                    }
                if (__any_sync(0xffffffffu, above))
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float most = fmaxf(sv[n][i][0], sv[n][i][1]);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                            const float to = most - m[n][i] > 7.f ? ceilf(most) - 3.f : m[n][i];
                            l[n][i] *= fast_exp2(m[n][i] - finite_ref(to));
                            m[n][i] = to;
                        }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float pr[2][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float ref = finite_ref(m[n][i]);
                        pr[i][0] = fast_exp2(sv[n][i][0] - ref);
                        pr[i][1] = fast_exp2(sv[n][i][1] - ref);
                        l[n][i] += pr[i][0] + pr[i][1];      // the sums keep the fp32 weights
                    }
                    // P rounds to bf16 (2^-8 of a weight), the type of the values it meets, or to f16:
                    // 2^-11 of it or 2^-25, where some weight is above 4
                    if constexpr (NARROW) {
                        frag[n].x = pack_f16x2(t & 2 ? (t & 1 ? pr[1][1] : pr[0][1]) : (t & 1 ? pr[1][0] : pr[0][0]), 0.f);
                    } else {
                        frag[n].x = transpose8x8(pack_p<BITS>(pr[0][0], pr[1][0]));
                        frag[n].y = transpose8x8(pack_p<BITS>(pr[0][1], pr[1][1]));
                    }
                }
                if (it >= P_BUFFERS && !wait(&p_empty[buffer], it / P_BUFFERS - 1)) {
                    ok = false;
                    break;
                }
                float* out_ref = s_ref + (buffer * BLOCKS + block) * 8 * NT;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (NARROW)         // a row's 16: positions 2 i, 2 i + 1, 2 i + 8, 2 i + 9 together
                        s_p2[(buffer * BLOCKS + block) * 32 + 16 * (t & 1) + (g >> 1) * 4 + (t & 2) + (g & 1)] =
                            static_cast<uint16_t>(frag[n].x);
                    else
                        s_p[((buffer * BLOCKS + block) * NT + n) * 32 + lane] = frag[n];
                    if (g == 0 && (!NARROW || t == 0))
                        *reinterpret_cast<float2*>(out_ref + row_of(n, 0)) = make_float2(m[n][0], m[n][1]);
                }
                done_with(&p_full[buffer]);
            }
            // The next segment's notes are there once its first tile is: the warps that will
            // read that tile wait for it, and the group meets below.
            if (ok && end < total && end % TURNS == turn && !wait(&k_full[end % K_BARS], end / K_BARS)) ok = false;
            // ---- (m, l) of the segment: the four warps' sums brought to one reference
            float2* sums = s_sums + (segment & 1) * WARPS * 8 * NT;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], off);
                    if (g == 0 && (!NARROW || t == 0)) sums[warp * 8 * NT + row_of(n, i)] = make_float2(m[n][i], l[n][i]);
                }
            k_warps();
            if (ok && warp == 0 && lane < R) {
                float ref = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) ref = fmaxf(ref, sums[w * 8 * NT + lane].x);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float2 x = sums[w * 8 * NT + lane];
                    sum += x.y * fast_exp2(x.x - finite_ref(ref));
                }
                if (sum != sum && ref == -INFINITY) ref = 0.f;   // only scores of NaN: not an empty segment
                float2* ml = reinterpret_cast<float2*>(p.ws_ml) + row_index(seg.b, lane) * S;
                const int mine = seg.index & ~Segment::LAST;
                ml[mine] = make_float2(ref, ref == -INFINITY ? 0.f : sum);
                if (seg.index & Segment::LAST)    // the places behind it are empty
                    for (int i = mine + 1; i < S; ++i) ml[i] = make_float2(-INFINITY, 0.f);
            }
        }
    } else if (role == 1) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(V_REGS));
        __syncthreads();                          // barriers, the first tiles' notes
        const int total = *s_total;

        int it = 0;
        for (int segment = 0; it < total && ok; ++segment) {
            // (P of a segment's first tile comes after its notes)
            if (!wait(&p_full[it % P_BUFFERS], it / P_BUFFERS)) {
                ok = false;
                break;
            }
            const Segment seg = s_seg[segment % META];
            // O's references are the largest of the K warps'; lane 8 w + r keeps K warp w's of row
            // 8 n + r (NARROW: r), O's, and the factor from the one to the other.  A warp's weights
            // reach 2^7 whatever its reference, so the factor counts down to where they end: times
            // JOIN, as O is then, f16 holds it to 2^-32, and the largest product is 2^15.  (From
            // 2^-33 on it is 0: such weights are below 2^-28 of the row's largest, which is above
            // 2^2.  Without JOIN that came at 2^-20.)
            constexpr float JOIN = BITS == 16 ? 1.f : 256.f;
            float ref[NT], top[NT], factor[NT];
            float o[NT][MTILES][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                ref[n] = top[n] = -INFINITY;
                factor[n] = 0.f;
#pragma unroll
                for (int i = 0; i < MTILES; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
            }
            const int w_lo = seg.len - p.q_len + 1 - p.window, lo = p.window > 0 && w_lo > 0 ? w_lo : 0, hi = seg.len;
            for (const int end = it + seg.run; it < end; ++it) {
                const int slot = it % SLOTS, buffer = it % P_BUFFERS;
                if (!wait(&p_full[buffer], it / P_BUFFERS)) {
                    ok = false;
                    break;
                }
                // ---- one reference for the tile; most change nothing
                uint32_t pb[BLOCKS][NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // K warp lane / 8 wrote this tile's block of its, in its turn
                    const bool wrote = lane / 8 / BLOCKS == it % TURNS && (!NARROW || (lane & 7) < 2);
                    const float now = wrote ? s_ref[(buffer * BLOCKS + lane / 8 % BLOCKS) * 8 * NT + 8 * n + (lane & 7)] : ref[n];
                    if (__any_sync(0xffffffffu, now != ref[n])) {
                        ref[n] = now;
                        float to = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 8));
                        to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 16));
                        const float al = fast_exp2(top[n] - finite_ref(to));
                        top[n] = to;
                        factor[n] = fast_exp2(now - finite_ref(to)) * JOIN;
                        const float al0 = __shfl_sync(0xffffffffu, al, NARROW ? 0 : 2 * t);
                        const float al1 = __shfl_sync(0xffffffffu, al, NARROW ? 1 : 2 * t + 1);
#pragma unroll
                        for (int i = 0; i < MTILES; ++i) {
                            o[n][i][0] *= al0;
                            o[n][i][1] *= al1;
                            o[n][i][2] *= al0;
                            o[n][i][3] *= al1;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < BLOCKS; ++w) {
                        const float f = __shfl_sync(0xffffffffu, factor[n], (it % TURNS * BLOCKS + w) * 8 + (NARROW ? g & 1 : g));
                        const uint32_t f2 = pack_p<BITS>(f, f);
                        const uint2 x = NARROW ? *reinterpret_cast<const uint2*>(s_p2 + (buffer * BLOCKS + w) * 32 + 16 * (g & 1) + 4 * t)
                                               : s_p[((buffer * BLOCKS + w) * NT + n) * 32 + lane];
                        pb[w][n][0] = mul_p<BITS>(x.x, f2);
                        pb[w][n][1] = mul_p<BITS>(x.y, f2);
                    }
                }
                done_with(&p_empty[buffer]);
                if (!wait(&v_full[slot], it / SLOTS)) {
                    ok = false;
                    break;
                }
                // ---- This warp's columns of the positions that no row sees become 0, whatever they
                // hold (in 4 bits their scales: codes are finite); a position a lane
                uint8_t* rows = smem + Smem::v + slot * F::SLOT;
                const int* bases = s_base + (it % META) * BLOCKS;
                bool edge = false;
#pragma unroll
                for (int w = 0; w < BLOCKS; ++w) edge |= bases[w] < lo || bases[w] + 16 > hi;
                if (edge) {
                    for (int i = lane; i < TILE; i += 32) {
                        const int base = bases[i / 16], kp = base + (i & 15);
                        if (base >= 0 && kp >= lo && kp < hi) continue;
                        if constexpr (BITS == 4) {
                            *reinterpret_cast<uint2*>(rows + i * F::ROW + CODES + 8 * warp) = make_uint2(0u, 0u);
                        } else {
                            constexpr int BOXES = F::BOXES / WARPS;
                            for (int j = 0; j < BOXES * 8; ++j)
                                *reinterpret_cast<uint4*>(rows + ((warp * BOXES + j / 8) * TILE + i) * 128 + 16 * (j & 7)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();     // before the slot is loaded again
                    __syncwarp();
                }
                // ---- O^T += V^T P^T for this warp's columns
#pragma unroll
                for (int w = 0; w < BLOCKS; ++w) {
                    if constexpr (BITS == 4) add_values_4<NT>(rows + 16 * w * F::ROW, warp, lane, pb[w], o);
                    else if constexpr (BITS == 8) add_values_8<NT>(rows, 16 * w, warp, lane, pb[w], o);
                    else add_values_16<NT>(rows, warp, lane, pb[w], o);
                }
                done_with(&v_empty[slot]);
            }
            // ---- the segment's partial, unnormalised and times v_scale
            const int mine = seg.index & ~Segment::LAST;
            const float f = p.o_scale;            // (JOIN comes off before it: it may be next to the smallest float)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < MTILES; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][i][e] *= 1.f / JOIN;
            if constexpr (NARROW) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (r >= R) continue;
                    float* dst = p.ws_o + (row_index(seg.b, r) * S + mine) * D + 128 * warp + 16 * g;
#pragma unroll
                    for (int j = 0; j < MTILES / 2; ++j)
                        if (t == j)
                            *reinterpret_cast<float4*>(dst + 4 * j) =
                                make_float4(o[0][2 * j][r] * f, o[0][2 * j][2 + r] * f, o[0][2 * j + 1][r] * f,
                                            o[0][2 * j + 1][2 + r] * f);
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 8 * n + 2 * t + i;
                        if (r >= R) continue;
                        float* dst = p.ws_o + (row_index(seg.b, r) * S + mine) * D + 128 * warp;
#pragma unroll
                        for (int j = 0; j < MTILES / 2; ++j)
                            *reinterpret_cast<float4*>(dst + (BITS == 16 ? 64 * (j / 2) + 8 * g + 4 * (j & 1) : 16 * g + 4 * j)) =
                                make_float4(o[n][2 * j][i] * f, o[n][2 * j][2 + i] * f, o[n][2 * j + 1][i] * f,
                                                 o[n][2 * j + 1][2 + i] * f);
                    }
            }
        }
    } else {
        // ---- loads: warp 0 of K, warp 1 of V
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LOAD_REGS));
        if (warp == 0) {
            if (lane == 0) {
                for (int i = 0; i < K_BARS; ++i) mbar_init(&k_full[i], 1);
                for (int i = 0; i < SLOTS; ++i) {
                    mbar_init(&k_empty[i], BLOCKS);
                    mbar_init(&v_full[i], 1);
                    mbar_init(&v_empty[i], WARPS);
                }
                for (int i = 0; i < P_BUFFERS; ++i) {
                    mbar_init(&p_full[i], BLOCKS);
                    mbar_init(&p_empty[i], WARPS);
                }
                fence_mbar_init();
            }
            __syncwarp();
        }
        int range = 0;
        Walk<BITS, LIST> walk = {};
        if (warp < 2) walk = first_of_range<BITS, LIST>(p, index, gridDim.x / p.n_kv_heads, &range);
        if (warp == 0 && lane == 0) *s_total = walk.left;
        uint64_t *full = warp == 0 ? k_full : v_full, *empty = warp == 0 ? k_empty : v_empty;
        const int n_full = warp == 0 ? K_BARS : SLOTS;
        const CUtensorMap* map = warp == 0 ? &tmk : &tmv;
        uint8_t* ring = smem + (warp == 0 ? Smem::k : Smem::v);
        // A run is box_rows positions of one page; lane l keeps the first row and position
        // of run run0 + l of the sequence.
        const int box = p.box_rows, runs_per_tile = TILE / box, blocks_per_run = box / 16;
        int run0 = 0, run_row = -1, run_base = -1;
        auto look_up = [&]() {
            run_row = run_base = -1;
            const Item& x = walk.item;
            const int v = (x.lo / TILE) * TILE + (run0 + lane) * box;
            int lp = v >> p.page_shift, at = v;
            if constexpr (LIST) {
                const int off = v & (ps - 1);
                if (lp >= min(p.n_listed, x.held)) return;
                lp = list_page(p, list_of(p, walk.b, kvh), lp, x.held);
                if (lp < 0) return;
                at = lp * ps + off;
            }
            if (at >= x.len || at + box <= x.lo) return;
            const int page = p.page_table[static_cast<size_t>(walk.b) * p.max_pages_per_seq + lp];
            if (page < 0 || page >= p.num_pages) {
                report_error(p.err, FA512_DEVICE_ERR_INDEX);
                return;
            }
            run_row = page * ps + (at - lp * ps);
            run_base = at;
        };
        // tile i of the range, the sequence's `tile`-th, into its slot; K: what the masks need is noted
        auto load = [&](int i, int tile) {
            const int slot = i % SLOTS, bar = i % n_full, r = tile * runs_per_tile;
            if (r >= run0 + 32) {
                run0 += 32;
                look_up();
            }
            // lane l: box l % BOXES of the tile's run l / BOXES
            constexpr int BOXES = F::BOXES;
            const int run = lane / BOXES, row = __shfl_sync(0xffffffffu, run_row, (r - run0 + run) & 31);
            const bool mine = run < runs_per_tile && row >= 0;
            const unsigned some = __ballot_sync(0xffffffffu, mine);
            if (warp == 0) {
                // lanes below BLOCKS: the run of their 16 positions
                const int base = __shfl_sync(0xffffffffu, run_base, (r - run0 + lane / blocks_per_run) & 31);
                if (lane < BLOCKS) s_base[(i % META) * BLOCKS + lane] = base < 0 ? -1 : base + 16 * (lane % blocks_per_run);
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[bar], __popc(some) * box * (F::ROW / BOXES));
            __syncwarp();
            if (mine) {
                uint8_t* to = ring + slot * F::SLOT;
                if constexpr (BITS == 4) tma_load_3d(to + run * box * F::ROW, map, &full[bar], 0, kvh, row);
                else tma_load_3d(to + ((lane % BOXES) * TILE + run * box) * 128, map, &full[bar], (lane % BOXES) * (1024 / BITS), kvh, row);
            }
            loaded = i + 1;
        };
        // the first SLOTS tiles find their slots empty, and V's barriers wait for the one below
        bool started = false;
        auto start = [&]() {
            if (!started) __syncthreads();        // barriers, the first tiles' notes
            started = true;
        };
        if (warp == 3 && lane == 0) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
        if (warp >= 1) start();
        if (warp == 2) {
            // lengths out of range; sequences without a tile leave partials that say so
            for (int b = blockIdx.x * 32 + lane; b < p.batch; b += gridDim.x * 32)
                if (p.kv_lens[b] < 0 || p.kv_lens[b] > p.len_cap) report_error(p.err, FA512_DEVICE_ERR_INDEX);
            for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
                if (item_of<BITS, LIST>(p, b).tiles == 0)
                    for (int i = lane; i < p.q_len * p.n_q_heads * S; i += 32)
                        reinterpret_cast<float2*>(p.ws_ml)[static_cast<size_t>(b) * p.q_len * p.n_q_heads * S + i] =
                            make_float2(-INFINITY, 0.f);
            // entries of a list that is longer than its sequence's pages: none of them can name one (a page
            // there would be one too many, or not rise)
            if constexpr (LIST)
                for (int b = index; b < p.batch; b += static_cast<int>(gridDim.x) / p.n_kv_heads)
                    for (int e = item_of<BITS, LIST>(p, b).held + lane; e < p.n_listed; e += 32)
                        if (list_of(p, b, kvh)[e] >= 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        }
        int it = 0;
        for (int segment = 0; walk.left > 0 && ok; ++segment) {
            const int run = walk.run(), end = it + run, from = walk.tile - it;
            if (warp == 0 && lane == 0)
                s_seg[segment % META] = {walk.b, walk.item.len, run,
                                               (S == 1 ? 0 : index - walk.start / range) +
                                                   (walk.tile + run == walk.item.tiles ? Segment::LAST : 0)};
            run0 = walk.tile * runs_per_tile;
            look_up();
            for (; it < end; ++it) {
                if (it >= SLOTS) {
                    start();
                    if (!wait(&empty[it % SLOTS], it / SLOTS - 1)) {
                        ok = false;
                        break;
                    }
                }
                load(it, from + it);
                if (it == 0) start();             // (the others wait for the first segment's notes)
            }
            walk.next(p, run);
        }
        start();
    }
    // A wait that ran out: bounded waits for the copies in flight, so that none
    // lands after this CTA has gone.
    if (__syncthreads_or(!ok) && role == 2 && warp < 2) {
        uint64_t* full = warp == 0 ? k_full : v_full;
        const int n_full = warp == 0 ? K_BARS : SLOTS;
        for (int i = max(0, loaded - SLOTS); i < loaded; ++i) mbar_wait(&full[i % n_full], (i / n_full) & 1, p.err);
    }
}

// The rows' segments together: M = max m, O = sum 2^(m - M) O / sum 2^(m - M) l.  A block
// takes one row, a warp 128 columns of it; every warp finds the weights for itself, so
// nothing waits but for memory, and only segments with keys are read.  For many rows;
// few rows of many segments go faster where several groups of threads share a row's
// segments, in the merge of the other decode calls.  (300 sequences of up to 300
// positions, 8 heads: 47 us, with that merge 58; 64 x 8,192, 32 heads 198 and 207; but
// 16 x 16,384, 16 heads, up to 39 segments a row 51.4 and 50.1, 1 x 4,096, 8 heads 11.4
// and 9.1.)
constexpr int MERGE_AHEAD = 4;                       // segments whose O is read at a time, the first ones before the weights
__global__ void __launch_bounds__(128) merge_segments_kernel(const DecodeParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int S = p.num_splits, lane = threadIdx.x & 31;
    const size_t row = blockIdx.x;
    const float* ob = p.ws_o + row * S * D + threadIdx.x * 4;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row * S;
    auto o_of = [&](int i) { return *reinterpret_cast<const float4*>(ob + static_cast<size_t>(i) * D); };
    auto ml_of = [&](int i) { return i < S ? ml[i] : make_float2(-INFINITY, 0.f); };
    float4 x[MERGE_AHEAD];
#pragma unroll
    for (int i = 0; i < MERGE_AHEAD; ++i) x[i] = o_of(min(i, S - 1));
    const float2 first = ml_of(lane);
    float M = first.x;
    for (int i = lane + 32; i < S; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < S; s0 += 32) {
        const float2 v = s0 == 0 ? first : ml_of(s0 + lane);
        const float w = M == -INFINITY ? 0.f : fast_exp2(v.x - M);   // 0: nothing, whatever O holds
        L += w * v.y;
        const unsigned live = __ballot_sync(0xffffffffu, w != 0.f);
        for (int i0 = 0; live >> i0 != 0; i0 += MERGE_AHEAD) {
            if (s0 + i0 > 0)
#pragma unroll
                for (int i = 0; i < MERGE_AHEAD; ++i)
                    if (live >> (i0 + i) & 1) x[i] = o_of(s0 + i0 + i);
#pragma unroll
            for (int i = 0; i < MERGE_AHEAD; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i0 + i);
                if (wi != 0.f) {
                    acc.x = fmaf(wi, x[i].x, acc.x);
                    acc.y = fmaf(wi, x[i].y, acc.y);
                    acc.z = fmaf(wi, x[i].z, acc.z);
                    acc.w = fmaf(wi, x[i].w, acc.w);
                }
            }
            if (i0 + MERGE_AHEAD == 32) break;
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    reinterpret_cast<uint2*>(p.out + row * D)[threadIdx.x] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse && threadIdx.x == 0) p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

cudaError_t launch_merge(const DecodeParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.batch) * p.q_len * p.n_q_heads;
    if (rows < 512) return launch_decode_merge(p, stream);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_segments_kernel, p);
}

template <int BITS, int ROWS, bool LIST>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p, cudaStream_t stream) {
    constexpr int SMEM = Smem<BITS, (ROWS > 8 ? 2 : 1)>::total;
    auto kernel = decode_ranges_kernel<BITS, ROWS, LIST>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<p.groups * p.n_kv_heads, THREADS, SMEM, stream>>>(tmk, tmv, p);
    return cudaGetLastError();
}

template <int BITS, bool LIST>
cudaError_t launch_rows(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p, cudaStream_t stream) {
    const int rows = p.q_len * p.group;
    if constexpr (BITS == 4)
        if (rows <= 2) return launch<BITS, 2, LIST>(tmk, tmv, p, stream);
    return rows <= 8 ? launch<BITS, 8, LIST>(tmk, tmv, p, stream) : launch<BITS, 16, LIST>(tmk, tmv, p, stream);
}

}  // namespace ranges

int decode_ranges_tile(int bits) {
    return bits == 16 ? ranges::Format<16>::TILE : bits == 8 ? ranges::Format<8>::TILE : ranges::Format<4>::TILE;
}
int decode_ranges_ctas_per_sm() { return ranges::CTAS_PER_SM; }

cudaError_t launch_decode_ranges(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p, int bits,
                                 cudaStream_t stream) {
    cudaError_t e;
    if (bits == 4)
        e = p.listed ? ranges::launch_rows<4, true>(tmk, tmv, p, stream) : ranges::launch_rows<4, false>(tmk, tmv, p, stream);
    else
        e = bits == 8 ? ranges::launch_rows<8, true>(tmk, tmv, p, stream) : ranges::launch_rows<16, true>(tmk, tmv, p, stream);
    return e != cudaSuccess ? e : ranges::launch_merge(p, stream);
}

}  // namespace fa512
