// What the tree decode kernels share: the keys that the rows of a (sequence,
// row group, KV head) item walk, the equal ranges of those keys' tiles that
// the resident clusters take, operand layouts and small device helpers.
//
// With start = len - cnt the last cnt cached positions are the tokens' own.
// Token t sees a key j < start always and a key start + c if its mask has bit
// c (no mask: c <= t); with a window, only keys whose place is above the
// token's place - window or below n_sinks, where the place of a cached key is
// its position and that of token t is start + (tokens it sees) - 1.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_pair.cuh"

namespace fa512 {
namespace tree {

using pair::elect_one;

// The kernel's code is kept small enough for the instruction cache (roles run
// side by side, and what a segment runs once would otherwise be fetched from
// L2 between the streams' loads): what is seldom run or run from many places
// is not inlined.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    return pair::wait_or_abort(bar, parity, err, abort);
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    return mbar_try_wait(smem_u32(bar), parity) || wait_slow(bar, parity, err, abort);
}

constexpr int D = 512;
constexpr int MAX_NODES = 256;
constexpr int SIDE = 16384;              // 128 keys x 128 bytes of the head dim
constexpr int SLOT = 2 * SIDE;           // a ring slot

// Instruction descriptor of M x N products with an fp32 accumulator, without
// the operand types.
__host__ __device__ constexpr uint32_t idesc_shape(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
constexpr uint32_t BF16_AB = (1u << 7) | (1u << 10);
constexpr uint32_t B_E5M2 = 1u << 10;                    // beside an E4M3 A
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;

// The descriptor of an MN-major operand whose lines are `line` = 128, 64 or
// 32 bytes, swizzled over their own length (atoms of 8 lines).
template <int LINE>
__device__ __forceinline__ uint64_t make_sdesc_lines(uint32_t saddr) {
    constexpr uint64_t mode = LINE == 128 ? 2 : LINE == 64 ? 4 : 6;
    return (make_sdesc_sw128(saddr, 16, 8 * LINE) & ~(7ull << 61)) | (mode << 61);
}
// Place of 16-byte piece c of line k under that swizzle.
template <int LINE>
__device__ __forceinline__ int line_piece(int k, int c) {
    if constexpr (LINE == 128) return (c ^ (k & 7)) << 4;
    if constexpr (LINE == 64) return (c ^ ((k >> 1) & 3)) << 4;
    return (c ^ ((k >> 2) & 1)) << 4;
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

// E4M3 (E5M2) pair of two fp32 values (low byte first) and the pair's values.
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

// 16 weights of one key as the sum of three E5M2 terms.
__device__ __forceinline__ void split_weights(const float (&x)[16], float scale, uint4 (&term)[3]) {
    uint32_t w[3][4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float a = x[2 * j] * scale, d = x[2 * j + 1] * scale;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            float va, vd;
            w[e][j >> 1] |= e5m2_pair(a, d, va, vd) << (16 * (j & 1));
            a -= va;
            d -= vd;
        }
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) term[e] = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
}

// Reduces 16 values per lane over the warp at once: lane i gets everyone's
// v[i % 16] (15 shuffles in which halves swap the values that the other half
// keeps, and one that joins the warp's halves).
template <class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[16], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// A query row over an E4M3 cache, 16 elements a lane (x): scaled by a power of
// two so that its largest element comes to [128, 256), and written as the sum
// of two E4M3 terms.  An infinity has no such form (it would saturate to a
// finite code): it makes the scale NaN, and with it the terms and the scores.
__device__ __forceinline__ float query_scale(const uint4 (&x)[2]) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // 2^(7 - exponent of amax)
    const int E = (__float_as_uint(amax) >> 23) & 0xff;
    const int biased = E == 255 ? 255 : min(7 + 2 * 127 - E, 254);
    const uint32_t bits = static_cast<uint32_t>(biased) << 23 | (E == 255 ? 1u << 22 : 0u);
    return amax > 0.f ? __uint_as_float(bits) : 1.f;
}
__device__ __forceinline__ void split_query(const uint4 (&x)[2], float scale, uint4& first, uint4& second) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        hi[j] = lo[j] = 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float a = __uint_as_float(w[2 * j + k] << 16) * scale;
            const float c = __uint_as_float(w[2 * j + k] & 0xffff0000u) * scale;
            float va, vc, ra, rc;
            hi[j] |= e4m3_pair(a, c, va, vc) << (16 * k);
            lo[j] |= e4m3_pair(a - va, c - vc, ra, rc) << (16 * k);
        }
    }
    first = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    second = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// The keys that a row group of a sequence walks.
template <int TILE>
struct BandOf {
    int len, cnt, start;        // cached positions, tokens, first token's position
    int lo, hi;                 // keys that some row may see: [lo, hi) and those below sink_end
    int sink_end;
    int span, shift;            // the walk's place v is key v below span (the sinks), else key v + shift
    int place_max;              // no row's place is above
    int tiles;
    __device__ __forceinline__ int key(int v) const { return v < span ? v : v + shift; }
    // Whether every row sees every key of the tile at place v0: cached keys
    // inside every row's window, or sinks.
    __device__ __forceinline__ bool whole(const TreeParams& p, int v0) const {
        const int sinks = min(span, v0 + TILE);
        if (v0 < span && sinks > min(sink_end, start)) return false;
        const int first = max(v0, span) + shift, last = v0 + TILE - 1 + shift;
        return v0 + TILE <= span ||
               (last < min(start, hi) && (p.window <= 0 || first > place_max - p.window || last < sink_end));
    }
    // Whether some key of the tile may be seen by no row.  Without a mask every
    // key of [lo, hi) and every sink is seen by some row; with one, a drafted
    // key may be named by nobody, and the window's lower edge is known only to
    // lie in [lo, place_max - window].
    __device__ __forceinline__ bool dirty(const TreeParams& p, int v0) const {
        if (p.tree_mask) return !whole(p, v0);
        if (v0 < span && min(span, v0 + TILE) > sink_end) return true;
        const int first = max(v0, span) + shift, last = v0 + TILE - 1 + shift;
        return v0 + TILE > span && (last >= hi || (first < lo && last >= sink_end));
    }
};

// Which of GW rows (the first is row r0 of its item) see a key of the walk: bit
// i, row r0 + i.  low: the rows' last key below the window; of_mask(c): the bits
// of the rows whose masks name token c.
template <int GW, int TILE, class OfMask>
__device__ __forceinline__ uint32_t rows_that_see(const TreeParams& p, const BandOf<TILE>& d, int key, int r0, const int* depth,
                                                  const int* low, OfMask of_mask) {
    constexpr uint32_t ALL = 0xffffffffu >> (32 - GW);
    const int c = key - d.start;
    if (key >= d.hi) return 0u;
    if (!p.tree_mask) {
        // token t sees the key iff c <= t and (t < c + window or the key is a sink):
        // the rows [t0 G, t1 G) of the item, here [t0 G - r0, t1 G - r0)
        const int t0 = max(c, 0);
        const bool ends = p.window > 0 && key >= d.sink_end && c < d.cnt - p.window;
        const int t1 = ends ? max(0, c + p.window) : d.cnt;
        const int a = max(0, t0 * p.group - r0), z = min(GW, t1 * p.group - r0);
        return a >= z ? 0u : (0xffffffffu >> (32 - z)) & (0xffffffffu << a);
    }
    // the key's place; a drafted key's rows by their masks
    const int kp = c >= 0 ? d.start + depth[c] : key;
    uint32_t vis = c >= 0 ? of_mask(c) : 0xffffffffu;
    if (p.window > 0 && kp >= d.sink_end) {
        uint32_t in = 0u;
#pragma unroll 8
        for (int i = 0; i < GW; ++i) in |= kp > low[i] ? 1u << i : 0u;
        vis &= in;
    }
    return vis & ALL;
}

// Band of row group `grp` (group_rows rows) of sequence b.  It follows from
// the lengths alone: with a mask a token's place is only known to lie in
// [start - 1, start + cnt - 1], and its own tokens' keys are always walked.
template <int TILE>
__device__ __noinline__ BandOf<TILE> band_of(const TreeParams& p, int b, int grp, int group_rows, bool record) {
    BandOf<TILE> d;
    d.len = p.kv_lens[b];
    d.cnt = p.q_lens ? p.q_lens[b] : p.q_len;
    if (d.len < 0 || d.len > p.len_cap || d.cnt < 0 || d.cnt > p.q_len) {
        if (record) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        d.len = max(0, min(d.len, p.len_cap));
        d.cnt = max(0, min(d.cnt, p.q_len));
    }
    d.start = d.len - d.cnt;
    const int r0 = grp * group_rows;
    const int first = max(r0 / p.group, -d.start);
    const int last = min((r0 + group_rows - 1) / p.group, d.cnt - 1);
    d.hi = first > last ? 0 : p.tree_mask ? d.len : min(d.len, d.start + last + 1);
    d.lo = 0;
    d.sink_end = 0;
    d.place_max = d.start + (p.tree_mask ? d.cnt - 1 : last);
    if (p.window > 0 && d.hi > 0) {
        // (start may be below 0: less the window it could leave int32)
        const int from = p.tree_mask ? d.start : d.start + first + 1;
        d.lo = from > p.window ? from - p.window : 0;
        d.sink_end = min(p.n_sinks, d.hi);
    }
    // the walk is the sinks' boxes, then the boxes from lo on, so that neither
    // edge costs a tile of its own (57 trees of 64 tokens, window 36 and 4 sinks:
    // 220 -> 147 us)
    const int box = min(p.page_size, 128), lo_box = d.lo / box * box;
    d.span = (d.sink_end + box - 1) / box * box;
    d.shift = lo_box - d.span;
    if (d.shift <= 0) d.span = d.shift = 0;
    d.tiles = d.hi <= 0 ? 0 : (d.hi - d.shift + TILE - 1) / TILE;
    return d;
}

// Walk over this cluster's range of the items' tiles (an item without tiles
// counts as one, so that somebody writes its empty rows).
template <int TILE>
struct WalkOf {
    int pos, end, base;         // next unit, end of the range, first unit of the current item
    int per;
    int entry, kvh;             // current item: entry = sequence * groups + row group
    int entries, groups, group_rows;
    int stride;                 // entries from one of the walk's to its next: 1, or groups in a team
    BandOf<TILE> band;
    // the current segment
    int b, grp, first, n;       // tiles [first, first + n) of the band
    int index, count;           // which of how many segments of the item

    __device__ __forceinline__ int units() const { return max(1, band.tiles); }
    __device__ __forceinline__ void load(const TreeParams& p) {
        b = entry / groups;
        grp = entry - b * groups;
        band = band_of<TILE>(p, b, grp, group_rows, false);
    }
    __device__ __noinline__ bool next(const TreeParams& p) {
        while (pos < end) {
            const int w = units();
            if (pos >= base + w || (p.num_splits == 1 && pos > base)) {
                // a whole item belongs to the range that holds its first unit
                if (pos < base + w) pos = base + w;
                base += w;
                if (++kvh == p.n_kv_heads) {
                    kvh = 0;
                    if ((entry += stride) >= entries) return false;
                    load(p);
                }
                continue;
            }
            first = pos - base;
            if (p.num_splits == 1) {
                index = 0;
                count = 1;
                n = band.tiles;
                pos = base + w;
            } else {
                const int take = min(w - first, end - pos);
                const int seg0 = base / per;
                index = pos / per - seg0;
                count = (base + w - 1) / per - seg0 + 1;
                n = min(take, band.tiles);
                pos += take;
            }
            return true;
        }
        return false;
    }
};

// The range of cluster `me` of `clusters`: the total of all items' units, then
// the item that holds the range's first unit.  Every thread of the block calls
// it; s_scan: SCAN_INTS int of shared memory.
//
// Where there is a cluster for every item and equal segments of the longest
// item are hardly longer than a range, a cluster takes one segment of one item,
// for a change of item costs about as much as three tiles (8 sequences of 52
// tokens with 8 heads on one KV head, 2,061 positions: 56.9 us with ranges, 46.6
// with segments; 12 of 9 tokens, 4 KV heads, 1,937 positions in E4M3: 45.0, 36.7).
//
// Otherwise the ranges.  The row groups of a KV head read the same keys.  One walk over all items
// would come to them at different times, when L2 has lost them (8 sequences of
// 600 rows a KV head, window 4,096: 1.36 GB from memory for 0.27 GB of keys), so
// the clusters form teams of one cluster per row group: each walks its group's
// items alone, and a team's members reach the same keys together (294 -> 262
// us).  Where a padded batch leaves the groups unlike (the longest group's range more than a
// tenth above everybody's equal share) all walk all items.
constexpr int MAX_TEAM = 16;
constexpr int SCAN_INTS = 36 + 32 + MAX_TEAM;          // without teams: 36 + 32
template <int TILE, int THREADS>
__device__ __forceinline__ void start_walk(WalkOf<TILE>& walk, const TreeParams& p, int clusters, int me, int* s_scan) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    walk.entries = p.batch * walk.groups;
    int* s_at = s_scan + 32;                                // start's entry, unit
    constexpr int NW = THREADS / 32;
    auto entry_units = [&](int e, bool record) -> int {
        if (e >= walk.entries) return 0;
        const int eb = e / walk.groups;
        const BandOf<TILE> d = band_of<TILE>(p, eb, e - eb * walk.groups, walk.group_rows, record && e == eb * walk.groups);
        return max(1, d.tiles) * p.n_kv_heads;
    };
    int* s_most = s_scan + 36;                              // units of each warp's longest item
    int* s_team = s_scan + 68;                              // units of each row group
    const int teams = walk.groups > 1 && walk.groups <= MAX_TEAM ? clusters / walk.groups : 0;
    if (teams > 0) {
        if (tid < MAX_TEAM) s_team[tid] = 0;
        __syncthreads();
    }
    int total = 0, longest = 0, mine0 = 0;           // mine0: entry tid's units
    for (int e = tid; e < walk.entries; e += THREADS) {
        const int u = entry_units(e, blockIdx.x == 0);
        if (e == tid) mine0 = u;
        total += u;
        longest = max(longest, u / p.n_kv_heads);
        if (teams > 0) atomicAdd(&s_team[e % walk.groups], u);
    }
    total = __reduce_add_sync(0xffffffffu, total);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
        s_scan[warp] = total;
        s_most[warp] = longest;
    }
    __syncthreads();
    total = __reduce_add_sync(0xffffffffu, lane < NW ? s_scan[lane] : 0);
    walk.stride = 1;
    const long long items = static_cast<long long>(walk.entries) * p.n_kv_heads;
    if (items <= clusters) {
        longest = __reduce_max_sync(0xffffffffu, lane < NW ? s_most[lane] : 0);
        const int segments = min(clusters / static_cast<int>(items), p.num_splits);
        const int range = max((total + clusters - 1) / clusters, p.min_range);
        if (segments == 1 ? p.num_splits == 1 || longest <= range + 2 : (longest + segments - 1) / segments <= range + 2) {
            const int item = me / segments, segment = me - item * segments;
            walk.pos = walk.end = walk.base = 0;
            if (item < items) {
                walk.entry = item / p.n_kv_heads;
                walk.kvh = item - walk.entry * p.n_kv_heads;
                walk.load(p);
                walk.per = (walk.units() + segments - 1) / segments;
                walk.pos = min(segment * walk.per, walk.units());
                walk.end = min(walk.pos + walk.per, walk.units());
            }
            return;
        }
    }
    int start = 0;                                          // first entry of the walk's
    if (teams > 0) {
        const int most = __reduce_max_sync(0xffffffffu, lane < walk.groups ? s_team[lane] : 0);
        const long long share = (total + clusters - 1) / clusters;
        if (10LL * ((most + teams - 1) / teams) <= 11 * share) {
            start = me % walk.groups;
            walk.stride = walk.groups;
            total = me / walk.groups < teams ? s_team[start] : 0;
            clusters = teams;
            me = min(me / walk.groups, teams);
        }
    }
    // ranges short enough to balance, long enough that no item has more
    // than num_splits segments
    walk.per = (total + clusters - 1) / clusters;
    if (p.num_splits > 1) walk.per = max(walk.per, p.min_range);
    walk.per = max(walk.per, 1);
    const long long begin = static_cast<long long>(me) * walk.per;
    walk.pos = static_cast<int>(min(begin, static_cast<long long>(total)));
    walk.end = min(total - walk.pos, walk.per) + walk.pos;
    int before = 0;
    if (walk.pos < walk.end) {
        for (int e0 = start; e0 < walk.entries; e0 += THREADS * walk.stride) {
            const int e = e0 + tid * walk.stride;
            const int u = e == tid ? mine0 : entry_units(e, false);
            int x = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            const int ws = lane < NW ? s_scan[lane] : 0;
            x += before + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
            const int sum = before + __reduce_add_sync(0xffffffffu, ws);
            if (walk.pos >= x - u && walk.pos < x) {
                s_at[0] = e;
                s_at[1] = x - u;
            }
            before = sum;
            if (walk.pos < before) break;
        }
    }
    __syncthreads();
    walk.entry = s_at[0];
    walk.kvh = 0;
    walk.base = s_at[1];
    if (walk.pos < walk.end) {
        walk.load(p);
        walk.kvh = (walk.pos - walk.base) / walk.units();
        walk.base += walk.kvh * walk.units();
    }
}

// Place of row r (of its group; `row` of the call) of the walk's segment among
// the partials, for cluster `me`.
__device__ __forceinline__ size_t partial_at(const TreeParams& p, size_t row, int r, int index, int me) {
    if (p.slot_rows == 0) return row * p.num_splits + index;
    // an item's first segment is the last of its cluster, any other the first
    return static_cast<size_t>((2 * me + (index == 0)) * p.slot_rows + r);
}
// Where the merge finds a row's segments, as an item's first one left it.
__device__ __forceinline__ void leave_item(const TreeParams& p, int entry, int kvh, int count, int stride, int me) {
    reinterpret_cast<int2*>(p.ws_item)[static_cast<size_t>(entry) * p.n_kv_heads + kvh] = make_int2(count | stride << 16, me);
}
struct Segments {
    size_t base;                // place of segment s > 0: base + s * step; of segment 0: base + first
    int first, step, n;
    __device__ __forceinline__ size_t at(int s) const { return base + (s == 0 ? first : static_cast<size_t>(s) * step); }
};
template <bool SLOTS>
__device__ __forceinline__ Segments segments_of(const TreeParams& p, size_t row, int b, int t, int h, int group_rows) {
    const int r = t * p.group + h % p.group, grp = r / group_rows;
    const int32_t* item = p.ws_item + 2 * ((static_cast<size_t>(b) * p.row_groups + grp) * p.n_kv_heads + h / p.group);
    Segments s;
    // an attention that ran into a timeout may not have left its items
    if constexpr (SLOTS) {
        const int2 left = *reinterpret_cast<const int2*>(item);
        const int stride = left.x >> 16;
        s.n = min(p.num_splits, left.x & 0xffff);
        if (left.y < 0 || stride < 1 || left.y + static_cast<long long>(s.n - 1) * stride >= p.clusters) s.n = 0;
        s.base = static_cast<size_t>(2 * left.y) * p.slot_rows + (r - grp * group_rows);
        s.first = p.slot_rows;
        s.step = 2 * stride * p.slot_rows;
    } else {
        s.n = min(p.num_splits, *item & 0xffff);
        s.base = row * p.num_splits;
        s.first = 0;
        s.step = 1;
    }
    return s;
}

// Whether a row's softmax has weight, from the row's `low` (INT_MAX: it sees
// nothing), maximum and sum.  A NaN score is no maximum (fmaxf passes over it)
// but makes the sum NaN, and so it has to come out.
__device__ __forceinline__ bool some_key(int low, float top, float sum) {
    return low != INT_MAX && (top != -INFINITY || sum != 0.f);
}
// The maximum that goes with a partial: +inf beside a NaN sum, which makes the
// merged row NaN whatever its other segments hold.
__device__ __forceinline__ float partial_max(bool some, float top, float sum) {
    return !some ? -INFINITY : sum != sum ? INFINITY : top;
}

// Word w of token t's mask; bits at and behind cnt name no token.
__device__ __forceinline__ uint32_t mask_word(const TreeParams& p, int b, int cnt, int t, int w) {
    const int left = cnt - 32 * w;
    const uint32_t m =
        static_cast<uint32_t>(p.tree_mask[(static_cast<size_t>(b) * p.q_len + t) * p.mask_words + w]);
    return left >= 32 ? m : left <= 0 ? 0u : m & ((1u << left) - 1u);
}

// The depths of all cnt tokens, by `threads` threads.
__device__ __forceinline__ void load_depths(const TreeParams& p, int b, int cnt, int* s_depth, int thread,
                                            int threads) {
#pragma unroll 1
    for (int t = thread; t < cnt; t += threads) {
        int c = 0;
#pragma unroll 1
        for (int w = 0; w < p.mask_words; ++w) c += __popc(mask_word(p, b, cnt, t, w));
        s_depth[t] = c - 1;
    }
}

}  // namespace tree

// decode_tree_pair_sm103.cu: more than 64 rows per KV head.
cudaError_t launch_tree_pair(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                             cudaStream_t stream);
// decode_tree_sm103.cu: combines the segments' partials of rows in groups of group_rows.
cudaError_t launch_tree_merge(const TreeParams& p, int group_rows, cudaStream_t stream);

}  // namespace fa512
