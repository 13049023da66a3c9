// Drafted tokens (a tree of them, or a plain run) over a paged cache, head
// dim 512, sm_103a.
//
// With start = len - cnt the last cnt cached positions are the tokens' own.
// Token t sees a key j < start always and a key start + c if its mask has bit
// c (no mask: c <= t); with a window, only keys whose place is above the
// token's place - window or below n_sinks, where the place of a cached key is
// its position and that of token t is start + (tokens it sees) - 1.
//
// A CTA takes ROWS = 64 (or 32) rows ((token, query head) pairs) of one KV
// head and walks key tiles of 128, computing both products transposed on
// tcgen05: S^T = K Q^T (M = 128 keys, N = ROWS, K = 512) and
// O^T += V^T P^T (four M = 128 blocks of the head dim, N = ROWS, K = 128
// keys).  So the whole fp32 O of 64 rows takes 256 TMEM columns and leaves
// room for three S^T buffers, and K and V stream through shared memory once:
//   K rows are the K-major A operand, V rows the MN-major A operand (its M
//   dimension, the head dim, is the contiguous one), Q stays in shared memory
//   as the K-major B operand, and P^T is written by the softmax threads as
//   an MN-major B operand: a thread holds one key, so its rows' values are
//   contiguous.
// Per 128 keys a CTA streams 256 KiB (bf16): ~5.9 us at an SM's share of the
// measured HBM rate, against ~0.85 us of tensor work.  Row tiles of the same
// keys form a cluster that loads each slot once and multicasts it.
//
// The row maxima lie across lanes here, so they are not reduced every tile:
// each thread compares its scores with the reference its rows hold, and only
// when some score is above it by 2^THR (a vote at the tile's one barrier) do
// the four warps of a column group reduce the maxima and rescale O.  The row
// sums stay per-thread partials until the end.
//
// FP8 E4M3 cache: the bytes are MMA operands as stored (kind::f8f6f4).  Each
// query row is scaled by a power of two so that its largest element is in
// [128, 256) and written as the sum of two E4M3 terms (exact for elements
// above 2^-10 of the largest, off by at most 2^-18 of it below), and P as the
// sum of three E5M2 terms (relative error 2^-9, down to 2^-28 of the
// reference), so every product keeps at least the accuracy of the bf16 path
// without widening a byte of the cache.
//
// Work: the (sequence, row group, KV head) items' tiles, one after another,
// are cut into equal ranges, one per resident cluster, so every SM streams
// the same number of tiles whatever the lengths; an item that spans several
// ranges leaves (O, m, l) partials that merge_kernel combines, any other is
// written directly.
#include <cuda.h>
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
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    return pair::wait_or_abort(bar, parity, err, abort);
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    return mbar_try_wait(smem_u32(bar), parity) || wait_slow(bar, parity, err, abort);
}

constexpr int D = 512;
constexpr int MAX_NODES = 256;
constexpr int TILE = 128;                // keys per tile: M of S^T
constexpr int SIDE = 16384;              // 128 keys x 128 bytes of the head dim
constexpr int SLOT = 2 * SIDE;           // a ring slot: 256 bytes of the head dim of a key tile
constexpr int GW = 16;                   // rows (columns of S^T) of a softmax warp
constexpr int LOOK = 2;                  // S^T tiles computed ahead of O^T += V^T P^T
constexpr int NB = LOOK + 1;             // S^T buffers
constexpr int MAX_CLUSTER = 8;

template <bool FP8, int ROWS>
struct Cfg {
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int GROUPS = ROWS / GW;
    static constexpr int SOFTMAX_WARPS = 4 * GROUPS;     // (column group, TMEM lane quadrant)
    static constexpr int THREADS = 64 + SOFTMAX_WARPS * 32;
    static constexpr int CHUNKS = D * EB / 128;          // 128-byte column chunks of the head dim: 8 or 4
    static constexpr int SLOTS = CHUNKS / 2;             // ring slots of a K (V) tile: 4 or 2
    static constexpr int Q_CHUNK = ROWS * 128;           // one 128-byte column chunk of Q
    static constexpr int Q_TERM = CHUNKS * Q_CHUNK;
    static constexpr int Q_TERMS = FP8 ? 2 : 1;
    static constexpr int P_LINE = ROWS * EB;             // bytes of a key's row values: 128, 64 or 32
    static constexpr int P_TERM = TILE * P_LINE;
    static constexpr int P_TERMS = FP8 ? 3 : 1;
    static constexpr float THR = FP8 ? 4.f : 8.f;        // log2 of the growth that rescales
    static constexpr float P_SCALE = FP8 ? 2048.f : 1.f; // keeps E5M2 terms of small p normal
    static constexpr uint32_t TM_O = 0, TM_S = 4 * ROWS;
    static constexpr uint32_t TM_COLS = ROWS == 64 ? 512 : 256;
    static_assert(TM_S + NB * ROWS <= TM_COLS, "tensor memory");
    // shared memory, from a 1 KiB aligned base
    static constexpr int p = 0;
    static constexpr int q = p + ((P_TERMS * P_TERM + 1023) & ~1023);
    static constexpr int mask = q + Q_TERMS * Q_TERM;    // [ROWS tokens][words]
    static constexpr int depth = mask + ROWS * (MAX_NODES / 32) * 4;
    static constexpr int red = depth + MAX_NODES * 4;    // [4][ROWS] float
    static constexpr int mult = red + 4 * ROWS * 4;      // [ROWS] float: score -> log2 units
    static constexpr int see = mult + ROWS * 4;          // [ROWS] int4: last key, key below the window, mask row
    static constexpr int rows = see + ROWS * 16;         // [4 tiles][8 boxes] int: the producer's pool rows
    static constexpr int seen = rows + 4 * 8 * 4;         // [GROUPS][TILE] bytes: some row of the group sees the key
    static constexpr int scan = seen + GROUPS * TILE;    // 32 int, then the walk's start
    static constexpr int info = scan + 32 * 4 + 16;      // [ROWS] 16 bytes: what the epilogue writes
    static constexpr int bars = info + ROWS * 16;
    static constexpr int MAX_NS = 6;
    static constexpr int FULL = 0, EMPTY = MAX_NS, S_FULL = 2 * MAX_NS, S_FREE = S_FULL + NB, P_FULL = S_FREE + NB,
                         PV_DONE = P_FULL + 1, Q_FULL = PV_DONE + 1, O_FREE = Q_FULL + 1, DRAIN = O_FREE + 1,
                         N_BARS = DRAIN + 1;
    static constexpr int misc = bars + N_BARS * 8;       // tmem address, abort flag
    static constexpr int ring = (misc + 16 + 1023) & ~1023;
    static constexpr int NS_FIT = (232448 - 1024 - ring) / SLOT;
    static constexpr int NS = NS_FIT < MAX_NS ? NS_FIT : MAX_NS;
    static constexpr int total = ring + NS * SLOT;
    static_assert(NS >= 4, "ring slots");
};

// D[tmem] (+)= A[smem] * B[smem]^T, 8-bit floating-point operands.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptors: M = 128, N = rows, fp32 accumulator.
__host__ __device__ constexpr uint32_t shape(int rows) { return (1u << 4) | (static_cast<uint32_t>(rows >> 3) << 17) | (128u >> 4 << 24); }
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

// Arrives on the barrier at this offset in CTA `rank` of the cluster when
// every MMA issued so far has completed.
__device__ __forceinline__ void tc_commit_to(uint64_t* bar, uint32_t rank) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(1u << rank))
        : "memory");
}
// A tile load into the same shared-memory place of every CTA in `ctas`,
// counted on each one's barrier at this offset.
__device__ __forceinline__ void tma_load_3d_multicast(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                                      int c1, int c2, uint16_t ctas) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "h"(ctas)
        : "memory");
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

// Reduces 16 values per lane over the warp at once: lane i gets everyone's
// v[i % 16] (15 shuffles in which halves swap the values that the other half
// keeps, and one that joins the warp's halves).
template <class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[GW], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = GW / 2; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
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

// The keys that a row group of a sequence walks.
struct Band {
    int len, cnt, start;        // cached positions, tokens, first token's position
    int lo, hi;                 // keys that some row may see: [lo, hi) and those below sink_end
    int sink_end;
    int sink_tiles, lo_tile;    // tile i is i < sink_tiles ? i : lo_tile + i - sink_tiles
    int place_max;              // no row's place is above
    int tiles;
    __device__ __forceinline__ int key0(int i) const {
        return (i < sink_tiles ? i : lo_tile + i - sink_tiles) * TILE;
    }
};

// Band of row group `grp` (group_rows rows) of sequence b.  It follows from
// the lengths alone: with a mask a token's place is only known to lie in
// [start - 1, start + cnt - 1], and its own tokens' keys are always walked.
__device__ __noinline__ Band band_of(const TreeParams& p, int b, int grp, int group_rows, bool record) {
    Band d;
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
        d.lo = max(0, p.tree_mask ? d.start - p.window : d.start + first - p.window + 1);
        d.sink_end = min(p.n_sinks, d.hi);
    }
    d.lo_tile = d.lo / TILE;
    d.sink_tiles = min((d.sink_end + TILE - 1) / TILE, d.lo_tile);
    d.tiles = d.hi <= 0 ? 0 : d.sink_tiles + (d.hi + TILE - 1) / TILE - d.lo_tile;
    return d;
}

// Walk over this cluster's range of the items' tiles (an item without tiles
// counts as one, so that somebody writes its empty rows).
struct Walk {
    int pos, end, base;         // next unit, end of the range, first unit of the current item
    int per;
    int entry, kvh;             // current item: entry = sequence * groups + row group
    int entries, groups, group_rows;
    Band band;
    // the current segment
    int b, grp, first, n;       // tiles [first, first + n) of the band
    int index, count;           // which of how many segments of the item

    __device__ __forceinline__ int units() const { return max(1, band.tiles); }
    __device__ __forceinline__ void load(const TreeParams& p) {
        b = entry / groups;
        grp = entry - b * groups;
        band = band_of(p, b, grp, group_rows, false);
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
                    if (++entry == entries) return false;
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

template <bool FP8, int ROWS>
__global__ void __launch_bounds__(Cfg<FP8, ROWS>::THREADS, 1)
tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
            const __grid_constant__ TreeParams p) {
    using C = Cfg<FP8, ROWS>;
    constexpr int NS = C::NS, THREADS = C::THREADS;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = p.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[C::FULL + i], 1);
            mbar_init(&bars[C::EMPTY + i], cs);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&bars[C::S_FULL + i], 1);
            mbar_init(&bars[C::S_FREE + i], C::SOFTMAX_WARPS);
        }
        mbar_init(&bars[C::P_FULL], C::SOFTMAX_WARPS);
        mbar_init(&bars[C::PV_DONE], 1);
        mbar_init(&bars[C::Q_FULL], C::SOFTMAX_WARPS);
        mbar_init(&bars[C::O_FREE], C::SOFTMAX_WARPS);
        mbar_init(&bars[C::DRAIN], 1);
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TM_COLS);
        tmem_relinquish();
    }

    // ---- this cluster's range: total units, then the item that holds its start
    Walk walk;
    walk.groups = p.row_groups;
    walk.group_rows = ROWS * cs;
    walk.entries = p.batch * p.row_groups;
    {
        int* s_scan = reinterpret_cast<int*>(smem + C::scan);
        int* s_at = s_scan + 32;                         // start's entry, unit
        constexpr int NW = THREADS / 32;
        const int clusters = gridDim.x / cs, me = blockIdx.x / cs;
        auto entry_units = [&](int e, bool record) -> int {
            if (e >= walk.entries) return 0;
            const int eb = e / walk.groups;
            const Band d = band_of(p, eb, e - eb * walk.groups, walk.group_rows, record && e == eb * walk.groups);
            return max(1, d.tiles) * p.n_kv_heads;
        };
        int total = 0, mine0 = 0;                        // mine0: entry tid's units
        for (int e = tid; e < walk.entries; e += THREADS) {
            const int u = entry_units(e, blockIdx.x == 0);
            if (e == tid) mine0 = u;
            total += u;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) s_scan[warp] = total;
        __syncthreads();
        total = __reduce_add_sync(0xffffffffu, lane < NW ? s_scan[lane] : 0);
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
            for (int e0 = 0; e0 < walk.entries; e0 += THREADS) {
                const int u = e0 == 0 ? mine0 : entry_units(e0 + tid, false);
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
                    s_at[0] = e0 + tid;
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
    if (cs > 1) cluster_sync_all(); else __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // The warp walks the slots and waits; one elected lane issues.  Slot s
        // is loaded by CTA s % cs for the whole cluster, in boxes of
        // {128 bytes of the head dim, box_rows positions of a page}.
        const int oob = p.num_pages * p.page_size;           // past the pool: filled with zeros
        const uint16_t everyone = static_cast<uint16_t>((1u << cs) - 1u);
        const int box_rows = min(p.page_size, TILE), boxes = TILE / box_rows;
        int* s_rows = reinterpret_cast<int*>(smem + C::rows);
        int slot = 0, owner = 0;
        uint32_t use = 0;                                    // use number of the slot
        bool ok = true;
        int seq = 0;
        auto load_tile = [&](const CUtensorMap* tm, int kvh, const int* rows) {
#pragma unroll 1
            for (int c = 0; c < C::SLOTS; ++c) {
                const bool mine = owner == rank;
                if (use > 0) {
                    // issuer: everyone has read the slot; others: it was filled here
                    const int bar = mine ? C::EMPTY : C::FULL;
                    ok = __all_sync(0xffffffffu, wait_or_abort(&bars[bar + slot], (use & 1) ^ 1, p.err, abort));
                    if (!ok) return;
                }
                if (elect_one()) {
                    uint64_t* full = &bars[C::FULL + slot];
                    mbar_arrive_expect_tx(full, SLOT);
                    if (mine) {
                        uint8_t* dst = smem + C::ring + slot * SLOT;
                        const int c0 = c * (256 / C::EB);
#pragma unroll 1
                        for (int i = 0; i < boxes; ++i) {
                            const int row = rows[i];
                            if (cs > 1) {
                                tma_load_3d_multicast(dst, tm, full, c0, kvh, row, everyone);
                                tma_load_3d_multicast(dst + SIDE, tm, full, c0 + 128 / C::EB, kvh, row, everyone);
                            } else {
                                tma_load_3d(dst, tm, full, c0, kvh, row);
                                tma_load_3d(dst + SIDE, tm, full, c0 + 128 / C::EB, kvh, row);
                            }
                            dst += box_rows * 128;
                        }
                    }
                }
                __syncwarp();
                ++seq;
                owner = owner + 1 == cs ? 0 : owner + 1;
                if (++slot == NS) {
                    slot = 0;
                    owner = 0;
                    ++use;
                }
            }
        };
        while (ok && walk.next(p)) {
            const int n = walk.n;
            // lane i: pool row of box i of tile t, or oob where no row sees a position of it
            auto row_of = [&](int t) -> int {
                if (t >= n || lane >= boxes) return oob;
                const Band& d = walk.band;
                const int pos = d.key0(walk.first + t) + lane * box_rows;
                if (pos >= d.hi || !(pos + box_rows > d.lo || pos < d.sink_end)) return oob;
                const int page = p.page_table[static_cast<size_t>(walk.b) * p.max_pages_per_seq + pos / p.page_size];
                if (page < 0 || page >= p.num_pages) {
                    report_error(p.err, FA512_DEVICE_ERR_INDEX);
                    return oob;
                }
                return page * p.page_size + pos % p.page_size;
            };
            // K(0) .. K(LOOK - 1), then K(j) V(j - LOOK) by turns
            int row_next = n > 0 ? row_of(0) : oob;          // of K(j), a step ahead of its use
            for (int j2 = 0; j2 < 2 * (n + LOOK) && ok; ++j2) {
                const int j = j2 >> 1, t = j - LOOK;
                const bool v = j2 & 1;
                if (v ? t < 0 : j >= n) continue;
                const int slot_rows = ((v ? t : j) & 3) * 8;
                if (!v) {
                    const int row = row_next;
                    row_next = row_of(j + 1);
                    if (lane < 8) s_rows[slot_rows + lane] = row;
                    __syncwarp();
                }
                load_tile(v ? &tmv : &tmk, walk.kvh, s_rows + slot_rows);
            }
        }
        // after an abort: no copy may land once this CTA has gone
        if (!ok)
            for (int i = max(0, seq - NS); i < seq; ++i)
                (void)mbar_wait(&bars[C::FULL + i % NS], (i / NS) & 1, p.err);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        // the whole warp walks the tiles and waits; one elected lane issues
        const uint32_t ring = smem_u32(smem + C::ring);
        const uint64_t qd = make_sdesc_sw128(smem_u32(smem + C::q), 16, 1024);
        const uint64_t pd = make_sdesc_lines<C::P_LINE>(smem_u32(smem + C::p));
        constexpr uint32_t IDESC_QK = shape(ROWS) | (FP8 ? 0u : BF16_AB);
        constexpr uint32_t IDESC_PV = shape(ROWS) | (FP8 ? B_E5M2 : BF16_AB) | A_MN | B_MN;
        bool ok = true;
        int slot = 0, segment = 0;
        uint32_t use = 0;
        int g_p = 0;                                         // running tile number of P V
        int sbuf = 0;
        uint32_t suse = 0;
        auto wait = [&](int bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_abort(&bars[bar], parity, p.err, abort));
        };
        int owner = 0;                                       // the CTA that loads the slot
        auto next_slot = [&]() {
            owner = owner + 1 == cs ? 0 : owner + 1;
            if (++slot == NS) {
                slot = 0;
                owner = 0;
                ++use;
            }
        };
        auto free_slot = [&]() {                             // by the issuing lane
            if (cs > 1) tc_commit_to(&bars[C::EMPTY + slot], owner); else tc_commit(&bars[C::EMPTY + slot]);
        };
        auto issue_qk = [&]() -> bool {
            if (suse > 0 && !wait(C::S_FREE + sbuf, (suse & 1) ^ 1)) return false;
            const uint32_t sb = tmem + C::TM_S + static_cast<uint32_t>(sbuf * ROWS);
#pragma unroll 1
            for (int c = 0; c < C::SLOTS; ++c) {
                if (!wait(C::FULL + slot, use & 1)) return false;
                tc_fence_after_sync();
                const uint64_t kd = make_sdesc_sw128(ring + slot * SLOT, 16, 1024);
                const uint64_t qc = qd + static_cast<uint64_t>((c * 2 * C::Q_CHUNK) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {            // 32 bytes of the head dim at a time
                        const uint64_t a = kd + static_cast<uint64_t>(((k >> 2) * SIDE + (k & 3) * 32) >> 4);
                        const uint64_t q = qc + static_cast<uint64_t>(((k >> 2) * C::Q_CHUNK + (k & 3) * 32) >> 4);
                        if constexpr (FP8) {
                            tc_mma_f8(sb, a, q, IDESC_QK, (c | k) ? 1u : 0u);
                            tc_mma_f8(sb, a, q + static_cast<uint64_t>(C::Q_TERM >> 4), IDESC_QK, 1u);
                        } else {
                            tc_mma_ss(sb, a, q, IDESC_QK, (c | k) ? 1u : 0u);
                        }
                    }
                    free_slot();
                    if (c == C::SLOTS - 1) tc_commit(&bars[C::S_FULL + sbuf]);
                }
                __syncwarp();
                next_slot();
            }
            if (++sbuf == NB) {
                sbuf = 0;
                ++suse;
            }
            return true;
        };
        auto issue_pv = [&](bool fresh) -> bool {
            if (!wait(C::P_FULL, g_p & 1)) return false;
            const uint32_t acc0 = fresh ? 0u : 1u;
#pragma unroll 1
            for (int c = 0; c < C::SLOTS; ++c) {
                if (!wait(C::FULL + slot, use & 1)) return false;
                tc_fence_after_sync();
                const uint64_t vd = make_sdesc_sw128(ring + slot * SLOT, SIDE, 1024);
                if (elect_one()) {
                    if constexpr (FP8) {
                        // two 128-element blocks of the head dim
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int k = 0; k < TILE / 32; ++k)
#pragma unroll
                                for (int e = 0; e < C::P_TERMS; ++e)
                                    tc_mma_f8(tmem + C::TM_O + static_cast<uint32_t>((2 * c + m) * ROWS),
                                              vd + static_cast<uint64_t>((m * SIDE + k * 32 * 128) >> 4),
                                              pd + static_cast<uint64_t>((e * C::P_TERM + k * 32 * C::P_LINE) >> 4),
                                              IDESC_PV, (k | e) ? 1u : acc0);
                    } else {
                        // one block of 128: two boxes of 64 elements
#pragma unroll
                        for (int k = 0; k < TILE / 16; ++k)
                            tc_mma_ss(tmem + C::TM_O + static_cast<uint32_t>(c * ROWS),
                                      vd + static_cast<uint64_t>((k * 16 * 128) >> 4),
                                      pd + static_cast<uint64_t>((k * 16 * C::P_LINE) >> 4), IDESC_PV, k ? 1u : acc0);
                    }
                    free_slot();
                    if (c == C::SLOTS - 1) tc_commit(&bars[C::PV_DONE]);
                }
                __syncwarp();
                next_slot();
            }
            ++g_p;
            return true;
        };
        while (ok && walk.next(p)) {
            const int n = walk.n;
            if (n == 0) continue;
            if (!(ok = wait(C::Q_FULL, segment & 1))) break;
            for (int j = 0; j < n + LOOK && ok; ++j) {
                if (j < n) ok = issue_qk();
                if (ok && j >= LOOK) {
                    // an item's first P V overwrites O: the last one's must have been read
                    if (j == LOOK && segment > 0) {
                        ok = wait(C::O_FREE, (segment - 1) & 1);
                        tc_fence_after_sync();
                    }
                    if (ok) ok = issue_pv(j == LOOK);
                }
            }
            ++segment;
        }
        if (elect_one()) tc_commit(&bars[C::DRAIN]);
        __syncwarp();
        (void)mbar_wait(&bars[C::DRAIN], 0, p.err);
    } else {
        // -------------------------------------------------------------------- softmax
        constexpr int SW = C::SOFTMAX_WARPS;
        const int sw = warp - 2, quad = warp & 3, grp = sw >> 2;
        const int bar = 1 + grp;                             // the column group's four warps
        constexpr int ALL = 7;                               // barrier of all softmax warps
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int kk = quad * 32 + lane;                     // this thread's key of a tile
        const int col0 = grp * GW;                           // its rows
        const int W = p.mask_words, G = p.group;
        int* s_depth = reinterpret_cast<int*>(smem + C::depth);
        uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + C::mask);
        float* s_red = reinterpret_cast<float*>(smem + C::red);
        float* s_mult = reinterpret_cast<float*>(smem + C::mult);
        int4* s_see = reinterpret_cast<int4*>(smem + C::see);
        uint8_t* s_seen = smem + C::seen;
        bool ok = true;
        int g = 0;                                           // running tile number
        int sbuf = 0;
        uint32_t suse = 0;
        int ring_base = 0;                                   // ring entries of the segments before
        // Brings a segment's Q and tables in: after the S^T tiles of the last
        // segment (its Q has been read by then) and while its last P V runs.
        auto prologue = [&]() {
            const Band& bd = walk.band;
            const int n = walk.n, b = walk.b;
            const int row0 = (walk.grp * cs + rank) * ROWS;
            const int tok0 = row0 / G;
            if (n > 0) {
                // Q: rows as K-major B operand, zeros where there is no row
                constexpr int PER = ROWS / SW;               // rows of a warp: 4
                uint4 x[PER][2];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int r = sw + i * SW, t = (row0 + r) / G;
                    const bool real = t < bd.cnt;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        p.q + ((static_cast<size_t>(b) * p.q_len + (real ? t : 0)) * p.n_q_heads + walk.kvh * G +
                               (real ? (row0 + r) % G : 0)) * D) + 2 * lane;
                    x[i][0] = real ? src[0] : make_uint4(0u, 0u, 0u, 0u);
                    x[i][1] = real ? src[1] : make_uint4(0u, 0u, 0u, 0u);
                }
                bar_sync(ALL, SW * 32);                      // nobody uses the last segment's tables any more
                const int toks = max(0, min((row0 + ROWS - 1) / G, p.q_len - 1) - tok0 + 1);
                if (p.tree_mask) {
                    // bits at and behind cnt name no token
                    auto word = [&](int t, int w) -> uint32_t {
                        const int left = bd.cnt - 32 * w;
                        const uint32_t m = static_cast<uint32_t>(p.tree_mask[(static_cast<size_t>(b) * p.q_len + t) * W + w]);
                        return left >= 32 ? m : left <= 0 ? 0u : m & ((1u << left) - 1u);
                    };
                    for (int t = tid - 64; t < bd.cnt; t += SW * 32) {
                        int c = 0;
                        for (int w = 0; w < W; ++w) c += __popc(word(t, w));
                        s_depth[t] = c - 1;
                    }
                    for (int i = tid - 64; i < toks * W; i += SW * 32) {
                        const int t = tok0 + i / W, w = i % W;
                        s_mask[i] = t < bd.cnt ? word(t, w) : 0u;
                    }
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int r = sw + i * SW;
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
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::Q_FULL]);
            }
            if (n == 0) bar_sync(ALL, SW * 32);
            bar_sync(ALL, SW * 32);
            if (sw < ROWS / 32) {
                // row r sees key k iff k <= x and (k > y or k is a sink), and
                // its mask (from word z on) allows; x = INT_MIN: nothing
                const int r = sw * 32 + lane, t = (row0 + r) / G;
                const bool real = t < bd.cnt && bd.start + t >= 0;
                const int place = bd.start + (p.tree_mask && real && n > 0 ? s_depth[t] : t);
                s_see[r] = make_int4(!real ? INT_MIN : p.tree_mask ? bd.len : place,
                                     p.window > 0 ? place - p.window : INT_MIN, real ? (t - tok0) * W : 0, 0);
            }
            bar_sync(ALL, SW * 32);
        };
        int done = -1;                                       // tiles of the segment whose O is to be read, -1: none
        bool direct = false;                                 // its rows are whole
        for (;;) {
            const bool have = walk.next(p);
            if (have) prologue();
            if (done >= 0) {
                // ---- O of the last segment: four 128-element blocks, this
                // thread's element of each; the new one's S^T runs meanwhile
                if (!have) bar_sync(bar, 128);               // what to write is in shared memory
                if (done > 0) ok = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                if (!(ok = pair::bar_and(ALL, SW * 32, ok))) break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int o = 0; o < 4; ++o) {
                    uint32_t r[GW];
                    if (done > 0) {
                        pair::tmem_ld16(tmem + lanes + C::TM_O + static_cast<uint32_t>(o * ROWS + col0), r);
                        tmem_ld_wait();
                        if (o == 3) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars[C::O_FREE]);
                        }
                    }
                    const int d = o * 128 + kk;
#pragma unroll
                    for (int i = 0; i < GW; ++i) {
                        const uint4 info = *reinterpret_cast<const uint4*>(smem + C::info + (col0 + i) * 16);
                        const float f = __uint_as_float(info.z);
                        const size_t at = (static_cast<size_t>(info.y) << 32 | info.x) * D + d;
                        const float val = f != 0.f ? __uint_as_float(r[i]) * f : 0.f;
                        if (info.w) {
                            if (direct)
                                p.out[at] = __float2bfloat16_rn(val);
                            else
                                p.ws_o[at] = val;
                        }
                    }
                }
            }
            if (!have) break;
            const Band bd = walk.band;
            const int n = walk.n, first = walk.first;
            const int row0 = (walk.grp * cs + rank) * ROWS;
            float m[GW], l[GW];
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            bool out = false;
            bool fresh = true;                               // some row may not have a reference yet
            for (int t = 0; t < n; ++t, ++g) {
                const int key0 = bd.key0(first + t), key = key0 + kk;
                ok = ok && wait_or_abort(&bars[C::S_FULL + sbuf], suse & 1, p.err, abort);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after_sync();
                float x[GW];
                {
                    uint32_t raw[GW];
                    pair::tmem_ld16(tmem + lanes + C::TM_S + static_cast<uint32_t>(sbuf * ROWS + col0), raw);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < GW; ++i) x[i] = __uint_as_float(raw[i]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::S_FREE + sbuf]);
                if (++sbuf == NB) {
                    sbuf = 0;
                    ++suse;
                }
                // log2 units, less the rows' references
#pragma unroll
                for (int i = 0; i < GW; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&s_mult[col0 + i]);
                    x[i] = fmaf(x[i], f.x, fresh && m[i] == -INFINITY ? 0.f : -m[i]);
                    x[i + 1] = fmaf(x[i + 1], f.y, fresh && m[i + 1] == -INFINITY ? 0.f : -m[i + 1]);
                    x[i + 2] = fmaf(x[i + 2], f.z, fresh && m[i + 2] == -INFINITY ? 0.f : -m[i + 2]);
                    x[i + 3] = fmaf(x[i + 3], f.w, fresh && m[i + 3] == -INFINITY ? 0.f : -m[i + 3]);
                }
                // a tile of cached keys inside every row's window needs no mask
                const bool whole = key0 + TILE <= min(bd.start, bd.hi) &&
                                   (p.window <= 0 || key0 > bd.place_max - p.window || key0 + TILE <= bd.sink_end);
                bool seen = true;                            // by some row of the group
                if (!whole) {
                    const int c = key - bd.start;
                    const bool drafted = c >= 0 && p.tree_mask;
                    // the key's place; its own mask says whether a drafted one is seen
                    const int kp = drafted ? bd.start + s_depth[max(0, min(c, bd.cnt - 1))] : key;
                    const int last = key < bd.hi ? (drafted ? bd.start : key) : INT_MAX;
                    const bool sink = kp < bd.sink_end;
                    uint32_t bits = 0xffffffffu;
                    if (drafted && key < bd.hi) {
                        bits = 0u;
#pragma unroll
                        for (int i = 0; i < GW; ++i)
                            bits |= ((s_mask[s_see[col0 + i].z + (c >> 5)] >> (c & 31)) & 1u) << i;
                    }
                    seen = false;
#pragma unroll
                    for (int i = 0; i < GW; ++i) {
                        const int4 r = s_see[col0 + i];
                        const bool see = last <= r.x && (kp > r.y || sink) && ((bits >> i) & 1u);
                        x[i] = see ? x[i] : -INFINITY;
                        seen = seen || see;
                    }
                }
                float high = x[0];
#pragma unroll
                for (int i = 1; i < GW; ++i) high = fmaxf(high, x[i]);
                bool pv_waited = g == 0;
                if (bar_or(bar, 128, high > C::THR || fresh || !ok)) {
                    if (!(ok = pair::bar_and(bar, 128, ok))) break;
                    float v[GW];
#pragma unroll
                    for (int i = 0; i < GW; ++i) v[i] = x[i];
                    const float mx = reduce_columns(v, [](float a, float c) { return fmaxf(a, c); });
                    if (lane < GW) s_red[quad * ROWS + col0 + lane] = mx;
                    bar_sync(bar, 128);
                    const int cl = col0 + (lane & (GW - 1));
                    const float top = fmaxf(fmaxf(s_red[cl], s_red[ROWS + cl]),
                                            fmaxf(s_red[2 * ROWS + cl], s_red[3 * ROWS + cl]));
                    float mine = 1.f;                        // lane i: the factor of row col0 + i
                    fresh = false;
#pragma unroll
                    for (int i = 0; i < GW; ++i) {
                        // growth over the reference (over 0 where there was none)
                        const float up = __shfl_sync(0xffffffffu, top, i);
                        const bool none = m[i] == -INFINITY;
                        const float shift = none ? (up == -INFINITY ? 0.f : up) : fmaxf(up, 0.f);
                        const float a = none ? 1.f : fast_exp2(-shift);
                        m[i] = none ? up : m[i] + shift;
                        x[i] -= shift;
                        l[i] *= a;
                        fresh = fresh || m[i] == -INFINITY;
                        mine = lane == i ? a : mine;
                    }
                    if (t > 0) {
                        // O is at rest once P V of the last tile has completed
                        ok = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, ok);
                        pv_waited = true;
                        tc_fence_after_sync();
                        if (__any_sync(0xffffffffu, mine != 1.f)) {
#pragma unroll 1
                            for (int o = 0; o < 4; ++o) {
                                const uint32_t ta = tmem + lanes + C::TM_O + static_cast<uint32_t>(o * ROWS + col0);
                                uint32_t r[GW];
                                pair::tmem_ld16(ta, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < GW; ++i)
                                    r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xffffffffu, mine, i));
                                pair::tmem_st16(ta, r);
                            }
                            tmem_st_wait();
                        }
                    }
                    bar_sync(bar, 128);                      // s_red is free again
                }
#pragma unroll
                for (int i = 0; i < GW; ++i) {
                    x[i] = fast_exp2(x[i]);
                    l[i] += x[i];
                }
                // P's buffer is free, and V of this tile will be read, after P V of the last tile
                if (!pv_waited) {
                    ok = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                    ok = __all_sync(0xffffffffu, ok);
                }
                uint8_t* line = smem + C::p + kk * C::P_LINE;
                if constexpr (FP8) {
                    uint32_t w[3][4] = {};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a = x[2 * j] * C::P_SCALE, d = x[2 * j + 1] * C::P_SCALE;
#pragma unroll
                        for (int e = 0; e < 3; ++e) {
                            float va, vd;
                            w[e][j >> 1] |= e5m2_pair(a, d, va, vd) << (16 * (j & 1));
                            a -= va;
                            d -= vd;
                        }
                    }
                    const int piece = line_piece<C::P_LINE>(kk, grp);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        *reinterpret_cast<uint4*>(line + e * C::P_TERM + piece) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                } else {
#pragma unroll
                    for (int c = 0; c < GW / 8; ++c)
                        *reinterpret_cast<uint4*>(line + line_piece<C::P_LINE>(kk, grp * (GW / 8) + c)) =
                            make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                                       pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
                }
                // P = 0 must not meet the V row of a key that no row sees: it
                // may hold anything.  The column groups share out the tile's
                // slots and clear such a key's row there.  Every ring entry
                // before V(t) has been read once the last S^T tile before it
                // is complete (and P V of t - 1 is), so the wait for a slot is
                // one phase ahead at most.
                bool clear = false;
                if (!whole) {
                    s_seen[grp * TILE + kk] = seen;
                    if (!(ok = pair::bar_and(ALL, SW * 32, ok))) {
                        out = true;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < C::GROUPS; ++i) seen = seen || s_seen[i * TILE + kk];
                    clear = !pair::bar_and(ALL, SW * 32, seen);
                }
                if (clear) {
                    const int ahead = min(t + LOOK, n - 1);
                    for (int a = t + 1; a <= ahead; ++a) {
                        const int gs = g + a - t;
                        const bool got = wait_or_abort(&bars[C::S_FULL + gs % NB], (gs / NB) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                    }
                    const int seq0 = ring_base + (ahead + 1 + t) * C::SLOTS;
#pragma unroll 1
                    for (int c = grp; c < C::SLOTS; c += C::GROUPS) {
                        const int s = (seq0 + c) % NS;
                        const bool got = wait_or_abort(&bars[C::FULL + s], ((seq0 + c) / NS) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                        if (got && !seen) {
                            uint4* v = reinterpret_cast<uint4*>(smem + C::ring + s * SLOT + kk * 128);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = v[SIDE / 16 + e] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C::P_FULL]);
            }
            ring_base += 2 * n * C::SLOTS;
            // all go on or all stop (here or at a vote inside a tile): no warp
            // may wait at a barrier for one that has left
            if (out || !(ok = pair::bar_and(ALL, SW * 32, ok))) break;
            // ---- row sums: lanes, then the four quadrants' warps
            const float part = reduce_columns(l, [](float a, float c) { return a + c; });
            if (lane < GW) s_red[quad * ROWS + col0 + lane] = part;
            bar_sync(bar, 128);
            // ---- what to write: O / sum where this is the whole row, else the
            // unnormalised partial (zeros for a row that saw nothing)
            direct = walk.count == 1;
            const size_t S = static_cast<size_t>(p.num_splits);
            if (quad == 0) {
                float top = -INFINITY;                       // lane i: row col0 + i
#pragma unroll
                for (int i = 0; i < GW; ++i) top = lane == i ? m[i] : top;
                const int cl = col0 + (lane & (GW - 1)), r = row0 + cl, t = r / G;
                const float sum = (s_red[cl] + s_red[ROWS + cl]) + (s_red[2 * ROWS + cl] + s_red[3 * ROWS + cl]);
                const bool some = s_see[cl].x != INT_MIN && top != -INFINITY;
                const size_t row = (static_cast<size_t>(walk.b) * p.q_len + t) * p.n_q_heads + walk.kvh * G + (r - t * G);
                const size_t at = direct ? row : row * S + walk.index;
                const float unit = p.o_scale * (1.f / C::P_SCALE);
                const float factor = !some ? 0.f : direct ? unit / sum : unit;
                if (lane < GW) {
                    const bool mine = t < p.q_len;
                    *reinterpret_cast<uint4*>(smem + C::info + cl * 16) =
                        make_uint4(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), __float_as_uint(factor), mine);
                    if (mine && direct && p.lse)
                        p.lse[row] = some ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
                    if (mine && !direct) {
                        p.ws_ml[at * 2] = some ? top : -INFINITY;
                        p.ws_ml[at * 2 + 1] = some ? sum : 0.f;
                    }
                }
            }
            if (p.num_splits > 1 && walk.index == 0 && sw == 0 && lane == 0 && rank == 0)
                p.ws_count[static_cast<size_t>(walk.entry) * p.n_kv_heads + walk.kvh] = walk.count;
            done = n;
        }
    }
    // all threads of all CTAs: no copy or arrival may reach a CTA that has gone
    if (cs > 1) cluster_sync_all(); else __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::TM_COLS);
}

// One block per row that was left in segments and slice of its columns:
// combines the segments' (O, m, l) -- M = max m_s, w_s = 2^(m_s - M),
// O = sum w_s O_s / sum w_s l_s.  256 threads: column quads x groups of
// segments; every thread issues its first 16 segments' O loads before it
// needs a weight, so the merge costs about one round trip to memory.  Few
// rows are merged in four column slices each (CS = 4).
constexpr int MERGE_THREADS = 256;
constexpr int MERGE_AHEAD = 16;
constexpr int MAX_SPLITS = 1024;

template <int CS>
__global__ void __launch_bounds__(MERGE_THREADS) merge_kernel(const TreeParams p, int group_rows) {
    constexpr int QB = D / 4 / CS;                  // column quads of the slice
    constexpr int NG = MERGE_THREADS / QB;          // groups of segments
    __shared__ float sw[MAX_SPLITS];                // weights
    __shared__ float4 sacc[NG - 1][QB];
    __shared__ float sred[2][MERGE_THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x, bt = blockIdx.y;
    const int b = bt / p.q_len, t = bt - b * p.q_len;
    const int grp = (t * p.group + h % p.group) / group_rows;
    const int S = p.ws_count[(static_cast<size_t>(b) * p.row_groups + grp) * p.n_kv_heads + h / p.group];
    if (S <= 1) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = tid % QB, g = tid / QB;
    const int col = blockIdx.z * (D / CS) + quad * 4;
    const size_t row = static_cast<size_t>(bt) * p.n_q_heads + h;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + row * p.num_splits;
    const float* ob = p.ws_o + row * p.num_splits * D + col;
    float4 x[MERGE_AHEAD];
#pragma unroll
    for (int i = 0; i < MERGE_AHEAD; ++i) {
        const int s = g + i * NG;
        if (s < S) x[i] = *reinterpret_cast<const float4*>(ob + static_cast<size_t>(s) * D);
    }
    float M = -INFINITY;
    for (int s = tid; s < S; s += MERGE_THREADS) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) sred[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < MERGE_THREADS / 32; ++w) M = fmaxf(M, sred[0][w]);
    float L = 0.f;
    for (int s = tid; s < S; s += MERGE_THREADS) {
        const float2 v = ml[s];
        const float w = M == -INFINITY ? 0.f : fast_exp2(v.x - M);
        sw[s] = w;
        L = fmaf(w, v.y, L);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) sred[1][warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < MERGE_THREADS / 32; ++w) L += sred[1][w];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int s, const float4& v) {
        const float w = sw[s];
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    };
#pragma unroll
    for (int i = 0; i < MERGE_AHEAD; ++i)
        if (g + i * NG < S) add(g + i * NG, x[i]);
#pragma unroll 4
    for (int s = g + MERGE_AHEAD * NG; s < S; s += NG)
        add(s, *reinterpret_cast<const float4*>(ob + static_cast<size_t>(s) * D));
    if (g > 0) sacc[g - 1][quad] = acc;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < NG - 1; ++i) {
        const float4 a = sacc[i][quad];
        acc.x += a.x;
        acc.y += a.y;
        acc.z += a.z;
        acc.w += a.w;
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    uint2 packed;
    packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * D + col) = packed;
    if (p.lse && tid == 0 && blockIdx.z == 0)
        p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

// Resident clusters of `cs` CTAs of one kernel variant on the current device
// (0 when the query fails), asked once per device, which also opts the kernel
// into its shared memory there.
template <bool FP8, int ROWS>
int resident_clusters(int cs) {
    static std::mutex mu;
    static int known[64][MAX_CLUSTER + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    int& n = known[dev][cs];
    if (n == 0) {
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3(cs);
        cfg.blockDim = dim3(Cfg<FP8, ROWS>::THREADS);
        cfg.dynamicSmemBytes = Cfg<FP8, ROWS>::total + 1024;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cs;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int got = 0;
        if (cudaFuncSetAttribute(tree_kernel<FP8, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<FP8, ROWS>::total + 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&got, tree_kernel<FP8, ROWS>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n = got;
    }
    return n;
}

template <bool FP8, int ROWS>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    const int clusters = resident_clusters<FP8, ROWS>(p.cluster);
    if (clusters < 1) return cudaErrorLaunchOutOfResources;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    const long long units = static_cast<long long>(p.batch) * p.row_groups * p.n_kv_heads *
                            (p.num_splits == 1 ? 1 : p.max_tiles > 1 ? p.max_tiles : 1);
    cfg.gridDim = dim3(static_cast<unsigned>(units < clusters ? units : clusters) * p.cluster);
    cfg.blockDim = dim3(Cfg<FP8, ROWS>::THREADS);
    cfg.dynamicSmemBytes = Cfg<FP8, ROWS>::total + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_kernel<FP8, ROWS>, tmk, tmv, p);
    if (e != cudaSuccess || p.num_splits == 1) return e;
    // the merge may be scheduled while the tiles are walked (it waits for them)
    memset(&cfg, 0, sizeof cfg);
    const bool sliced = decode_merge_sliced(static_cast<long long>(p.n_q_heads) * p.batch * p.q_len);
    cfg.gridDim = dim3(p.n_q_heads, p.batch * p.q_len, sliced ? 4 : 1);
    cfg.blockDim = dim3(MERGE_THREADS);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return sliced ? cudaLaunchKernelEx(&cfg, merge_kernel<4>, p, ROWS * p.cluster)
                  : cudaLaunchKernelEx(&cfg, merge_kernel<1>, p, ROWS * p.cluster);
}

}  // namespace tree

int tree_max_nodes() { return tree::MAX_NODES; }
int tree_tile() { return tree::TILE; }

// 32-row CTAs where all rows of a KV head fit one, else 64-row CTAs, the row
// tiles of a KV head in clusters of at most 4 (as even as possible).
TreeShape tree_shape(int q_len, int group) {
    const long long rows = static_cast<long long>(q_len) * group;
    TreeShape s;
    s.rows = rows <= 32 ? 32 : 64;
    const long long tiles = (rows + s.rows - 1) / s.rows;
    const long long groups = (tiles + 3) / 4;
    s.cluster = static_cast<int>((tiles + groups - 1) / groups);
    s.groups = static_cast<int>((tiles + s.cluster - 1) / s.cluster);
    return s;
}

cudaError_t launch_decode_tree(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                               cudaStream_t stream) {
    if (p.rows == 32)
        return fp8 ? tree::launch<true, 32>(tmk, tmv, p, stream) : tree::launch<false, 32>(tmk, tmv, p, stream);
    return fp8 ? tree::launch<true, 64>(tmk, tmv, p, stream) : tree::launch<false, 64>(tmk, tmv, p, stream);
}

}  // namespace fa512
