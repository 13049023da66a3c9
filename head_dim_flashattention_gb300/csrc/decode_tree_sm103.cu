// Drafted tokens (a tree of them, or a plain run) over a paged cache, head
// dim 512, sm_103a.
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
// Bound: the cache's bytes.  Per 128 keys a CTA streams 256 KiB (bf16), ~5.9 us
// at an SM's share of the measured 6.77 TB/s, against ~1.6 us of tensor work
// (an M = 128, N = 64, K = 16 MMA takes 48 cycles: it reads its operands from
// shared memory at 128 bytes a cycle).  So the ring takes all shared memory
// that Q and P leave, in slots of 32 KiB (few barriers, one elected lane that
// issues; slots of 8 KiB left the producer the bound: 889 -> 617 us for 64
// rows over 16 caches of 20,000 to 28,672 positions).  Measured (box to box): 64
// sequences of 16,384 positions in E4M3, 32 rows: 625-648 us, 6.7-6.9 TB/s, 98-102
// % of the measured copy rate; 16 sequences of 8,192 positions in bf16: 172-174 us
// with 32 rows, 183-186 us with 64; one of 4,096 positions with 16 rows: 19.3-20.1
// us, where a bare read of its 32 MB takes ~12: start and lengths 4, Q 2, one
// tile's products 3, O and its partials 5, the merge 4 us after one another.
//
// The row maxima lie across lanes here, so they are not reduced every tile:
// each thread compares its scores with the reference its rows hold, and only
// when some score is above it by 2^THR (a vote at the tile's one barrier) do
// the four warps of a column group reduce the maxima and rescale O.  The row
// sums stay per-thread partials until the end.
//
// The 16-bit MMA takes P rounded to bf16 (half a step, 2^-8 of each weight);
// the row sums take the weights as they are, so that the LSE carries none of it
// and O is off by at most 2^-8 sum p |v| / sum p.
//
// FP8 E4M3 cache: the bytes are MMA operands as stored (kind::f8f6f4).  Each
// query row is scaled by a power of two so that its largest element is in
// [128, 256) and written as the sum of two E4M3 terms (exact for elements from
// 2^-9 of the largest upward, off by at most 2^-17 of it below), and P as the
// sum of three E5M2 terms (relative error 2^-9, down to 2^-28 of the
// reference), so every product keeps at least the accuracy of the bf16 path
// without widening a byte of the cache.
//
// Work: the (sequence, row group, KV head) items' tiles, one after another,
// are cut into equal ranges, one per SM, so every SM streams the same number
// of tiles whatever the lengths (where there is an SM for every item, each
// takes one equal segment of one item instead); an item in several pieces leaves
// (O, m, l) partials that a merge kernel combines, any other is written
// directly.
#include <cuda.h>

#include "fa512_tree.cuh"

namespace fa512 {
namespace tree {
namespace single {

constexpr int TILE = 128;                // keys per tile: M of S^T
constexpr int GW = 16;                   // rows (columns of S^T) of a softmax warp
constexpr int LOOK = 2;                  // S^T tiles computed ahead of O^T += V^T P^T
constexpr int NB = LOOK + 1;             // S^T buffers
using Walk = WalkOf<TILE>;
using Band = BandOf<TILE>;

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
    static constexpr int cols = q + Q_TERMS * Q_TERM;    // [MAX_NODES][ROWS / 32]: the rows that see a token
    static constexpr int depth = cols + MAX_NODES * (ROWS / 32) * 4;
    static constexpr int red = depth + MAX_NODES * 4;    // [4][ROWS] float
    static constexpr int mult = red + 4 * ROWS * 4;      // [ROWS] float: score -> log2 units
    static constexpr int low = mult + ROWS * 4;            // [ROWS] int: the rows' last key below the window; INT_MAX: sees nothing
    static constexpr int rows = low + ROWS * 4;        // [4 tiles][8 boxes] int: the producer's pool rows
    static constexpr int seen = rows + 4 * 8 * 4;         // [GROUPS][TILE] bytes: some row of the group sees the key
    static constexpr int scan = seen + GROUPS * TILE;    // start_walk's
    static constexpr int info = scan + (36 + 32) * 4;      // [ROWS] 16 bytes: what the epilogue writes
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

__device__ __forceinline__ void tma_load_3d_hint(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                                 int c2, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, 8-bit floating-point operands.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

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

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[C::FULL + i], 1);
            mbar_init(&bars[C::EMPTY + i], 1);
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

    // ---- this block's range of the items' tiles
    Walk walk;
    walk.groups = 1;
    walk.group_rows = ROWS;
    start_walk<TILE, THREADS>(walk, p, gridDim.x, blockIdx.x, reinterpret_cast<int*>(smem + C::scan));
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // The warp walks the slots and waits; one elected lane issues boxes of
        // {128 bytes of the head dim, box_rows positions of a page}.
        const int oob = p.num_pages * p.page_size;           // past the pool: filled with zeros
        const int box_rows = min(p.page_size, TILE), boxes = TILE / box_rows;
        int* s_rows = reinterpret_cast<int*>(smem + C::rows);
        const uint64_t stream = pair::l2_policy_stream();    // the cache is read once (199 -> 187 us)
        int slot = 0;
        uint32_t use = 0;                                    // use number of the slot
        bool ok = true;
        int seq = 0;
        auto load_tile = [&](const CUtensorMap* tm, int kvh, const int* rows) {
#pragma unroll 1
            for (int c = 0; c < C::SLOTS; ++c) {
                if (use > 0) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&bars[C::EMPTY + slot], (use & 1) ^ 1, p.err, abort));
                    if (!ok) return;
                }
                if (elect_one()) {
                    uint64_t* full = &bars[C::FULL + slot];
                    mbar_arrive_expect_tx(full, SLOT);
                    uint8_t* dst = smem + C::ring + slot * SLOT;
                    const int c0 = c * (256 / C::EB);
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i) {
                        tma_load_3d_hint(dst, tm, full, c0, kvh, rows[i], stream);
                        tma_load_3d_hint(dst + SIDE, tm, full, c0 + 128 / C::EB, kvh, rows[i], stream);
                        dst += box_rows * 128;
                    }
                }
                __syncwarp();
                ++seq;
                if (++slot == NS) {
                    slot = 0;
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
                const int pos = d.key((walk.first + t) * TILE + lane * box_rows);
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
        constexpr uint32_t IDESC_QK = idesc_shape(128, ROWS) | (FP8 ? 0u : BF16_AB);
        constexpr uint32_t IDESC_PV = idesc_shape(128, ROWS) | (FP8 ? B_E5M2 : BF16_AB) | A_MN | B_MN;
        bool ok = true;
        int slot = 0, segment = 0;
        uint32_t use = 0;
        int g_p = 0;                                         // running tile number of P V
        int sbuf = 0;
        uint32_t suse = 0;
        auto wait = [&](int bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_abort(&bars[bar], parity, p.err, abort));
        };
        auto next_slot = [&]() {
            if (++slot == NS) {
                slot = 0;
                ++use;
            }
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
                    tc_commit(&bars[C::EMPTY + slot]);
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
                    tc_commit(&bars[C::EMPTY + slot]);
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
        uint32_t* s_cols = reinterpret_cast<uint32_t*>(smem + C::cols);
        float* s_red = reinterpret_cast<float*>(smem + C::red);
        float* s_mult = reinterpret_cast<float*>(smem + C::mult);
        int* s_low = reinterpret_cast<int*>(smem + C::low);
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
            constexpr int row0 = 0;                // one row group
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
                if (p.tree_mask) {
                    load_depths(p, b, bd.cnt, s_depth, tid - 64, SW * 32);
                    // a warp per (word, 32 rows): lane i brings row i's word, ballots turn it over
#pragma unroll 1
                    for (int u = sw; u < W * (ROWS / 32) && 32 * (u / (ROWS / 32)) < bd.cnt; u += SW) {
                        const int w = u / (ROWS / 32), half = u % (ROWS / 32);
                        const int t = (half * 32 + lane) / G;
                        const uint32_t word = t < bd.cnt && bd.start + t >= 0 ? mask_word(p, b, bd.cnt, t, w) : 0u;
                        uint32_t mine = 0u;
#pragma unroll 4
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t col = __ballot_sync(0xffffffffu, (word >> i) & 1u);
                            mine = lane == i ? col : mine;
                        }
                        s_cols[(32 * w + lane) * (ROWS / 32) + half] = mine;
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
                        const float qs = query_scale(x[i]);
                        uint4 hi, lo;
                        split_query(x[i], qs, hi, lo);
                        // this lane's 16 bytes: chunk lane / 8, piece lane % 8
                        uint8_t* line = smem + C::q + (lane >> 3) * C::Q_CHUNK + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                        *reinterpret_cast<uint4*>(line) = hi;
                        *reinterpret_cast<uint4*>(line + C::Q_TERM) = lo;
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
                const int r = sw * 32 + lane, t = (row0 + r) / G;
                const bool real = t < bd.cnt && bd.start + t >= 0;
                const int place = bd.start + (p.tree_mask && real && n > 0 ? s_depth[t] : t);
                s_low[r] = !real ? INT_MAX : p.window > 0 && place >= INT_MIN + p.window ? place - p.window : INT_MIN;
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
            constexpr int row0 = 0;
            float m[GW], l[GW];
#pragma unroll
            for (int i = 0; i < GW; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            bool out = false;
            bool fresh = true;                               // some row may not have a reference yet
            for (int t = 0; t < n; ++t, ++g) {
                const int v0 = (first + t) * TILE, key = bd.key(v0 + kk);
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
                const bool whole = bd.whole(p, v0);
                bool seen = true;                            // by some row of the group
                if (!whole) {
                    // bit i: row col0 + i sees this thread's key
                    const uint32_t vis = rows_that_see<GW>(p, bd, key, col0, s_depth, s_low + col0,
                                                           [&](int c) { return s_cols[c * (ROWS / 32) + (col0 >> 5)] >> (col0 & 31); });
                    seen = vis != 0u;
#pragma unroll
                    for (int i = 0; i < GW; ++i) x[i] = vis & (1u << i) ? x[i] : -INFINITY;
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
                    uint4 w[3];
                    split_weights(x, C::P_SCALE, w);
                    const int piece = line_piece<C::P_LINE>(kk, grp);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        *reinterpret_cast<uint4*>(line + e * C::P_TERM + piece) = w[e];
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
                            for (int e = 0; e < 8; ++e)                // no bank twice
                                v[(e + lane) & 7] = v[SIDE / 16 + ((e + lane) & 7)] = make_uint4(0u, 0u, 0u, 0u);
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
            if (quad == 0) {
                float top = -INFINITY;                       // lane i: row col0 + i
#pragma unroll
                for (int i = 0; i < GW; ++i) top = lane == i ? m[i] : top;
                const int cl = col0 + (lane & (GW - 1)), r = row0 + cl, t = r / G;
                const float sum = (s_red[cl] + s_red[ROWS + cl]) + (s_red[2 * ROWS + cl] + s_red[3 * ROWS + cl]);
                const bool some = some_key(s_low[cl], top, sum);
                const size_t row = (static_cast<size_t>(walk.b) * p.q_len + t) * p.n_q_heads + walk.kvh * G + (r - t * G);
                const size_t at = direct ? row : partial_at(p, row, cl, walk.index, blockIdx.x);
                const float unit = p.o_scale * (1.f / C::P_SCALE);
                const float factor = !some ? 0.f : direct ? unit / sum : unit;
                if (lane < GW) {
                    const bool mine = t < p.q_len;
                    *reinterpret_cast<uint4*>(smem + C::info + cl * 16) =
                        make_uint4(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), __float_as_uint(factor), mine);
                    if (mine && direct && p.lse)
                        p.lse[row] = some ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
                    if (mine && !direct) {
                        p.ws_ml[at * 2] = partial_max(some, top, sum);
                        p.ws_ml[at * 2 + 1] = some ? sum : 0.f;
                    }
                }
            }
            if (p.num_splits > 1 && walk.index == 0 && sw == 0 && lane == 0)
                leave_item(p, walk.entry, walk.kvh, walk.count, walk.stride, blockIdx.x);
            done = n;
        }
    }
    // all threads of all CTAs: no copy or arrival may reach a CTA that has gone
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::TM_COLS);
}

// SMs of the current device once the kernel is opted into its shared memory
// there (0: a query failed); asked once per device.
template <bool FP8, int ROWS>
int resident_blocks() {
    static std::mutex mu;
    static int known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        int n = 0;
        if (cudaFuncSetAttribute(tree_kernel<FP8, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<FP8, ROWS>::total + 1024) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev] = n;
    }
    return known[dev];
}

template <bool FP8, int ROWS>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    const int blocks = resident_blocks<FP8, ROWS>();
    if (blocks < 1) return cudaErrorLaunchOutOfResources;
    const long long units = static_cast<long long>(p.batch) * p.n_kv_heads *
                            (p.num_splits == 1 ? 1 : p.max_tiles > 1 ? p.max_tiles : 1);
    const int most = blocks < p.clusters ? blocks : p.clusters;
    tree_kernel<FP8, ROWS><<<static_cast<unsigned>(units < most ? units : most), Cfg<FP8, ROWS>::THREADS,
                             Cfg<FP8, ROWS>::total + 1024, stream>>>(tmk, tmv, p);
    return cudaGetLastError();
}

}  // namespace single

// One block per row that was left in segments and slice of its columns:
// combines the segments' (O, m, l) -- M = max m_s, w_s = 2^(m_s - M),
// O = sum w_s O_s / sum w_s l_s.  256 threads: column quads x groups of
// segments; every thread issues its first 16 segments' O loads before it
// needs a weight, so the merge costs about one round trip to memory.  Rows too
// few to give every SM a block are merged in four column slices each (CS = 4):
// 16 rows of 131,072 positions 91 us instead of 94 with the attention.  SLOTS:
// the partials are in slots (TreeParams); a step known when the kernel is
// compiled leaves the loads without address arithmetic (0.3 of 43 us).
constexpr int MERGE_THREADS = 256;
constexpr int MERGE_AHEAD = 16;
constexpr int MAX_SPLITS = 1024;

template <int CS, bool SLOTS>
__global__ void __launch_bounds__(MERGE_THREADS) merge_kernel(const TreeParams p, int group_rows) {
    constexpr int QB = D / 4 / CS;                  // column quads of the slice
    constexpr int NG = MERGE_THREADS / QB;          // groups of segments
    __shared__ float sw[MAX_SPLITS];                // weights
    __shared__ float4 sacc[NG - 1][QB];
    __shared__ float sred[2][MERGE_THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x, bt = blockIdx.y;
    const int b = bt / p.q_len, t = bt - b * p.q_len;
    const size_t row = static_cast<size_t>(bt) * p.n_q_heads + h;
    const Segments segs = segments_of<SLOTS>(p, row, b, t, h, group_rows);
    const int S = segs.n;
    if (S <= 1) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = tid % QB, g = tid / QB;
    const int col = blockIdx.z * (D / CS) + quad * 4;
    const float2* ml = reinterpret_cast<const float2*>(p.ws_ml);
    const float* ob = p.ws_o + segs.base * D + col;
    const float* ob0 = p.ws_o + segs.at(g) * D + col;
    const size_t step = SLOTS ? static_cast<size_t>(segs.step) * D : D;
    float4 x[MERGE_AHEAD];
#pragma unroll
    for (int i = 0; i < MERGE_AHEAD; ++i) {
        const int s = g + i * NG;
        if (s < S) x[i] = *reinterpret_cast<const float4*>(i == 0 ? ob0 : ob + s * step);
    }
    float M = -INFINITY;
    for (int s = tid; s < S; s += MERGE_THREADS) M = fmaxf(M, ml[segs.at(s)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) sred[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < MERGE_THREADS / 32; ++w) M = fmaxf(M, sred[0][w]);
    float L = 0.f;
    for (int s = tid; s < S; s += MERGE_THREADS) {
        const float2 v = ml[segs.at(s)];
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
        add(s, *reinterpret_cast<const float4*>(ob + s * step));
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

// The same for many rows of at most 32 segments: a warp per row, a lane per
// segment for the weights and per 16 columns for the sum, so that a row costs
// no block barrier and an SM has dozens of rows in flight.  It reads its
// segments one pair after another, so it pays from the fourth wave of blocks
// (two an SM) on; whole calls, warps / blocks: 512 rows 65.9 / 61.4 us, 768
// 81.8 / 80.8, 1,024 98.2 / 100.3, 2,048 81.0 / 88.7, 4,096 83.7 / 105.7,
// 19,200 260 / 322.
constexpr int MERGE_ROWS = 8;                       // warps, rows, of a block
__global__ void __launch_bounds__(MERGE_ROWS * 32) merge_rows_kernel(const TreeParams p, int group_rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const size_t row = static_cast<size_t>(blockIdx.x) * MERGE_ROWS + (threadIdx.x >> 5);
    if (row >= static_cast<size_t>(p.batch) * p.q_len * p.n_q_heads) return;
    const int h = static_cast<int>(row % p.n_q_heads);
    const size_t bt = row / p.n_q_heads;
    const int b = static_cast<int>(bt / p.q_len), t = static_cast<int>(bt - static_cast<size_t>(b) * p.q_len);
    const Segments segs = p.slot_rows > 0 ? segments_of<true>(p, row, b, t, h, group_rows)
                                            : segments_of<false>(p, row, b, t, h, group_rows);
    const int S = segs.n;
    if (S <= 1) return;
    constexpr int Q = D / 128, AHEAD = 2;           // column quads of a lane; segments loaded at once
    float4 x[AHEAD][Q];
    const float4* ob = reinterpret_cast<const float4*>(p.ws_o) + segs.at(0) * (D / 4) + lane;      // of the next segment
    int step = (segs.step - segs.first) * (D / 4);
    auto load = [&](int s0) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (s0 + a < S)
#pragma unroll
                for (int q = 0; q < Q; ++q) x[a][q] = ob[32 * q];
            ob += step;
            step = segs.step * (D / 4);
        }
    };
    load(0);
    const float2 ml = lane < S ? reinterpret_cast<const float2*>(p.ws_ml)[segs.at(lane)]
                               : make_float2(-INFINITY, 0.f);
    float M = ml.x;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float w = M == -INFINITY ? 0.f : fast_exp2(ml.x - M);
    float L = w * ml.y;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 acc[Q] = {};
    for (int s0 = 0;;) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const float ws = __shfl_sync(0xffffffffu, w, (s0 + a) & 31);
            if (s0 + a < S)
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    acc[q].x = fmaf(ws, x[a][q].x, acc[q].x);
                    acc[q].y = fmaf(ws, x[a][q].y, acc[q].y);
                    acc[q].z = fmaf(ws, x[a][q].z, acc[q].z);
                    acc[q].w = fmaf(ws, x[a][q].w, acc[q].w);
                }
        }
        if ((s0 += AHEAD) >= S) break;
        load(s0);
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    uint2* out = reinterpret_cast<uint2*>(p.out + row * D) + lane;
#pragma unroll
    for (int q = 0; q < Q; ++q)
        out[32 * q] = make_uint2(pack_bf16x2(acc[q].x * inv, acc[q].y * inv), pack_bf16x2(acc[q].z * inv, acc[q].w * inv));
    if (p.lse && lane == 0) p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

}  // namespace tree

// The merge may be scheduled while the tiles are walked (it waits for them).
cudaError_t launch_tree_merge(const TreeParams& p, int group_rows, cudaStream_t stream) {
    using namespace tree;
    const long long rows = static_cast<long long>(p.n_q_heads) * p.batch * p.q_len;
    const bool sliced = decode_merge_sliced(rows);
    const int sms = p.clusters * (p.rows == 128 ? 2 : 1);
    const bool by_warp = rows > 3 * 2 * sms && p.num_splits <= 32;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = by_warp ? dim3(static_cast<unsigned>((rows + MERGE_ROWS - 1) / MERGE_ROWS))
                          : dim3(p.n_q_heads, p.batch * p.q_len, sliced ? 4 : 1);
    cfg.blockDim = dim3(by_warp ? MERGE_ROWS * 32 : MERGE_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (by_warp) return cudaLaunchKernelEx(&cfg, merge_rows_kernel, p, group_rows);
    if (p.slot_rows > 0)
        return sliced ? cudaLaunchKernelEx(&cfg, merge_kernel<4, true>, p, group_rows)
                      : cudaLaunchKernelEx(&cfg, merge_kernel<1, true>, p, group_rows);
    return sliced ? cudaLaunchKernelEx(&cfg, merge_kernel<4, false>, p, group_rows)
                  : cudaLaunchKernelEx(&cfg, merge_kernel<1, false>, p, group_rows);
}

int tree_max_nodes() { return tree::MAX_NODES; }

// One CTA with 32 or 64 rows where all rows of a KV head fit, else CTA pairs
// with 128 rows each.  32 rows in the kernel for 32 / for 64 rows: 172 / 178 us
// (16 caches of 8,192 positions, bf16), 629 / 676 us (64 of 16,384, E4M3): the
// operands of the products that multiply zeros cost shared-memory reads and the
// softmax their time.  64 rows in the kernel for 64 / in a pair: 183 / 191 us
// (the 16), 38.6 / 46.5 us (one of 16,384), 119 / 177 us (the 16 in E4M3).
TreeShape tree_shape(int q_len, int group) {
    const long long rows = static_cast<long long>(q_len) * group;
    TreeShape s;
    s.rows = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    s.ctas = rows <= 64 ? 1 : 2;
    s.tile = 128 * s.ctas;
    s.groups = static_cast<int>((rows + s.rows - 1) / s.rows);
    return s;
}

cudaError_t launch_decode_tree(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                               cudaStream_t stream) {
    using namespace tree;
    cudaError_t e;
    if (p.rows == 128)
        e = launch_tree_pair(tmk, tmv, p, fp8, stream);
    else if (p.rows == 64)
        e = fp8 ? single::launch<true, 64>(tmk, tmv, p, stream) : single::launch<false, 64>(tmk, tmv, p, stream);
    else
        e = fp8 ? single::launch<true, 32>(tmk, tmv, p, stream) : single::launch<false, 32>(tmk, tmv, p, stream);
    return e != cudaSuccess || p.num_splits == 1 ? e : launch_tree_merge(p, p.rows, stream);
}

}  // namespace fa512
