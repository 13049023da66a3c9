// Tree decode of more than 64 rows per KV head: pairs of SMs, 128 rows each.
//
// The single-CTA kernel's products (S^T = K Q^T and O^T += V^T P^T) as 2-SM
// MMAs M = 256, N = 128: of a tile of 256 keys each CTA holds 128 keys of K
// (its 128 lanes of S^T, all 128 rows as columns) and the V of all 256 keys
// for half of the head dim (its 128 lanes of each of the two 256-element
// blocks of O^T).  So a pair streams every byte once, and a row of N costs an
// SM half its shared-memory reads: 48 cycles of operand reads per 64-cycle MMA
// where the single-CTA form reads 48 cycles for half the rows.
// Tensor memory: O^T 2 x 128 columns, S^T 2 buffers x 128 columns.
//
// Bound: the bytes of a cache that is read once (16 caches of 20,000 to 28,672
// positions, 128 rows: 476-490 us from box to box, 5.9-6.1 TB/s, 88-90 % of the
// measured copy rate).  Where several row groups share the keys, L2 brings them (8
// sequences of up to 75 tokens and 600 rows a KV head, window 4,096 and 4 sinks:
// 256-269 us, 0.45-0.48 PFLOP/s, 25 % of the measured rate) and the bound is the chain of a tile: its 64 MMAs take 2.1 us, and the MMA
// warp waits another 2.4 for loads and 0.9 for P; a change of item costs ~15 us
// of row sums, next Q, O and first references, two or three times a pair.
// Measured and not taken: slots of 16 KiB (355 -> 378 us: barriers and commits
// a slot; two slots of 32 KiB instead of three cost 12 us, so depth is not what
// bounds it), fetching the next tile into L2 ahead (354 -> 367), S^T two tiles
// ahead and P held in registers until P V is done (262 -> 264 each), a second
// warp that loads, in the cleaner's place and with its work on the courier (258
// -> 261; chunks of 300 tokens over 8,192 positions, where little is cleared,
// 357 -> 338).
//
// A CTA's softmax threads hold its 128 keys against all 128 rows; Q and P^T,
// the B operands, are split by rows, 64 in each CTA, so half of each P^T tile
// belongs in the other CTA: it is staged here, and a courier warp moves it
// with one bulk copy (a store into the other CTA would hold the softmax
// threads at their fence and release for two microseconds a tile).  Both CTAs
// have to scale by the same references: every tile, each column group (32
// rows) swaps its vote on "a score outgrew the reference" with the same group
// of the other CTA, and, when either says so, the column maxima; at the end of
// a segment the row sums.
//
// Keys that no row sees may hold anything, also NaN, which P = 0 would not
// silence: in the tiles where some may be (a sequence's end, a window's edges,
// the drafted tokens) V arrives on barriers of its own, and a cleaner warp
// clears the rows of such keys and hands each slot to the MMA.
#include <cuda.h>

#include <type_traits>

#include "fa512_tree.cuh"

namespace fa512 {
namespace tree {
namespace pairs {

using namespace fa512::pair;
using tree::wait_or_abort;
using tree::bar_sync;

constexpr int TILE = 256;                // keys per tile
constexpr int HALF_TILE = 128;           // keys of a CTA
constexpr int ROWS = 128;
constexpr int HALF_ROWS = 64;            // rows of a CTA's B operands
constexpr int GW = 32;                   // rows (columns of S^T) of a softmax warp
constexpr int GROUPS = ROWS / GW;
constexpr int SW = 4 * GROUPS;           // softmax warps: (column group, TMEM lane quadrant)
constexpr int COURIER = 2 + SW;          // warp that moves P to the other CTA
constexpr int CLEANER = COURIER + 1;     // warp that clears V rows
constexpr int THREADS = (CLEANER + 1) * 32;
constexpr int LOOK = 1;                  // S^T tiles computed ahead of O^T += V^T P^T
constexpr int NB = LOOK + 1;
constexpr uint32_t TM_O = 0, TM_S = 256;
constexpr int PLAIN = 0, FUSED = 1, LESS = 2;       // forms of the scores
using Walk = WalkOf<TILE>;
using Band = BandOf<TILE>;

template <bool FP8>
struct Cfg {
    static constexpr int EB = FP8 ? 1 : 2;
    static constexpr int NS = FP8 ? 2 : 3;               // ring slots
    static constexpr int CHUNKS = D * EB / 128;          // 128-byte column chunks of the head dim
    static constexpr int SLOTS = CHUNKS / 2;             // ring slots of a K (V) tile in a CTA: 4 or 2
    static constexpr int Q_CHUNK = HALF_ROWS * 128;
    static constexpr int Q_TERM = CHUNKS * Q_CHUNK;
    static constexpr int Q_TERMS = FP8 ? 2 : 1;
    static constexpr int P_LINE = HALF_ROWS * EB;        // a key's values of this CTA's rows
    static constexpr int P_TERM = TILE * P_LINE;
    static constexpr int P_TERMS = FP8 ? 3 : 1;
    static constexpr float THR = FP8 ? 4.f : 8.f;
    // E5M2 terms of small weights stay normal: the weights are 2^P_LOG times
    // theirs, by way of the references
    static constexpr float P_LOG = FP8 ? 11.f : 0.f, P_SCALE = FP8 ? 2048.f : 1.f;
    // shared memory, from a 1 KiB aligned base
    static constexpr int ring = 0;
    static constexpr int q = ring + NS * SLOT;
    static constexpr int p = q + Q_TERMS * Q_TERM;
    static constexpr int HALF_TERM = P_TERM / 2;         // one CTA's keys
    static constexpr int stage = p + P_TERMS * P_TERM;   // P of this CTA's keys for the other CTA's rows
    static constexpr int STAGE_BYTES = P_TERMS * HALF_TERM;
    static constexpr int cols = stage + STAGE_BYTES;     // [MAX_NODES][GROUPS]: the rows that see a token
    static constexpr int depth = cols + MAX_NODES * GROUPS * 4;
    static constexpr int red = depth + MAX_NODES * 4;    // [4][ROWS] float
    static constexpr int m = red + 4 * ROWS * 4;         // [ROWS] float: references
    static constexpr int mb = m + ROWS * 4;              // [ROWS / 2] float4: a row pair's factors (score -> log2 units) and negated references
    static constexpr int low = mb + ROWS * 8;            // [ROWS] int: the rows' last key below the window; INT_MAX: sees nothing
    static constexpr int info = low + ROWS * 4;        // [ROWS] 16 bytes: what the epilogue writes
    static constexpr int rows = info + ROWS * 16;        // [4 tiles][16 boxes] int: the producer's pool rows
    static constexpr int seen = rows + 4 * 16 * 4;       // [GROUPS][HALF_TILE] bytes
    static constexpr int pseen = seen + GROUPS * HALF_TILE;          // [2][HALF_TILE] int: the other CTA's keys
    static constexpr int vote = pseen + 2 * HALF_TILE * 4;           // [2][GROUPS][4] int: the other CTA's warps'
    static constexpr int top = vote + 2 * GROUPS * 16;               // [2][ROWS] float
    static constexpr int scan = top + 2 * ROWS * 4;
    static constexpr int bars = scan + ((SCAN_INTS * 4 + 15) & ~15);
    static constexpr int FULL = 0, EMPTY = NS, V_RAW = 2 * NS, V_CLEAN = 3 * NS, S_FULL = 4 * NS, S_FREE = S_FULL + NB,
                         P_FULL = S_FREE + NB, P_PEER = P_FULL + 1, STAGED = P_PEER + 1, PV_DONE = STAGED + 1, Q_FULL = PV_DONE + 1, O_FREE = Q_FULL + 1,
                         DRAIN = O_FREE + 1, VOTE = DRAIN + 1, TOP = VOTE + 2 * GROUPS, SEEN = TOP + 2 * GROUPS,
                         SEEN_HERE = SEEN + 2, N_BARS = SEEN_HERE + 1;
    static constexpr int misc = bars + N_BARS * 8;       // tmem address, abort flag
    static constexpr int total = misc + 16;
    static_assert(total + 1024 <= 232448, "shared memory of an SM");
    static_assert(vote % 16 == 0, "votes are read four at a time");
};

__device__ __forceinline__ void mma2_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void st_async_b32(uint32_t addr, uint32_t v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                 ::"r"(addr), "r"(v), "r"(bar)
                 : "memory");
}
// Bulk copy of `bytes` from this CTA's shared memory into another CTA's; the
// bytes complete_tx on the destination CTA's mbarrier.
__device__ __forceinline__ void bulk_copy_to_cluster(uint32_t dst_cluster, uint32_t src_cta, uint32_t bytes,
                                                     uint32_t bar_cluster) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst_cluster), "r"(src_cta), "r"(bytes), "r"(bar_cluster)
                 : "memory");
}

// Waits, bounded, with cluster-scope acquire: for arrivals of the other CTA.
static __device__ __noinline__ bool wait_cluster_slow(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    const uint32_t a = smem_u32(bar);
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_cluster(a, parity)) return true;
        if ((i & 255u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                report_error(err, FA512_DEVICE_ERR_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
    return mbar_try_wait_cluster(smem_u32(bar), parity) || wait_cluster_slow(bar, parity, err, abort);
}

// Brings the query rows of the walk's segment into L2, a lane a token: the
// softmax warps will ask for them when they come to it (22 runs of 46 tokens
// with 8 heads on one KV head: 298 -> 294 us).
__device__ __forceinline__ void prefetch_q(const TreeParams& p, const Walk& walk) {
    const int row0 = walk.grp * ROWS;
    const int end = min((row0 + ROWS - 1) / p.group + 1, walk.band.cnt);
#pragma unroll 1
    for (int t = row0 / p.group + static_cast<int>(threadIdx.x & 31); t < end; t += 32)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     ::"l"(p.q + ((static_cast<size_t>(walk.b) * p.q_len + t) * p.n_q_heads + walk.kvh * p.group) * D),
                     "r"(p.group * D * 2)
                     : "memory");
}

template <bool FP8>
__global__ void __launch_bounds__(THREADS, 1)
tree_pair_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                 const __grid_constant__ TreeParams p) {
    using C = Cfg<FP8>;
    constexpr int NS = C::NS;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::misc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    auto bar_of = [&](int i, int cta) -> uint32_t { return map_to_cta(smem_u32(&bars[i]), cta); };

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[C::FULL + i], 1);
            mbar_init(&bars[C::EMPTY + i], 1);
            mbar_init(&bars[C::V_RAW + i], 1);
            mbar_init(&bars[C::V_CLEAN + i], 2);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&bars[C::S_FULL + i], 1);
            mbar_init(&bars[C::S_FREE + i], 2 * SW);
        }
        mbar_init(&bars[C::P_FULL], SW);
        mbar_init(&bars[C::P_PEER], 1);
        mbar_init(&bars[C::STAGED], SW);
        mbar_init(&bars[C::PV_DONE], 1);
        mbar_init(&bars[C::Q_FULL], 2 * SW);
        mbar_init(&bars[C::O_FREE], 2 * SW);
        mbar_init(&bars[C::DRAIN], 1);
        for (int i = 0; i < 2 * GROUPS; ++i) {
            mbar_init(&bars[C::VOTE + i], 1);
            mbar_init(&bars[C::TOP + i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bars[C::SEEN + i], 1);
        mbar_init(&bars[C::SEEN_HERE], SW);
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    // ---- this pair's range of the items' tiles
    Walk walk;
    walk.groups = p.row_groups;
    walk.group_rows = ROWS;
    start_walk<TILE, THREADS>(walk, p, gridDim.x / 2, blockIdx.x / 2, reinterpret_cast<int*>(smem + C::scan));
    cluster_sync_all();
    if (warp == 1) {
        tmem_alloc2(tmem_slot, 512);
        tmem_relinquish2();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // Each CTA loads its own operands; a slot of both is counted on the
        // leader's barrier, a slot of V that has to be cleared on each CTA's own.
        const int oob = p.num_pages * p.page_size;           // past the pool: filled with zeros
        const int box_rows = min(p.page_size, HALF_TILE), boxes = HALF_TILE / box_rows;
        int* s_rows = reinterpret_cast<int*>(smem + C::rows);
        // a cache that one row group reads is read once: L2 drops its lines
        // first (16 caches of 20,000 to 28,672 positions: 508 -> 479 us); what
        // several groups read, it keeps
        const uint64_t policy = p.row_groups == 1 ? l2_policy_stream() : l2_policy_keep();
        int slot = 0;
        uint32_t use = 0;
        bool ok = true;
        bool start = true;                                   // the walk's first segment: its Q is being read
        uint32_t raw_used = 0, full_used = 0;                // per slot: parity of the uses of the two barriers
        while (ok && walk.next(p)) {
            const int n = walk.n;
            const Band& d = walk.band;
            if (rank == 0 && !start && n > 0) prefetch_q(p, walk);
            start = false;
            // lane i: pool row of box i of tile t, or oob where no row sees a position of it
            auto row_of = [&](int t) -> int {
                if (t >= n || lane >= 2 * boxes) return oob;
                const int pos = d.key((walk.first + t) * TILE + lane * box_rows);
                if (pos >= d.hi || !(pos + box_rows > d.lo || pos < d.sink_end)) return oob;
                const int page = p.page_table[static_cast<size_t>(walk.b) * p.max_pages_per_seq + pos / p.page_size];
                if (page < 0 || page >= p.num_pages) {
                    report_error(p.err, FA512_DEVICE_ERR_INDEX);
                    return oob;
                }
                return page * p.page_size + pos % p.page_size;
            };
            // K(0), then K(j) V(j - 1) by turns
            int row_next = n > 0 ? row_of(0) : oob;          // of K(j), a step ahead of its use
#pragma unroll 1
            for (int j2 = 0; j2 < 2 * (n + LOOK) && ok; ++j2) {
                const int j = j2 >> 1;
                const bool v = j2 & 1;
                const int t = v ? j - LOOK : j;
                if (t < 0 || t >= n) continue;
                int* rows = s_rows + (t & 3) * 16;
                if (!v) {
                    const int row = row_next;
                    row_next = row_of(j + 1);
                    if (lane < 16) rows[lane] = row;
                    __syncwarp();
                }
                const bool raw = v && d.dirty(p, (walk.first + t) * TILE);
                const CUtensorMap* tm = v ? &tmv : &tmk;
#pragma unroll 1
                for (int c = 0; c < C::SLOTS; ++c) {
                    if (use > 0) {
                        ok = __all_sync(0xffffffffu, wait_or_abort(&bars[C::EMPTY + slot], (use & 1) ^ 1, p.err, abort));
                        if (!ok) break;
                    }
                    if (elect_one()) {
                        uint64_t* full = &bars[(raw ? C::V_RAW : C::FULL) + slot];
                        const uint32_t bar = raw ? smem_u32(full) : bar_of(C::FULL + slot, 0);
                        if (raw) mbar_arrive_expect_tx(full, SLOT);
                        else if (rank == 0) mbar_arrive_expect_tx(full, 2 * SLOT);
#pragma unroll
                        for (int side = 0; side < 2; ++side) {
                            // K: columns of chunk 2c + side, this CTA's keys.  V: bf16 block c / 2, key
                            // half c % 2, its 64 elements `side`; FP8 block c, key half `side`.
                            const int col = !v ? (2 * c + side) * (128 / C::EB)
                                               : FP8 ? 256 * c + 128 * rank : 256 * (c >> 1) + 128 * rank + 64 * side;
                            const int half = !v ? rank : FP8 ? side : c & 1;
                            uint8_t* dst = smem + C::ring + slot * SLOT + side * SIDE;
#pragma unroll 1
                            for (int i = 0; i < boxes; ++i) {
                                tma2_load_3d_hint(dst, tm, bar, col, walk.kvh, rows[half * boxes + i], policy);
                                dst += box_rows * 128;
                            }
                        }
                    }
                    __syncwarp();
                    if (raw) raw_used ^= 1u << slot; else full_used ^= 1u << slot;
                    if (++slot == NS) {
                        slot = 0;
                        ++use;
                    }
                }
            }
        }
        // after an abort: no copy may land once this CTA has gone (the leader
        // sees its own and the other's slots, the other its clearing slots;
        // the cluster's barrier at the end holds both)
        if (!ok)
            for (int i = 0; i < NS; ++i) {
                if (rank == 0) (void)mbar_wait(&bars[C::FULL + i], ((full_used >> i) & 1) ^ 1, p.err);
                (void)mbar_wait(&bars[C::V_RAW + i], ((raw_used >> i) & 1) ^ 1, p.err);
            }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------------------ MMA issue, both SMs
            const uint32_t ring = smem_u32(smem + C::ring);
            const uint64_t qd = make_sdesc_sw128(smem_u32(smem + C::q), 16, 1024);
            const uint64_t pd = make_sdesc_lines<C::P_LINE>(smem_u32(smem + C::p));
            constexpr uint32_t IDESC_QK = idesc_shape(2 * 128, ROWS) | (FP8 ? 0u : BF16_AB);
            constexpr uint32_t IDESC_PV = idesc_shape(2 * 128, ROWS) | (FP8 ? B_E5M2 : BF16_AB) | A_MN | B_MN;
            bool ok = true;
            int slot = 0, segment = 0, g_p = 0, sbuf = 0;
            uint32_t suse = 0, full_used = 0, clean_used = 0;
            auto wait = [&](int bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait_cluster(&bars[bar], parity, p.err, abort));
            };
            auto next_slot = [&]() {
                if (++slot == NS) slot = 0;
            };
            auto issue_qk = [&]() -> bool {
                if (suse > 0 && !wait(C::S_FREE + sbuf, (suse & 1) ^ 1)) return false;
                const uint32_t sb = tmem + TM_S + static_cast<uint32_t>(sbuf * ROWS);
#pragma unroll 1
                for (int c = 0; c < C::SLOTS; ++c) {
                    if (!wait(C::FULL + slot, (full_used >> slot) & 1)) return false;
                    full_used ^= 1u << slot;
                    tc_fence_after_sync();
                    const uint64_t kd = make_sdesc_sw128(ring + slot * SLOT, 16, 1024);
                    const uint64_t qc = qd + static_cast<uint64_t>((c * 2 * C::Q_CHUNK) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {        // 32 bytes of the head dim at a time
                            const uint64_t a = kd + static_cast<uint64_t>(((k >> 2) * SIDE + (k & 3) * 32) >> 4);
                            const uint64_t q = qc + static_cast<uint64_t>(((k >> 2) * C::Q_CHUNK + (k & 3) * 32) >> 4);
                            if constexpr (FP8) {
                                mma2_f8(sb, a, q, IDESC_QK, (c | k) ? 1u : 0u);
                                mma2_f8(sb, a, q + static_cast<uint64_t>(C::Q_TERM >> 4), IDESC_QK, 1u);
                            } else {
                                mma2_ss(sb, a, q, IDESC_QK, (c | k) ? 1u : 0u);
                            }
                        }
                        commit2_both(&bars[C::EMPTY + slot]);
                        if (c == C::SLOTS - 1) commit2_both(&bars[C::S_FULL + sbuf]);
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
            auto issue_pv = [&](bool fresh, bool raw) -> bool {
                if (!wait(C::P_FULL, g_p & 1) || !wait(C::P_PEER, g_p & 1)) return false;
                const uint32_t acc0 = fresh ? 0u : 1u;
#pragma unroll 1
                for (int c = 0; c < C::SLOTS; ++c) {
                    uint32_t& used = raw ? clean_used : full_used;
                    if (!wait((raw ? C::V_CLEAN : C::FULL) + slot, (used >> slot) & 1)) return false;
                    used ^= 1u << slot;
                    tc_fence_after_sync();
                    const uint64_t vd = make_sdesc_sw128(ring + slot * SLOT, SIDE, 1024);
                    if (elect_one()) {
                        if constexpr (FP8) {
                            // block c of the head dim, both key halves
                            const uint32_t ob = tmem + TM_O + static_cast<uint32_t>(c * ROWS);
#pragma unroll
                            for (int k = 0; k < TILE / 32; ++k)
#pragma unroll
                                for (int e = 0; e < C::P_TERMS; ++e)
                                    mma2_f8(ob, vd + static_cast<uint64_t>((k * 32 * 128) >> 4),
                                            pd + static_cast<uint64_t>((e * C::P_TERM + k * 32 * C::P_LINE) >> 4),
                                            IDESC_PV, (k | e) ? 1u : acc0);
                        } else {
                            // block c / 2, key half c % 2
                            const uint32_t ob = tmem + TM_O + static_cast<uint32_t>((c >> 1) * ROWS);
                            const uint64_t ph = pd + static_cast<uint64_t>(((c & 1) * HALF_TILE * C::P_LINE) >> 4);
#pragma unroll
                            for (int k = 0; k < HALF_TILE / 16; ++k)
                                mma2_ss(ob, vd + static_cast<uint64_t>((k * 16 * 128) >> 4),
                                        ph + static_cast<uint64_t>((k * 16 * C::P_LINE) >> 4), IDESC_PV,
                                        (k | (c & 1)) ? 1u : acc0);
                        }
                        commit2_both(&bars[C::EMPTY + slot]);
                        if (c == C::SLOTS - 1) commit2_both(&bars[C::PV_DONE]);
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
#pragma unroll 1
                for (int j = 0; j < n + LOOK && ok; ++j) {
                    if (j < n) ok = issue_qk();
                    if (ok && j >= LOOK) {
                        // an item's first P V overwrites O: the last one's must have been read
                        if (j == LOOK && segment > 0) {
                            ok = wait(C::O_FREE, (segment - 1) & 1);
                            tc_fence_after_sync();
                        }
                        if (ok)
                            ok = issue_pv(j == LOOK,
                                          walk.band.dirty(p, (walk.first + j - LOOK) * TILE));
                    }
                }
                ++segment;
            }
            if (elect_one()) commit2_local(&bars[C::DRAIN]);
            __syncwarp();
            (void)mbar_wait(&bars[C::DRAIN], 0, p.err);
        }
    } else if (warp == COURIER) {
        // ------------------------------------------------ P for the other CTA's rows
        int g = 0;
        bool ok = true;
        while (ok && walk.next(p)) {
            const int n = walk.n;
#pragma unroll 1
            for (int t = 0; t < n && ok; ++t, ++g) {
                ok = __all_sync(0xffffffffu, wait_or_abort(&bars[C::STAGED], g & 1, p.err, abort));
                if (!ok) break;
                if (elect_one()) {
#pragma unroll
                    for (int e = 0; e < C::P_TERMS; ++e)
                        bulk_copy_to_cluster(map_to_cta(smem_u32(smem + C::p + e * C::P_TERM + rank * C::HALF_TERM), rank ^ 1),
                                             smem_u32(smem + C::stage + e * C::HALF_TERM), C::HALF_TERM,
                                             bar_of(C::P_FULL, rank ^ 1));
                }
                __syncwarp();
                if (rank == 1) {
                    // this CTA's operand is complete: the leader's MMA may read it
                    ok = __all_sync(0xffffffffu, wait_or_abort(&bars[C::P_FULL], g & 1, p.err, abort));
                    if (ok && lane == 0) mbar_arrive_remote(bar_of(C::P_PEER, 0));
                }
            }
        }
    } else if (warp == CLEANER) {
        // --------------------------------------- V rows of keys that no row sees
        const int box_rows = min(p.page_size, HALF_TILE);
        int* s_pseen = reinterpret_cast<int*>(smem + C::pseen);
        const uint8_t* s_seen = smem + C::seen;
        int slot = 0, masked = 0;
        uint32_t used = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_cluster(&bars[bar], parity, p.err, abort));
        };
        while (ok && walk.next(p)) {
            const int n = walk.n;
            const Band& bd = walk.band;
#pragma unroll 1
            for (int j = 0; j < n + LOOK && ok; ++j) {
                if (j < n) slot = (slot + C::SLOTS) % NS;    // K(j)
                if (j < LOOK) continue;
                const int v0 = (walk.first + j - LOOK) * TILE;
                if (!bd.dirty(p, v0)) {
                    slot = (slot + C::SLOTS) % NS;
                    continue;
                }
                // bits k + 4 h: this lane's key lane + 32 k of key half h is seen,
                // or lies in a box that no row needs and was filled with zeros
                uint32_t seen = 0u;
                if (p.tree_mask) {
                    // this CTA's keys: over the column groups; then both CTAs swap
                    const int par = masked & 1, peer = rank ^ 1;
                    ok = wait(C::SEEN_HERE, masked & 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars[C::SEEN + par], HALF_TILE * 4);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int kk = lane + 32 * k;
                        const bool any = s_seen[kk] || s_seen[HALF_TILE + kk] || s_seen[2 * HALF_TILE + kk] || s_seen[3 * HALF_TILE + kk];
                        seen |= any ? 1u << (k + 4 * rank) : 0u;
                        st_async_b32(map_to_cta(smem_u32(&s_pseen[par * HALF_TILE + kk]), peer), any ? 1u : 0u,
                                     bar_of(C::SEEN + par, peer));
                    }
                    ok = wait(C::SEEN + par, (masked >> 1) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        seen |= *const_cast<volatile int*>(&s_pseen[par * HALF_TILE + lane + 32 * k]) ? 1u << (k + 4 * peer) : 0u;
                    ++masked;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int key = bd.key(v0 + lane + 32 * k), pos = key & ~(box_rows - 1);
                    const bool loaded = pos < bd.hi && (pos + box_rows > bd.lo || pos < bd.sink_end);
                    const bool some = !p.tree_mask && key < bd.hi && (key >= bd.lo || key < bd.sink_end);
                    seen |= some || !loaded ? 1u << k : 0u;
                }
#pragma unroll 1
                for (int c = 0; c < C::SLOTS && ok; ++c) {
                    ok = wait(C::V_RAW + slot, (used >> slot) & 1);
                    if (!ok) break;
                    used ^= 1u << slot;
#pragma unroll 1
                    for (int side = 0; side < 2; ++side) {
                        const uint32_t here = seen >> (4 * (FP8 ? side : c & 1));
#pragma unroll 1
                        for (int k = 0; k < 4; ++k)
                            if (!((here >> k) & 1u)) {
                                uint4* v = reinterpret_cast<uint4*>(smem + C::ring + slot * SLOT + side * SIDE + (lane + 32 * k) * 128);
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[(e + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);   // no bank twice
                            }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(bar_of(C::V_CLEAN + slot, 0));
                    slot = slot + 1 == NS ? 0 : slot + 1;
                }
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax
        const int sw = warp - 2, quad = warp & 3, grp = sw >> 2;
        const int bar = 1 + grp;                             // the column group's four warps
        constexpr int ALL = 7;                               // barrier of all softmax warps
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int kk = quad * 32 + lane;                     // this thread's key of the CTA's half
        const int col0 = grp * GW;                           // its rows
        const int W = p.mask_words, G = p.group;
        const int peer = rank ^ 1;
        const bool speaker = (sw & 3) == 0;                  // the group's warp that talks to the other CTA
        int* s_depth = reinterpret_cast<int*>(smem + C::depth);
        uint32_t* s_cols = reinterpret_cast<uint32_t*>(smem + C::cols);
        float* s_red = reinterpret_cast<float*>(smem + C::red);
        float* s_m = reinterpret_cast<float*>(smem + C::m);
        float2* s_mb = reinterpret_cast<float2*>(smem + C::mb);
        auto mult_of = [&](int r) -> float& { return reinterpret_cast<float*>(s_mb + (r & ~1))[r & 1]; };
        auto less_of = [&](int r) -> float& { return reinterpret_cast<float*>(s_mb + (r & ~1))[2 + (r & 1)]; };
        int* s_low = reinterpret_cast<int*>(smem + C::low);
        uint8_t* s_seen = smem + C::seen;
        bool ok = true;
        int g = 0;                                           // running tile number
        int sbuf = 0, swaps = 0, votes = 0;                  // S^T buffer; column swaps and votes so far
        uint32_t suse = 0;

        // Swaps a value per column (lane) with the same group of the other
        // CTA; the answer comes to every warp of the group.
        auto swap_columns = [&](float v) -> float {
            const int par = swaps & 1;
            const int at = C::top + (par * ROWS + col0 + lane) * 4;
            if (speaker) {
                if (lane == 0) mbar_arrive_expect_tx(&bars[C::TOP + par * GROUPS + grp], 32 * 4);
                __syncwarp();
                st_async_b32(map_to_cta(smem_u32(smem + at), peer), __float_as_uint(v), bar_of(C::TOP + par * GROUPS + grp, peer));
            }
            const bool got = wait_cluster(&bars[C::TOP + par * GROUPS + grp], (swaps >> 1) & 1, p.err, abort);
            ok = __all_sync(0xffffffffu, got) && ok;
            ++swaps;
            return *reinterpret_cast<volatile float*>(smem + at);
        };

        // Brings a segment's Q and tables in: after the S^T tiles of the last
        // segment (its Q has been read by then) and while its last P V runs.
        auto prologue = [&]() {
            const Band& bd = walk.band;
            const int n = walk.n, b = walk.b;
            const int row0 = walk.grp * ROWS;
            bar_sync(ALL, SW * 32);                          // nobody uses the last segment's tables any more
            if (n > 0) {
                if (p.tree_mask) {
                    load_depths(p, b, bd.cnt, s_depth, tid - 64, SW * 32);
                    // a warp per (word, group): lane i brings row i's word, ballots turn it over
#pragma unroll 1
                    for (int u = sw; u < W * GROUPS && 32 * (u / GROUPS) < bd.cnt; u += SW) {
                        const int w = u / GROUPS, gr = u % GROUPS;
                        const int t = (row0 + gr * GW + lane) / G;
                        const uint32_t word = t < bd.cnt && bd.start + t >= 0 ? mask_word(p, b, bd.cnt, t, w) : 0u;
                        uint32_t mine = 0u;
#pragma unroll 4
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t col = __ballot_sync(0xffffffffu, (word >> i) & 1u);
                            mine = lane == i ? col : mine;
                        }
                        s_cols[(32 * w + lane) * GROUPS + gr] = mine;
                    }
                }
                // Q: this CTA's 64 rows as K-major B operand (FP8: the scales of all 128), zeros where there is no row
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (!FP8 && half != rank) continue;
                    constexpr int PER = HALF_ROWS / SW;      // rows of a warp: 4
                    uint4 x[PER][2];
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int row = row0 + half * HALF_ROWS + sw + i * SW, t = row / G;
                        const bool real = t < bd.cnt;
                        const uint4* src = reinterpret_cast<const uint4*>(
                            p.q + ((static_cast<size_t>(b) * p.q_len + (real ? t : 0)) * p.n_q_heads + walk.kvh * G +
                                   (real ? row - t * G : 0)) * D) + 2 * lane;
                        x[i][0] = real ? src[0] : make_uint4(0u, 0u, 0u, 0u);
                        x[i][1] = real ? src[1] : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int r = sw + i * SW;           // line of the operand
                        if constexpr (!FP8) {
                            uint8_t* line = smem + C::q + (lane >> 2) * C::Q_CHUNK + r * 128;
                            const int c = 2 * (lane & 3);
                            *reinterpret_cast<uint4*>(line + ((c ^ (r & 7)) << 4)) = x[i][0];
                            *reinterpret_cast<uint4*>(line + (((c + 1) ^ (r & 7)) << 4)) = x[i][1];
                        } else {
                            const float qs = query_scale(x[i]);
                            if (lane == 0) mult_of(half * HALF_ROWS + r) = p.scale_log2 / qs;
                            if (half != rank) continue;
                            uint4 hi, lo;
                            split_query(x[i], qs, hi, lo);
                            uint8_t* line = smem + C::q + (lane >> 3) * C::Q_CHUNK + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                            *reinterpret_cast<uint4*>(line) = hi;
                            *reinterpret_cast<uint4*>(line + C::Q_TERM) = lo;
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(bar_of(C::Q_FULL, 0));
            }
            bar_sync(ALL, SW * 32);                          // the depths are there
            if (sw < ROWS / 32) {
                const int r = sw * 32 + lane, t = (row0 + r) / G;
                const bool real = t < bd.cnt && bd.start + t >= 0;
                const int place = bd.start + (p.tree_mask && real && n > 0 ? s_depth[t] : t);
                s_low[r] = !real ? INT_MAX : p.window > 0 && place >= INT_MIN + p.window ? place - p.window : INT_MIN;
                s_m[r] = -INFINITY;
                less_of(r) = 0.f;
                if (!FP8) mult_of(r) = p.scale_log2;
            }
            bar_sync(ALL, SW * 32);
        };

        int done = -1;                                       // tiles of the segment whose O is to be read, -1: none
        bool direct = false;                                 // its rows are whole
        for (;;) {
            const bool have = walk.next(p);
            if (have) prologue();
            if (done >= 0) {
                // ---- O of the last segment: this CTA's element of each of the
                // two blocks; the new segment's S^T runs meanwhile
                if (!have) bar_sync(bar, 128);               // what to write is in shared memory
                if (done > 0) ok = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                if (!(ok = bar_and(ALL, SW * 32, ok))) break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int o = 0; o < 4; ++o) {                // (block, half of the group's rows)
                    uint32_t r[16];
                    const int c0 = col0 + (o & 1) * 16;
                    if (done > 0) {
                        tmem_ld16(tmem + lanes + TM_O + static_cast<uint32_t>((o >> 1) * ROWS + c0), r);
                        tmem_ld_wait();
                        if (o == 3) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_remote_relaxed(bar_of(C::O_FREE, 0));
                        }
                    }
                    const int d = (o >> 1) * 256 + rank * 128 + kk;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const uint4 ia = *reinterpret_cast<const uint4*>(smem + C::info + (c0 + i) * 16);
                        const uint4 ib = *reinterpret_cast<const uint4*>(smem + C::info + (c0 + i + 1) * 16);
                        const float fa = __uint_as_float(ia.z), fb = __uint_as_float(ib.z);
                        const float a = fa != 0.f ? __uint_as_float(r[i]) * fa : 0.f;
                        const float b = fb != 0.f ? __uint_as_float(r[i + 1]) * fb : 0.f;
                        if (direct) {
                            // lane pairs trade: the even lane stores both elements of row i, the odd one of row i + 1
                            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
                            const uint4 info = lane & 1 ? ib : ia;
                            const size_t at = (static_cast<size_t>(info.y) << 32 | info.x) * D + (d & ~1);
                            const uint32_t two = lane & 1 ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                            if (info.w) *reinterpret_cast<uint32_t*>(p.out + at) = two;
                        } else {
                            if (ia.w) p.ws_o[(static_cast<size_t>(ia.y) << 32 | ia.x) * D + d] = a;
                            if (ib.w) p.ws_o[(static_cast<size_t>(ib.y) << 32 | ib.x) * D + d] = b;
                        }
                    }
                }
            }
            if (!have) break;
            const Band bd = walk.band;
            const int n = walk.n, first = walk.first;
            const int row0 = walk.grp * ROWS;
            float l[GW];
#pragma unroll
            for (int i = 0; i < GW; ++i) l[i] = 0.f;
            bool fresh = true;                               // some row may not have a reference yet
#pragma unroll 1
            for (int t = 0; t < n; ++t, ++g) {
                const int v0 = (first + t) * TILE, key = bd.key(v0 + rank * HALF_TILE + kk);
                ok = ok && wait_or_abort(&bars[C::S_FULL + sbuf], suse & 1, p.err, abort);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after_sync();
                const uint32_t s_at = tmem + lanes + TM_S + static_cast<uint32_t>(sbuf * ROWS + col0);
                const int s_free = C::S_FREE + sbuf;
                if (++sbuf == NB) {
                    sbuf = 0;
                    ++suse;
                }
                const bool whole = bd.whole(p, v0);
                uint32_t vis = 0xffffffffu;                  // bit i: row col0 + i sees this thread's key
                if (!whole)
                    vis = rows_that_see<GW>(p, bd, key, row0 + col0, s_depth, s_low + col0,
                                            [&](int c) { return s_cols[c * GROUPS + grp]; });
                // Scores of 16 of the group's rows in log2 units (PLAIN) or less
                // the rows' references.  They are read from tensor memory where they
                // are needed, not kept: 32 scores beside the 32 row sums would spill.
                // A reference is one of these scores, rounded as it is here: a
                // product that is not rounded before the reference is taken off
                // would leave half its last place, for a score of 2^32 and more an
                // exponent that overflows.  The vote may take one (FUSED): what it
                // finds below its limit is above it when rounded only where a score's
                // last place is 2 and more, and then by less than that.
                auto scores = [&](int c0, float (&x)[16], auto form) {
                    uint32_t raw[16];
                    tmem_ld16(s_at + static_cast<uint32_t>(c0), raw);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float4 f = *reinterpret_cast<const float4*>(&s_mb[col0 + c0 + i]);
                        const float2 r = make_float2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]));
                        const float2 mult = make_float2(f.x, f.y), less = make_float2(f.z, f.w);
                        float2 z;
                        if constexpr (FP8 && form.value == FUSED) {
                            // beside this kernel's conversions two FMAs are faster than a
                            // packed one (263 -> 257 us), in bf16 slower (268 -> 270)
                            z = make_float2(__fmaf_rn(r.x, mult.x, less.x), __fmaf_rn(r.y, mult.y, less.y));
                        } else {
                            z = ffma2(r, mult, form.value == FUSED ? less : make_float2(0.f, 0.f));
                            if constexpr (form.value == LESS) z = fadd2(z, less);
                        }
                        x[i] = z.x;
                        x[i + 1] = z.y;
                    }
                    if (!whole) {
                        const uint32_t v = vis >> c0;
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = v & (1u << i) ? x[i] : -INFINITY;
                    }
                };
                // ---- the vote, with the other CTA's keys; a segment's first tile
                // sets the references in any case.  Each warp sends its own, and the
                // group's barrier comes after the answers: its four warps have to
                // come to one decision also when the wait runs out in some of them
                // only (a warp that took the branch alone would wait at its barriers
                // for ever).
                bool over = true;
                if (t > 0) {
                    float high = -INFINITY;
#pragma unroll 1
                    for (int c0 = 0; c0 < GW; c0 += 16) {
                        float x[16];
                        scores(c0, x, std::integral_constant<int, FUSED>());
#pragma unroll
                        for (int i = 0; i < 16; ++i) high = fmaxf(high, x[i]);
                    }
                    const bool mine = __any_sync(0xffffffffu, high >= C::THR + C::P_LOG || fresh || !ok);
                    const int par = votes & 1;
                    uint64_t* vb = &bars[C::VOTE + par * GROUPS + grp];
                    const uint32_t sv = smem_u32(smem + C::vote) + (par * GROUPS + grp) * 16;
                    if (lane == 0) {
                        if (speaker) mbar_arrive_expect_tx(vb, 16);
                        st_async_b32(map_to_cta(sv + (sw & 3) * 4, peer), mine ? 1u : 0u, bar_of(C::VOTE + par * GROUPS + grp, peer));
                    }
                    const bool got = wait_cluster(vb, (votes >> 1) & 1, p.err, abort);
                    ok = __all_sync(0xffffffffu, got) && ok;
                    uint32_t a0, a1, a2, a3;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(sv) : "memory");
                    over = bar_or(bar, 128, mine || (a0 | a1 | a2 | a3) != 0u || !ok);
                    ++votes;
                }
                bool pv_waited = g == 0;
                if (over) {
                    if (!(ok = bar_and(bar, 128, ok))) break;
#pragma unroll 1
                    for (int c0 = 0; c0 < GW; c0 += 16) {
                        float x[16];
                        scores(c0, x, std::integral_constant<int, PLAIN>());
                        const float mx = reduce_columns(x, [](float a, float c) { return fmaxf(a, c); });
                        if (lane < 16) s_red[quad * ROWS + col0 + c0 + lane] = mx;
                    }
                    bar_sync(bar, 128);
                    const int cl = col0 + lane;
                    float up = fmaxf(fmaxf(s_red[cl], s_red[ROWS + cl]), fmaxf(s_red[2 * ROWS + cl], s_red[3 * ROWS + cl]));
                    up = fmaxf(up, swap_columns(up));
                    // column `lane`: the highest score so far and the factor that it costs
                    const float m0 = s_m[cl];
                    const float m1 = fmaxf(m0, up);
                    const float a = m0 == m1 || m0 == -INFINITY ? 1.f : fast_exp2(m0 - m1);
                    fresh = __any_sync(0xffffffffu, m1 == -INFINITY);
#pragma unroll
                    for (int i = 0; i < GW; ++i) l[i] *= __shfl_sync(0xffffffffu, a, i);
                    if (t > 0) {
                        // O is at rest once P V of the last tile has completed
                        const bool got = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                        pv_waited = true;
                        tc_fence_after_sync();
                        if (__any_sync(0xffffffffu, a != 1.f)) {
#pragma unroll 1
                            for (int o = 0; o < 4; ++o) {
                                const uint32_t ta = tmem + lanes + TM_O + static_cast<uint32_t>((o >> 1) * ROWS + col0 + (o & 1) * 16);
                                uint32_t r[16];
                                tmem_ld16(ta, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xffffffffu, a, (o & 1) * 16 + i));
                                tmem_st16(ta, r);
                            }
                            tmem_st_wait();
                        }
                    }
                    bar_sync(bar, 128);                      // everyone has read the references
                    if (speaker) {
                        s_m[cl] = m1;
                        less_of(cl) = m1 == -INFINITY ? 0.f : C::P_LOG - m1;
                    }
                    bar_sync(bar, 128);
                }
                // rows 0-63 are CTA 0's operand, 64-127 CTA 1's: this CTA's go
                // into its operand, the other's are staged
                const bool own = (grp >> 1) == rank;
                uint8_t* dst = smem + (own ? C::p + rank * C::HALF_TERM : C::stage) + kk * C::P_LINE;
                const int term = own ? C::P_TERM : C::HALF_TERM;
#pragma unroll
                for (int h = 0; h < GW / 16; ++h) {
                    float x[16];
                    scores(16 * h, x, std::integral_constant<int, LESS>());
                    if (h == GW / 16 - 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote_relaxed(bar_of(s_free, 0));
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = fast_exp2(x[i]);
                        l[16 * h + i] += x[i];
                    }
                    // P's buffers are free, and V of this tile will be read, after P V of the last tile
                    if (h == 0 && !pv_waited) {
                        const bool got = wait_or_abort(&bars[C::PV_DONE], (g - 1) & 1, p.err, abort);
                        ok = __all_sync(0xffffffffu, got) && ok;
                    }
                    if constexpr (FP8) {
                        uint4 w[3];
                        split_weights(x, 1.f, w);
                        const int piece = line_piece<C::P_LINE>(kk, (grp & 1) * (GW / 16) + h);
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            *reinterpret_cast<uint4*>(dst + e * term + piece) = w[e];
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            *reinterpret_cast<uint4*>(dst + line_piece<C::P_LINE>(kk, (grp & 1) * (GW / 8) + 2 * h + c)) =
                                make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                                           pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[C::STAGED]);
                    if (sw == 0) mbar_arrive_expect_tx(&bars[C::P_FULL], C::STAGE_BYTES);
                    else mbar_arrive(&bars[C::P_FULL]);
                }

                // with masks only the rows know whether some row sees a key
                if (p.tree_mask && !whole) {
                    s_seen[grp * HALF_TILE + kk] = vis != 0u;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::SEEN_HERE]);
                }
            }
            // all go on or all stop: no warp may wait at a barrier for one that has left
            if (!(ok = bar_and(ALL, SW * 32, ok))) break;
            // ---- row sums: lanes, the four quadrants' warps, the other CTA
#pragma unroll
            for (int h = 0; h < GW / 16; ++h) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = l[16 * h + i];
                const float part = reduce_columns(v, [](float a, float c) { return a + c; });
                if (lane < 16) s_red[quad * ROWS + col0 + 16 * h + lane] = part;
            }
            bar_sync(bar, 128);
            const int cl = col0 + lane;
            const float mine = (s_red[cl] + s_red[ROWS + cl]) + (s_red[2 * ROWS + cl] + s_red[3 * ROWS + cl]);
            const float other = swap_columns(mine);
            // in one order, so that both CTAs have the same sum
            const float sum = rank == 0 ? mine + other : other + mine;
            // ---- what to write: O / sum where this is the whole row, else the
            // unnormalised partial (zeros for a row that saw nothing)
            direct = walk.count == 1;
            if (speaker) {
                const float top = s_m[cl];
                const int r = row0 + cl, t = r / G;
                const bool some = some_key(s_low[cl], top, sum);
                const size_t row = (static_cast<size_t>(walk.b) * p.q_len + t) * p.n_q_heads + walk.kvh * G + (r - t * G);
                const size_t at = direct ? row : partial_at(p, row, cl, walk.index, blockIdx.x / 2);
                const float factor = !some ? 0.f : direct ? p.o_scale / sum : p.o_scale * (1.f / C::P_SCALE);
                const bool real = t < p.q_len;
                *reinterpret_cast<uint4*>(smem + C::info + cl * 16) =
                    make_uint4(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), __float_as_uint(factor), real);
                if (real && rank == 0) {
                    if (!direct) {
                        p.ws_ml[at * 2] = partial_max(some, top, sum);
                        p.ws_ml[at * 2 + 1] = some ? sum * (1.f / C::P_SCALE) : 0.f;
                    } else if (p.lse) {
                        p.lse[row] = some ? (top + (log2f(sum) - C::P_LOG)) * 0.69314718055994530942f : -INFINITY;
                    }
                }
            }
            if (p.num_splits > 1 && walk.index == 0 && sw == 0 && lane == 0 && rank == 0)
                leave_item(p, walk.entry, walk.kvh, walk.count, walk.stride, blockIdx.x / 2);
            done = n;
        }
    }
    // all threads of both CTAs: no copy or arrival may reach a CTA that has
    // gone.  After a timeout in either CTA a courier's copy may still be on its
    // way with nobody to wait for it: then both stay until P's barrier has
    // counted it, or a millisecond.
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0 && *abort)
        st_cluster_u32(map_to_cta(smem_u32(smem + C::misc + 4), rank ^ 1), 1u);
    __syncwarp();
    cluster_sync_all();
    if (*abort) {
        if (tid == 0) {
            (void)mbar_wait(&bars[C::P_FULL], 0, p.err, 1000000ull);
            (void)mbar_wait(&bars[C::P_FULL], 1, p.err, 1000000ull);
        }
        __syncwarp();
        cluster_sync_all();
    }
    if (warp == 1) tmem_dealloc2(tmem, 512);
}

// Resident pairs on the current device (0: a query failed), asked once per
// device, which also opts the kernel into its shared memory there.
template <bool FP8>
int resident_pairs() {
    static std::mutex mu;
    static int known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev] == 0) {
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = Cfg<FP8>::total + 1024;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(tree_pair_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<FP8>::total + 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, tree_pair_kernel<FP8>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev] = n;
    }
    return known[dev];
}

template <bool FP8>
cudaError_t launch(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    const int resident = resident_pairs<FP8>();
    if (resident < 1) return cudaErrorLaunchOutOfResources;
    const long long units = static_cast<long long>(p.batch) * p.row_groups * p.n_kv_heads *
                            (p.num_splits == 1 ? 1 : p.max_tiles > 1 ? p.max_tiles : 1);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    const int most = resident < p.clusters ? resident : p.clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(units < most ? units : most) * 2);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Cfg<FP8>::total + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_pair_kernel<FP8>, tmk, tmv, p);
}

}  // namespace pairs
}  // namespace tree

cudaError_t launch_tree_pair(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                             cudaStream_t stream) {
    return fp8 ? tree::pairs::launch<true>(tmk, tmv, p, stream) : tree::pairs::launch<false>(tmk, tmv, p, stream);
}

}  // namespace fa512
