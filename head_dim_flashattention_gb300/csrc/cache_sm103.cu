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
#include <stdint.h>
#include <string.h>

#include "fa512_device.cuh"
#include "fa512_internal.h"
#include "fa512_pair.cuh"

namespace fa512 {
namespace cache {

constexpr int D = 512;

// ------------------------------------------------------------------- append
//
// One thread moves 16 stored bytes of a key row and of the value row beside
// it (8 bf16 elements, or 16 elements rounded to E4M3).  blockIdx.y is the
// sequence; the units of its tokens are dealt along blockIdx.x.
constexpr int APPEND_THREADS = 256;

__device__ __forceinline__ uint32_t e4m3x4(const float (&x)[4]) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// 16 bf16 elements -> the 16 E4M3 bytes of x / scale (an IEEE division: the
// nearest fp32 quotient, then the nearest code, ties to even).
__device__ __forceinline__ uint4 quantise16(const uint4 a, const uint4 b, float scale) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x[4] = {__fdiv_rn(__uint_as_float(w[2 * i] << 16), scale),
                            __fdiv_rn(__uint_as_float(w[2 * i] & 0xffff0000u), scale),
                            __fdiv_rn(__uint_as_float(w[2 * i + 1] << 16), scale),
                            __fdiv_rn(__uint_as_float(w[2 * i + 1] & 0xffff0000u), scale)};
        r[i] = e4m3x4(x);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool FP8>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams p) {
    constexpr int UNITS_PER_HEAD = FP8 ? D / 16 : D / 8;
    const int b = blockIdx.y;
    const int units = p.n_kv_heads * UNITS_PER_HEAD;      // per token
    const long long idx = static_cast<long long>(blockIdx.x) * APPEND_THREADS + threadIdx.x;
    const int t = static_cast<int>(idx / units);
    const int u = static_cast<int>(idx - static_cast<long long>(t) * units);
    if (t >= p.q_len) return;
    int n_new = p.q_lens ? p.q_lens[b] : p.q_len;
    if (n_new < 0 || n_new > p.q_len) {
        if (idx == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        n_new = n_new < 0 ? 0 : p.q_len;
    }
    if (t >= n_new) return;
    const long long pos = static_cast<long long>(p.kv_lens[b]) - n_new + t;
    if (pos < 0 || pos >= static_cast<long long>(p.max_pages_per_seq) * p.page_size) {
        if (u == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const int lp = static_cast<int>(pos / p.page_size);
    const int page = p.page_table[static_cast<size_t>(b) * p.max_pages_per_seq + lp];
    if (page < 0 || page >= p.num_pages) {
        if (u == 0) report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return;
    }
    const size_t row = static_cast<size_t>(page) * p.page_size + static_cast<size_t>(pos - static_cast<long long>(lp) * p.page_size);
    const long long ks = b * p.k_batch_stride + t * p.k_token_stride;
    const long long vs = b * p.v_batch_stride + t * p.v_token_stride;
    uint4* kd = static_cast<uint4*>(p.k_pages) + row * units + u;
    uint4* vd = static_cast<uint4*>(p.v_pages) + row * units + u;
    if constexpr (FP8) {
        const uint4* k = reinterpret_cast<const uint4*>(p.k_new + ks) + 2 * u;
        const uint4* v = reinterpret_cast<const uint4*>(p.v_new + vs) + 2 * u;
        const uint4 k0 = k[0], k1 = k[1], v0 = v[0], v1 = v[1];
        *kd = quantise16(k0, k1, p.k_scale);
        *vd = quantise16(v0, v1, p.v_scale);
    } else {
        const uint4 k = reinterpret_cast<const uint4*>(p.k_new + ks)[u];
        const uint4 v = reinterpret_cast<const uint4*>(p.v_new + vs)[u];
        *kd = k;
        *vd = v;
    }
}

// ------------------------------------------------------------------ compact
//
// accepted[i] >= i, rising: a row only ever moves down.  A thread owns one
// 16-byte column of the rows of one sequence, layer and tensor and moves its
// rows in rising order.  The write of row i cannot hit the source of a later
// row (accepted[i'] >= i' > i), and it can only hit a source of an earlier
// row, which this thread has read already; so loading a batch of sources
// ahead and storing afterwards is safe, and no two threads touch one byte.
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
// One cluster of blocks plans the pages: (A) copies the reference counts and
// (fork) finds the first child of every parent, (B) writes the new tables,
// moves the counts by integer atomics (their order does not matter) and scans
// how many fresh pages each sequence needs, (C) counts the free pages of its
// part of the pool, learns the other blocks' counts through distributed
// shared memory, and deals the free pages, lowest first, to the needs in
// order: the page of rank r goes to the sequence whose scan interval holds r.
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_MAX_BATCH = 8192;
constexpr int PLAN_CLUSTER = 8;

struct PlanSmem {
    int off[PLAN_MAX_BATCH + 1];        // fresh pages needed before sequence b
    int first[PLAN_MAX_BATCH];          // fork: first child of each parent
    int warp_sum[PLAN_THREADS / 32];
    int counts[PLAN_CLUSTER];           // free pages of each block's part
};

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
    int w = warp_sum[lane];             // 32 warps
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

// A length clipped to the table, recorded when it was outside.
__device__ __forceinline__ int clip_len(int n, const PagePlanParams& p) {
    const long long cap = static_cast<long long>(p.max_pages_per_seq) * p.page_size;
    if (n < 0 || n > cap) {
        report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return n < 0 ? 0 : static_cast<int>(cap);
    }
    return n;
}

__device__ __forceinline__ int pages_of(int n, int page_size) {
    return static_cast<int>((static_cast<long long>(n) + page_size - 1) / page_size);
}

// The page of a held entry, -1 (recorded) outside the pool.
__device__ __forceinline__ int held_page(const PagePlanParams& p, size_t entry) {
    const int page = p.page_table[entry];
    if (page < 0 || page >= p.num_pages) {
        report_error(p.err, FA512_DEVICE_ERR_INDEX);
        return -1;
    }
    return page;
}

template <bool FORK>
__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(const PagePlanParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) uint8_t raw[];
    PlanSmem& s = *reinterpret_cast<PlanSmem*>(raw);
    const int tid = threadIdx.x;
    const int rank = blockIdx.x, blocks = gridDim.x;     // the grid is one cluster
    const int gtid = rank * PLAN_THREADS + tid, all = blocks * PLAN_THREADS;
    const int width = p.max_pages_per_seq, ps = p.page_size;

    // ---- A
    if (p.new_refs != p.page_refs)
        for (int i = gtid; i < p.num_pages; i += all) p.new_refs[i] = p.page_refs[i];
    if constexpr (FORK) {
        for (int i = tid; i < p.batch; i += PLAN_THREADS) s.first[i] = INT_MAX;
        __syncthreads();
        for (int c = tid; c < p.n_new; c += PLAN_THREADS) {
            const int a = p.parents[c];
            if (a >= 0 && a < p.batch) atomicMin(&s.first[a], c);
        }
    }
    cluster_sync_all();

    // ---- B: needs
    int total = 0;
    for (int b0 = 0; b0 < p.n_new; b0 += PLAN_THREADS) {
        const int b = b0 + tid;
        int need = 0;
        if (b < p.n_new) {
            if constexpr (FORK) {
                const int a = p.parents[b];
                int n = 0;
                if (a >= 0 && a < p.batch) {
                    n = clip_len(p.kv_lens[a], p);
                    need = (n % ps != 0 && s.first[a] != b) ? 1 : 0;
                } else if (rank == 0) {
                    report_error(p.err, FA512_DEVICE_ERR_INDEX);
                }
                if (rank == 0) p.new_lens[b] = n;
            } else {
                need = pages_of(clip_len(p.next_lens[b], p), ps) - pages_of(clip_len(p.kv_lens[b], p), ps);
                need = need > 0 ? need : 0;
            }
        }
        int sum;
        const int before = block_scan(need, s.warp_sum, &sum);
        if (b < p.n_new) s.off[b] = total + before;
        total += sum;
    }
    if (tid == 0) s.off[p.n_new] = total;
    __syncthreads();

    // ---- B: tables and counts
    const long long entries = static_cast<long long>(p.n_new) * width;
    for (long long e = gtid; e < entries; e += all) {
        const int b = static_cast<int>(e / width), i = static_cast<int>(e - static_cast<long long>(b) * width);
        int page = -1;
        if constexpr (FORK) {
            const int a = p.parents[b];
            if (a >= 0 && a < p.batch) {
                const int n = clip_len(p.kv_lens[a], p);
                const bool fresh = s.off[b + 1] > s.off[b] && i == n / ps;
                if (i < pages_of(n, ps) && !fresh) {
                    page = held_page(p, static_cast<size_t>(a) * width + i);
                    if (page >= 0) atomicAdd(&p.new_refs[page], 1);
                }
            }
        } else {
            const bool now = i < pages_of(clip_len(p.kv_lens[b], p), ps);
            const bool then = i < pages_of(clip_len(p.next_lens[b], p), ps);
            if (now) {
                page = held_page(p, static_cast<size_t>(e));
                if (!then) {
                    if (page >= 0) atomicAdd(&p.new_refs[page], -1);
                    page = -1;
                }
            }
        }
        p.new_table[e] = page;
    }
    if constexpr (FORK) {
        const long long old = static_cast<long long>(p.batch) * width;
        for (long long e = gtid; e < old; e += all) {
            const int a = static_cast<int>(e / width), i = static_cast<int>(e - static_cast<long long>(a) * width);
            if (i < pages_of(clip_len(p.kv_lens[a], p), ps)) {
                const int page = held_page(p, static_cast<size_t>(e));
                if (page >= 0) atomicAdd(&p.new_refs[page], -1);
            }
        }
    }
    cluster_sync_all();

    // ---- C: free pages of this block's part
    const int part = (p.num_pages + blocks - 1) / blocks;
    const int lo = min(p.num_pages, rank * part), hi = min(p.num_pages, lo + part);
    int mine = 0;
    for (int i = lo + tid; i < hi; i += PLAN_THREADS) mine += __ldcg(&p.new_refs[i]) == 0;
    int part_free;
    block_scan(mine, s.warp_sum, &part_free);
    if (tid < blocks) pair::st_cluster_u32(map_to_cta(smem_u32(&s.counts[rank]), tid), static_cast<uint32_t>(part_free));
    cluster_sync_all();
    int base = 0, free_pages = 0;
    for (int r = 0; r < blocks; ++r) {
        if (r < rank) base += s.counts[r];
        free_pages += s.counts[r];
    }
    if (total > free_pages && rank == 0 && tid == 0) report_error(p.err, FA512_DEVICE_ERR_PAGES);
    for (int i0 = lo; i0 < hi && base < total; i0 += PLAN_THREADS) {
        const int i = i0 + tid;
        const bool free_here = i < hi && __ldcg(&p.new_refs[i]) == 0;
        int sum;
        const int r = base + block_scan(free_here ? 1 : 0, s.warp_sum, &sum);
        if (free_here && r < total) {
            // the last b with off[b] <= r
            int a = 0, z = p.n_new;
            while (z - a > 1) {
                const int m = (a + z) >> 1;
                if (s.off[m] <= r) a = m; else z = m;
            }
            int entry;
            if constexpr (FORK)
                entry = clip_len(p.kv_lens[p.parents[a]], p) / ps;
            else
                entry = pages_of(clip_len(p.kv_lens[a], p), ps) + (r - s.off[a]);
            p.new_table[static_cast<size_t>(a) * width + entry] = i;
            p.new_refs[i] = 1;
        }
        base += sum;
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

cudaError_t launch_cache_append(const AppendParams& p, bool fp8, cudaStream_t stream) {
    using namespace cache;
    const long long units = static_cast<long long>(p.q_len) * p.n_kv_heads * (fp8 ? D / 16 : D / 8);
    const dim3 grid(static_cast<unsigned>((units + APPEND_THREADS - 1) / APPEND_THREADS), p.batch);
    if (fp8)
        append_kernel<true><<<grid, APPEND_THREADS, 0, stream>>>(p);
    else
        append_kernel<false><<<grid, APPEND_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

int compact_max_accepted() { return cache::COMPACT_MAX; }

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream) {
    using namespace cache;
    const long long units = 2LL * p.n_layers * (p.row_bytes / 16);
    const dim3 grid(static_cast<unsigned>((units + COMPACT_THREADS - 1) / COMPACT_THREADS), p.batch);
    compact_kernel<<<grid, COMPACT_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

int page_plan_max_batch() { return cache::PLAN_MAX_BATCH; }

cudaError_t launch_page_plan(const PagePlanParams& p, bool fork, cudaStream_t stream) {
    using namespace cache;
    auto kernel = fork ? page_plan_kernel<true> : page_plan_kernel<false>;
    const int smem = static_cast<int>(sizeof(PlanSmem));
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(PLAN_CLUSTER);
    cfg.blockDim = dim3(PLAN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PLAN_CLUSTER;
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
