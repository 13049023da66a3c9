// C ABI of the fa512 library: argument validation, TMA tensor-map encoding,
// split-count choice, workspace sizing and kernel launch on the caller's
// stream.  See include/fa512.h for the contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "fa512.h"
#include "fa512_internal.h"

// Device error word: bit 0 = a pipeline wait ran past its bound, bit 1 = a
// page index or kv length outside the declared ranges.  One per device.
__device__ unsigned fa512_device_error_word;

namespace {

constexpr int kHeadDim = FA512_HEAD_DIM;
constexpr unsigned long long kDefaultWaitLimitNs = 2000000000ull;   // the kernels' own default
thread_local char g_last_error[512];

fa512_status fail(fa512_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

fa512_status fail(fa512_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

fa512_status cuda_fail(cudaError_t e, const char* what) {
    return fail(FA512_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---- per-device state: address of the device error word
std::mutex g_mu;
constexpr int kMaxDevices = 64;
unsigned* g_err_ptr[kMaxDevices];

cudaError_t device_error_ptr(unsigned** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_err_ptr[dev]) {
        void* ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, fa512_device_error_word);
        if (e != cudaSuccess) return e;
        g_err_ptr[dev] = static_cast<unsigned*>(ptr);
    }
    *out = g_err_ptr[dev];
    return cudaSuccess;
}

// ---- tensor maps through the driver entry point (no link-time libcuda)
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

fa512_status get_encoder(EncodeTiledFn* fn) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                         cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f)
            return fail(FA512_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
        g_encode = reinterpret_cast<EncodeTiledFn>(f);
    }
    *fn = g_encode;
    return FA512_OK;
}

// Tensor map; dims/strides innermost first, strides in bytes for dims
// 1..rank-1.
fa512_status encode_map(CUtensorMap* m, CUtensorMapDataType dtype, CUtensorMapSwizzle swizzle,
                        const void* base, int rank, const uint64_t* dims,
                        const uint64_t* strides_bytes, const uint32_t* box) {
    EncodeTiledFn enc;
    fa512_status st = get_encoder(&enc);
    if (st != FA512_OK) return st;
    cuuint64_t gd[5], gs[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        gd[i] = dims[i];
        bx[i] = box[i];
        es[i] = 1;
    }
    for (int i = 0; i < rank - 1; ++i) gs[i] = strides_bytes[i];
    CUresult r = enc(m, dtype, static_cast<cuuint32_t>(rank),
                     const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FA512_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return FA512_OK;
}

// bf16 tensor map with 128-byte swizzle.
fa512_status encode_bf16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                         const uint64_t* strides_bytes, const uint32_t* box) {
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, rank,
                      dims, strides_bytes, box);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 152;
    }
    return n;
}

bool pow2_page(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

// Tiles of the decode band (upper bound over sequences) for a host-side bound
// on the kv length.  A window can straddle one extra tile boundary.
long long band_tiles(int max_kv_len, int window) {
    const int tk = fa512::decode_tile_positions();
    long long band = max_kv_len;
    if (window > 0 && window < band) band = window;
    long long t = (band + tk - 1) / tk;
    if (window > 0 && window < max_kv_len) t += 1;
    return t;
}

// Split count for `items` (sequence, KV head) pairs of `tiles` key tiles,
// one 16-warp split CTA per SM.
int choose_splits(long long items, long long tiles, int n_sm) {
    if (items <= 0 || tiles <= 1) return 1;
    long long best_s = 1;
    double best = 1e300;
    const long long s_max = tiles < 1024 ? tiles : 1024;
    for (long long s = 1; s <= s_max; ++s) {
        const long long waves = (items * s + n_sm - 1) / n_sm;
        const long long per = (tiles + s - 1) / s;
        // time model: waves x (tiles per split + fixed cost of ~2 tiles)
        const double cost = static_cast<double>(waves) * static_cast<double>(per + 2);
        if (cost < best) {
            best = cost;
            best_s = s;
        }
    }
    return static_cast<int>(best_s);
}

// Split count for the FP8 kernel, four CTAs per SM, one split each, `rows`
// (sequence, token, query head) rows to merge.  Times in tile times of one
// CTA.  Large batches (the merge takes whole rows): a finished CTA's slot
// takes the next split at once, so the work spreads over the slots in
// fractions of a round rather than whole waves:
//   max(1, items x s / slots) x (tiles per split + 2)   streaming + start
//   + 0.75 x tiles per split                             the ragged end
//   + 0.2 x max(0, s - 32)                               merge loads past the
//                                                        merge kernel's first 32
// Small batches (every CTA resident at once, the merge in column slices):
// an SM's time is its CTAs x tiles per split, and one CTA alone runs no
// faster than two sharing the SM (it is latency-bound), so
//   max(2, CTAs on the busiest SM) x tiles per split.
// Both fitted to times of batch 1/16/64 x KV 4096/16384/28672, 4 KV heads,
// over 8 split counts each: within 0.5 % of the best count per shape.
int choose_splits_fp8(long long items, long long tiles, int n_sm, long long rows) {
    if (items <= 0 || tiles <= 1) return 1;
    const bool small = fa512::decode_merge_sliced(rows);
    const double slots = static_cast<double>(fa512::decode_fp8_ctas_per_sm()) * n_sm;
    long long best_s = 1;
    double best = 1e300;
    const long long s_max = tiles < 128 ? tiles : 128;
    for (long long s = 1; s <= s_max; ++s) {
        const double per = static_cast<double>((tiles + s - 1) / s);
        double cost;
        if (small) {
            const long long busiest = (items * s + n_sm - 1) / n_sm;
            cost = static_cast<double>(busiest > 2 ? busiest : 2) * per;
        } else {
            const double x = static_cast<double>(items * s) / slots;
            cost = (x > 1.0 ? x : 1.0) * (per + 2.0) + 0.75 * per +
                   0.2 * static_cast<double>(s > 32 ? s - 32 : 0);
        }
        if (cost < best) {
            best = cost;
            best_s = s;
        }
    }
    return static_cast<int>(best_s);
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t workspace_for(int batch, int n_q_heads, int splits) {
    const size_t rows = static_cast<size_t>(batch) * n_q_heads * splits;
    return round256(rows * kHeadDim * sizeof(float)) + round256(rows * 2 * sizeof(float));
}

}  // namespace

void fa512::set_last_error_message(const char* msg) {
    snprintf(g_last_error, sizeof g_last_error, "%s", msg ? msg : "");
}

extern "C" {

const char* fa512_status_string(fa512_status s) {
    switch (s) {
        case FA512_OK: return "FA512_OK";
        case FA512_ERR_INVALID_ARG: return "FA512_ERR_INVALID_ARG";
        case FA512_ERR_UNSUPPORTED: return "FA512_ERR_UNSUPPORTED";
        case FA512_ERR_CUDA: return "FA512_ERR_CUDA";
        case FA512_ERR_TIMEOUT: return "FA512_ERR_TIMEOUT";
        case FA512_ERR_WORKSPACE: return "FA512_ERR_WORKSPACE";
        case FA512_ERR_DEVICE_INDEX: return "FA512_ERR_DEVICE_INDEX";
        case FA512_ERR_OUT_OF_PAGES: return "FA512_ERR_OUT_OF_PAGES";
    }
    return "FA512_UNKNOWN_STATUS";
}

const char* fa512_last_error_message(void) { return g_last_error; }

}  // extern "C"

namespace {

// Body of fa512_prefill; the test hook below reaches it with a short wait
// bound and one K load left out.
fa512_status prefill_call(const void* q, const void* k, const void* v, void* out, float* lse,
                          int seqlen_q, int seqlen_k, int q_offset, int n_q_heads, int n_kv_heads,
                          float scale, int causal, int window, fa512_stream_t stream,
                          unsigned long long wait_limit_ns, int skip_first_k_load) {
    g_last_error[0] = 0;
    if (seqlen_q < 0 || seqlen_k < 0 || q_offset < 0)
        return fail(FA512_ERR_INVALID_ARG, "negative length or offset");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(FA512_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)",
                    n_q_heads, n_kv_heads);
    const int G = n_q_heads / n_kv_heads;
    if (G > 128) return fail(FA512_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (!(scale == scale) || isinf(scale)) return fail(FA512_ERR_INVALID_ARG, "scale is not finite");
    if (static_cast<long long>(q_offset) + seqlen_q > 0x7fffffffLL)
        return fail(FA512_ERR_INVALID_ARG, "q_offset + seqlen_q overflows int32 positions");
    if (seqlen_q == 0) return FA512_OK;
    if (!q || !out || (seqlen_k > 0 && (!k || !v)))
        return fail(FA512_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(q) || !aligned16(out) || (seqlen_k > 0 && (!aligned16(k) || !aligned16(v))))
        return fail(FA512_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA512_ERR_INVALID_ARG, "lse must be 4-byte aligned");

    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");

    fa512::PrefillParams p;
    memset(&p, 0, sizeof p);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.seqlen_q = seqlen_q;
    p.total_q = seqlen_q;
    p.seqlen_k = seqlen_k;
    p.q_offset = q_offset;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.tokens_per_tile = 128 / G;
    p.rows_per_tile = p.tokens_per_tile * G;
    p.num_q_tiles = (seqlen_q + p.tokens_per_tile - 1) / p.tokens_per_tile;
    p.causal = causal ? 1 : 0;
    p.window = window > 0 ? window : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    p.wait_limit_ns = wait_limit_ns;
    p.test_skip_first_k_load = skip_first_k_load;
    if (static_cast<long long>(p.num_q_tiles) * n_kv_heads * 2 > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "grid too large");

    CUtensorMap tmq, tmk, tmv;
    memset(&tmk, 0, sizeof tmk);
    memset(&tmv, 0, sizeof tmv);
    {
        const uint64_t dims[4] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(G),
                                  static_cast<uint64_t>(n_kv_heads), static_cast<uint64_t>(seqlen_q)};
        const uint64_t strides[3] = {kHeadDim * 2ull, static_cast<uint64_t>(G) * kHeadDim * 2ull,
                                     static_cast<uint64_t>(n_q_heads) * kHeadDim * 2ull};
        const uint32_t box[4] = {64u, static_cast<uint32_t>(G), 1u,
                                 static_cast<uint32_t>(p.tokens_per_tile)};
        fa512_status st = encode_bf16(&tmq, q, 4, dims, strides, box);
        if (st != FA512_OK) return st;
    }
    if (seqlen_k > 0) {
        const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(n_kv_heads),
                                  static_cast<uint64_t>(seqlen_k)};
        const uint64_t strides[2] = {kHeadDim * 2ull, static_cast<uint64_t>(n_kv_heads) * kHeadDim * 2ull};
        // the kernel streams K in head-dim chunks of a whole key tile and V
        // in key slices; it states the box height of each
        const uint32_t kbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill_k_box_rows())};
        const uint32_t vbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill_v_box_rows())};
        fa512_status st = encode_bf16(&tmk, k, 3, dims, strides, kbox);
        if (st != FA512_OK) return st;
        st = encode_bf16(&tmv, v, 3, dims, strides, vbox);
        if (st != FA512_OK) return st;
    }
    e = fa512::launch_prefill(tmq, tmk, tmv, p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    return FA512_OK;
}

}  // namespace

extern "C" {

fa512_status fa512_prefill(const void* q, const void* k, const void* v, void* out, float* lse,
                           int seqlen_q, int seqlen_k, int q_offset, int n_q_heads,
                           int n_kv_heads, float scale, int causal, int window,
                           fa512_stream_t stream) {
    return prefill_call(q, k, v, out, lse, seqlen_q, seqlen_k, q_offset, n_q_heads, n_kv_heads,
                        scale, causal, window, stream, kDefaultWaitLimitNs, 0);
}

fa512_status fa512_test_prefill_missing_load(const void* q, const void* k, const void* v, void* out,
                                             float* lse, int seqlen_q, int seqlen_k, int q_offset,
                                             int n_q_heads, int n_kv_heads, float scale, int causal,
                                             int window, uint64_t wait_limit_ns,
                                             fa512_stream_t stream) {
    if (wait_limit_ns < 1000000ull || wait_limit_ns > kDefaultWaitLimitNs)
        return fail(FA512_ERR_INVALID_ARG, "wait_limit_ns must lie in [1 ms, 2 s]");
    if (seqlen_k < 1) return fail(FA512_ERR_INVALID_ARG, "the hook needs at least one key");
    return prefill_call(q, k, v, out, lse, seqlen_q, seqlen_k, q_offset, n_q_heads, n_kv_heads,
                        scale, causal, window, stream, wait_limit_ns, 1);
}

fa512_status fa512_prefill_d256(const void* q, const void* k, const void* v, void* out, float* lse,
                                int seqlen_q, int seqlen_k, int q_offset, int n_q_heads,
                                int n_kv_heads, float scale, int causal, int window,
                                fa512_stream_t stream) {
    g_last_error[0] = 0;
    constexpr int kD = 256;
    if (seqlen_q < 0 || seqlen_k < 0 || q_offset < 0)
        return fail(FA512_ERR_INVALID_ARG, "negative length or offset");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(FA512_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)",
                    n_q_heads, n_kv_heads);
    const int G = n_q_heads / n_kv_heads;
    if (G > 128) return fail(FA512_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (!(scale == scale) || isinf(scale)) return fail(FA512_ERR_INVALID_ARG, "scale is not finite");
    if (static_cast<long long>(q_offset) + seqlen_q > 0x7fffffffLL)
        return fail(FA512_ERR_INVALID_ARG, "q_offset + seqlen_q overflows int32 positions");
    if (seqlen_q == 0) return FA512_OK;
    if (!q || !out || (seqlen_k > 0 && (!k || !v)))
        return fail(FA512_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(q) || !aligned16(out) || (seqlen_k > 0 && (!aligned16(k) || !aligned16(v))))
        return fail(FA512_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA512_ERR_INVALID_ARG, "lse must be 4-byte aligned");

    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");

    fa512::Prefill256Params p;
    memset(&p, 0, sizeof p);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.seqlen_q = seqlen_q;
    p.seqlen_k = seqlen_k;
    p.q_offset = q_offset;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.tokens_per_tile = 128 / G;
    p.rows_per_tile = p.tokens_per_tile * G;
    p.num_q_tiles = (seqlen_q + p.tokens_per_tile - 1) / p.tokens_per_tile;
    p.n_pairs = (p.num_q_tiles + 1) / 2;
    if (static_cast<long long>(p.n_pairs) * n_kv_heads > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "too many work items");
    p.n_items = p.n_pairs * n_kv_heads;
    p.causal = causal ? 1 : 0;
    p.window = window > 0 ? window : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    fa512::plan_prefill256(p, sm_count());

    CUtensorMap tmq, tmk, tmv, tmo;
    memset(&tmk, 0, sizeof tmk);
    memset(&tmv, 0, sizeof tmv);
    {
        const uint64_t dims[4] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(G),
                                  static_cast<uint64_t>(n_kv_heads), static_cast<uint64_t>(seqlen_q)};
        const uint64_t strides[3] = {kD * 2ull, static_cast<uint64_t>(G) * kD * 2ull,
                                     static_cast<uint64_t>(n_q_heads) * kD * 2ull};
        const uint32_t box[4] = {64u, static_cast<uint32_t>(G), 1u,
                                 static_cast<uint32_t>(p.tokens_per_tile)};
        fa512_status st = encode_bf16(&tmq, q, 4, dims, strides, box);
        if (st != FA512_OK) return st;
        // O leaves through the same box shape (a staged tile per TMA store)
        st = encode_bf16(&tmo, out, 4, dims, strides, box);
        if (st != FA512_OK) return st;
    }
    if (seqlen_k > 0) {
        const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(n_kv_heads),
                                  static_cast<uint64_t>(seqlen_k)};
        const uint64_t strides[2] = {kD * 2ull, static_cast<uint64_t>(n_kv_heads) * kD * 2ull};
        // K in {64 columns, 48 keys} boxes (each CTA of a pair holds half a
        // 96-key tile), V in {64 columns, 96 keys} boxes
        const uint32_t kbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill256_k_box_rows())};
        const uint32_t vbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill256_v_box_rows())};
        fa512_status st = encode_bf16(&tmk, k, 3, dims, strides, kbox);
        if (st != FA512_OK) return st;
        st = encode_bf16(&tmv, v, 3, dims, strides, vbox);
        if (st != FA512_OK) return st;
    }
    e = fa512::launch_prefill256(tmq, tmk, tmv, tmo, p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "head-dim-256 prefill launch");
    return FA512_OK;
}

fa512_status fa512_prefill_paged(const void* q, const void* k_pages, const void* v_pages,
                                 const int32_t* page_table, const int32_t* cu_seqlens_q,
                                 const int32_t* seqused_k, void* out, float* lse, int batch,
                                 int total_q, int max_seqlen_q, int n_q_heads, int n_kv_heads,
                                 int page_size, int num_pages, int max_pages_per_seq, float scale,
                                 int causal, int window, fa512_stream_t stream) {
    g_last_error[0] = 0;
    if (batch < 0 || total_q < 0 || max_seqlen_q < 0)
        return fail(FA512_ERR_INVALID_ARG, "negative batch, total_q or max_seqlen_q");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(FA512_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)",
                    n_q_heads, n_kv_heads);
    const int G = n_q_heads / n_kv_heads;
    if (G > 128) return fail(FA512_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (page_size != 64 && page_size != 128 && page_size != 256)
        return fail(FA512_ERR_UNSUPPORTED, "prefill over a paged cache needs page_size 64, 128 or 256");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(FA512_ERR_INVALID_ARG, "num_pages and max_pages_per_seq must be >= 1");
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL - 256 ||
        static_cast<long long>(max_pages_per_seq) * page_size > 0x7fffffffLL - 256)
        return fail(FA512_ERR_UNSUPPORTED, "page pool or page table too large for int32 key rows");
    if (!(scale == scale) || isinf(scale)) return fail(FA512_ERR_INVALID_ARG, "scale is not finite");
    if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return FA512_OK;
    if (!q || !out || !k_pages || !v_pages || !page_table || !cu_seqlens_q || !seqused_k)
        return fail(FA512_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_pages) || !aligned16(v_pages))
        return fail(FA512_ERR_INVALID_ARG, "q, k_pages, v_pages and out must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(cu_seqlens_q) |
         reinterpret_cast<uintptr_t>(seqused_k)) & 3u)
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u))
        return fail(FA512_ERR_INVALID_ARG, "lse must be 4-byte aligned");

    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");

    fa512::PrefillParams p;
    memset(&p, 0, sizeof p);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.total_q = total_q;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.tokens_per_tile = 128 / G;
    p.rows_per_tile = p.tokens_per_tile * G;
    p.causal = causal ? 1 : 0;
    p.window = window > 0 ? window : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    p.page_table = page_table;
    p.cu_seqlens_q = cu_seqlens_q;
    p.seqused_k = seqused_k;
    p.batch = batch;
    p.max_seqlen_q = max_seqlen_q;
    const long long tiles = (static_cast<long long>(max_seqlen_q) + p.tokens_per_tile - 1) / p.tokens_per_tile;
    p.max_pairs = static_cast<int>((tiles + 1) / 2);
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    p.page_shift = shift;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.oob_row = num_pages * page_size;
    if (static_cast<long long>(batch) * n_kv_heads * p.max_pairs * 4 > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "grid too large");

    CUtensorMap tmq, tmk, tmv;
    {
        const uint64_t dims[4] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(G),
                                  static_cast<uint64_t>(n_kv_heads), static_cast<uint64_t>(total_q)};
        const uint64_t strides[3] = {kHeadDim * 2ull, static_cast<uint64_t>(G) * kHeadDim * 2ull,
                                     static_cast<uint64_t>(n_q_heads) * kHeadDim * 2ull};
        const uint32_t box[4] = {64u, static_cast<uint32_t>(G), 1u,
                                 static_cast<uint32_t>(p.tokens_per_tile)};
        fa512_status st = encode_bf16(&tmq, q, 4, dims, strides, box);
        if (st != FA512_OK) return st;
    }
    {
        // the pool as rows of keys: [num_pages * page_size, n_kv_heads, 512]
        const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(n_kv_heads),
                                  static_cast<uint64_t>(num_pages) * page_size};
        const uint64_t strides[2] = {kHeadDim * 2ull, static_cast<uint64_t>(n_kv_heads) * kHeadDim * 2ull};
        const uint32_t kbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill_k_box_rows())};
        const uint32_t vbox[3] = {64u, 1u, static_cast<uint32_t>(fa512::prefill_paged_v_box_rows())};
        fa512_status st = encode_bf16(&tmk, k_pages, 3, dims, strides, kbox);
        if (st != FA512_OK) return st;
        st = encode_bf16(&tmv, v_pages, 3, dims, strides, vbox);
        if (st != FA512_OK) return st;
    }
    e = fa512::launch_prefill_paged(tmq, tmk, tmv, p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged prefill launch");
    return FA512_OK;
}

int fa512_decode_auto_splits(int batch, int n_kv_heads, int page_size, int max_kv_len) {
    (void)page_size;
    if (batch <= 0 || n_kv_heads <= 0 || max_kv_len <= 0) return 1;
    return choose_splits(static_cast<long long>(batch) * n_kv_heads, band_tiles(max_kv_len, 0),
                         sm_count());
}

int fa512_decode_auto_splits_fp8(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                 int page_size, int max_kv_len) {
    if (batch <= 0 || q_len < 1 || n_kv_heads <= 0 || n_q_heads <= 0 || max_kv_len <= 0) return 1;
    if (q_len * (n_q_heads / n_kv_heads) > fa512::decode_fp8_mma_rows())
        return fa512_decode_auto_splits(batch, n_kv_heads, page_size, max_kv_len);
    return choose_splits_fp8(static_cast<long long>(batch) * n_kv_heads, band_tiles(max_kv_len, 0),
                             sm_count(), static_cast<long long>(batch) * q_len * n_q_heads);
}

size_t fa512_decode_workspace_bytes_fp8(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                        int page_size, int max_kv_len, int num_splits) {
    if (batch < 0 || q_len < 1 || n_q_heads <= 0 || n_kv_heads <= 0 || max_kv_len < 0 ||
        num_splits < 0 || num_splits > 1024)
        return 0;
    const int s = num_splits > 0 ? num_splits
                                 : fa512_decode_auto_splits_fp8(batch, q_len, n_q_heads, n_kv_heads,
                                                                page_size, max_kv_len);
    return workspace_for(batch * q_len, n_q_heads, s);
}

size_t fa512_decode_workspace_bytes_q(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                      int page_size, int max_kv_len, int num_splits) {
    if (batch < 0 || q_len < 1 || n_q_heads <= 0 || n_kv_heads <= 0 || max_kv_len < 0 ||
        num_splits < 0 || num_splits > 1024)
        return 0;
    const int s = num_splits > 0 ? num_splits
                                 : fa512_decode_auto_splits(batch, n_kv_heads, page_size, max_kv_len);
    return workspace_for(batch * q_len, n_q_heads, s);
}

size_t fa512_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int page_size,
                                    int max_kv_len, int num_splits) {
    return fa512_decode_workspace_bytes_q(batch, 1, n_q_heads, n_kv_heads, page_size, max_kv_len,
                                          num_splits);
}

}  // extern "C"

namespace {

// Body of the decode entry points.  fp8: k_pages / v_pages hold e4m3 bytes
// and a key (value) element is k_scale (v_scale) times its e4m3 value.
fa512_status decode_call(const void* q, const void* k_pages, const void* v_pages,
                         const int32_t* page_table, const int32_t* kv_lens, void* out, float* lse,
                         int batch, int q_len, int n_q_heads, int n_kv_heads, int page_size,
                         int num_pages, int max_pages_per_seq, int max_kv_len, float scale,
                         int window, int num_splits, void* workspace, size_t workspace_bytes,
                         bool fp8, float k_scale, float v_scale, fa512_stream_t stream) {
    g_last_error[0] = 0;
    if (batch < 0) return fail(FA512_ERR_INVALID_ARG, "negative batch");
    if (q_len < 1) return fail(FA512_ERR_INVALID_ARG, "q_len must be >= 1");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(FA512_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)",
                    n_q_heads, n_kv_heads);
    const int G = n_q_heads / n_kv_heads;
    if (G > 16) return fail(FA512_ERR_UNSUPPORTED, "decode supports at most 16 query heads per KV head");
    if (q_len * G > 16)
        return fail(FA512_ERR_UNSUPPORTED, "q_len x query heads per KV head (%d x %d) must be at most 16",
                    q_len, G);
    if (!pow2_page(page_size)) return fail(FA512_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(FA512_ERR_INVALID_ARG, "num_pages and max_pages_per_seq must be >= 1");
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "page pool larger than 2^31 rows");
    if (max_kv_len < 0 || static_cast<long long>(max_kv_len) > static_cast<long long>(max_pages_per_seq) * page_size)
        return fail(FA512_ERR_INVALID_ARG, "max_kv_len outside [0, max_pages_per_seq * page_size]");
    if (num_splits < 0 || num_splits > 1024) return fail(FA512_ERR_INVALID_ARG, "num_splits outside [0, 1024]");
    if (!(scale == scale) || isinf(scale)) return fail(FA512_ERR_INVALID_ARG, "scale is not finite");
    if (fp8 && (!(k_scale == k_scale) || isinf(k_scale) || !(v_scale == v_scale) || isinf(v_scale)))
        return fail(FA512_ERR_INVALID_ARG, "k_scale and v_scale must be finite");
    if (batch == 0) return FA512_OK;
    if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !out)
        return fail(FA512_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return fail(FA512_ERR_INVALID_ARG, "q, pages and out must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(page_table) & 3u) || (reinterpret_cast<uintptr_t>(kv_lens) & 3u) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
        return fail(FA512_ERR_INVALID_ARG, "page_table, kv_lens and lse must be 4-byte aligned");

    const int splits = num_splits > 0 ? num_splits
                       : fp8 ? fa512_decode_auto_splits_fp8(batch, q_len, n_q_heads, n_kv_heads,
                                                            page_size, max_kv_len)
                             : fa512_decode_auto_splits(batch, n_kv_heads, page_size, max_kv_len);
    const size_t need = workspace_for(batch * q_len, n_q_heads, splits);
    if (!workspace || workspace_bytes < need)
        return fail(FA512_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(FA512_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (static_cast<long long>(batch) * n_kv_heads > 65535LL * 65535LL)
        return fail(FA512_ERR_UNSUPPORTED, "grid too large");
    if (batch > 65535 || n_kv_heads > 65535) return fail(FA512_ERR_UNSUPPORTED, "grid too large");

    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");

    fa512::DecodeParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16*>(q);
    if (fp8) {
        p.k8 = static_cast<const uint8_t*>(k_pages);
        p.v8 = static_cast<const uint8_t*>(v_pages);
        p.o_scale = v_scale;
    } else {
        p.k_pages = static_cast<const __nv_bfloat16*>(k_pages);
        p.v_pages = static_cast<const __nv_bfloat16*>(v_pages);
        p.o_scale = 1.f;
    }
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    const size_t rows = static_cast<size_t>(batch) * q_len * n_q_heads * splits;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256(rows * kHeadDim * sizeof(float)));
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.batch = batch;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.q_len = q_len;
    p.page_size = page_size;
    p.box_rows = page_size < 32 ? page_size : 32;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.len_cap = max_kv_len;
    p.window = window > 0 ? window : 0;
    const long long tiles = band_tiles(max_kv_len, p.window);
    p.num_splits = splits;
    p.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
    if (p.tiles_per_split < 1) p.tiles_per_split = 1;
    p.scale_log2 = scale * 1.4426950408889634f;
    // FP8: k_scale scales every score; applied after the bf16 path's factor
    // so that a power-of-two k_scale changes no rounding
    if (fp8) p.scale_log2 *= k_scale;
    p.err = err;

    CUtensorMap tmk, tmv;
    const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(n_kv_heads),
                              static_cast<uint64_t>(num_pages) * page_size};
    fa512_status st;
    if (fp8) {
        // e4m3 bytes: 256-byte boxes, no swizzle (the kernel converts them to
        // the swizzled bf16 tile itself)
        const uint64_t strides[2] = {static_cast<uint64_t>(kHeadDim),
                                     static_cast<uint64_t>(n_kv_heads) * kHeadDim};
        const uint32_t box[3] = {static_cast<uint32_t>(fa512::decode_fp8_box_bytes()), 1u,
                                 static_cast<uint32_t>(p.box_rows)};
        st = encode_map(&tmk, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, k_pages, 3,
                        dims, strides, box);
        if (st != FA512_OK) return st;
        st = encode_map(&tmv, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, v_pages, 3,
                        dims, strides, box);
        if (st != FA512_OK) return st;
        e = fa512::launch_decode_fp8(tmk, tmv, p, reinterpret_cast<cudaStream_t>(stream));
    } else {
        const uint64_t strides[2] = {kHeadDim * 2ull, static_cast<uint64_t>(n_kv_heads) * kHeadDim * 2ull};
        const uint32_t box[3] = {64u, 1u, static_cast<uint32_t>(p.box_rows)};
        st = encode_bf16(&tmk, k_pages, 3, dims, strides, box);
        if (st != FA512_OK) return st;
        st = encode_bf16(&tmv, v_pages, 3, dims, strides, box);
        if (st != FA512_OK) return st;
        e = fa512::launch_decode(tmk, tmv, p, reinterpret_cast<cudaStream_t>(stream));
    }
    if (e != cudaSuccess) return cuda_fail(e, "decode launch");
    return FA512_OK;
}

}  // namespace

extern "C" {

fa512_status fa512_decode_paged_q(const void* q, const void* k_pages, const void* v_pages,
                                  const int32_t* page_table, const int32_t* kv_lens, void* out,
                                  float* lse, int batch, int q_len, int n_q_heads, int n_kv_heads,
                                  int page_size, int num_pages, int max_pages_per_seq,
                                  int max_kv_len, float scale, int window, int num_splits,
                                  void* workspace, size_t workspace_bytes,
                                  fa512_stream_t stream) {
    return decode_call(q, k_pages, v_pages, page_table, kv_lens, out, lse, batch, q_len, n_q_heads,
                       n_kv_heads, page_size, num_pages, max_pages_per_seq, max_kv_len, scale,
                       window, num_splits, workspace, workspace_bytes, false, 1.f, 1.f, stream);
}

fa512_status fa512_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* page_table, const int32_t* kv_lens, void* out,
                                    float* lse, int batch, int q_len, int n_q_heads,
                                    int n_kv_heads, int page_size, int num_pages,
                                    int max_pages_per_seq, int max_kv_len, float scale,
                                    float k_scale, float v_scale, int window, int num_splits,
                                    void* workspace, size_t workspace_bytes,
                                    fa512_stream_t stream) {
    return decode_call(q, k_pages, v_pages, page_table, kv_lens, out, lse, batch, q_len, n_q_heads,
                       n_kv_heads, page_size, num_pages, max_pages_per_seq, max_kv_len, scale,
                       window, num_splits, workspace, workspace_bytes, true, k_scale, v_scale,
                       stream);
}

fa512_status fa512_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                const int32_t* page_table, const int32_t* kv_lens, void* out,
                                float* lse, int batch, int n_q_heads, int n_kv_heads,
                                int page_size, int num_pages, int max_pages_per_seq,
                                int max_kv_len, float scale, int window, int num_splits,
                                void* workspace, size_t workspace_bytes,
                                fa512_stream_t stream) {
    return fa512_decode_paged_q(q, k_pages, v_pages, page_table, kv_lens, out, lse, batch, 1,
                                n_q_heads, n_kv_heads, page_size, num_pages, max_pages_per_seq,
                                max_kv_len, scale, window, num_splits, workspace, workspace_bytes,
                                stream);
}

fa512_status fa512_device_status(fa512_stream_t stream, int clear) {
    g_last_error[0] = 0;
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
    unsigned word = 0;
    e = cudaMemcpyFromSymbol(&word, fa512_device_error_word, sizeof word);
    if (e != cudaSuccess) return cuda_fail(e, "read device error word");
    if (clear && word) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(fa512_device_error_word, &zero, sizeof zero);
        if (e != cudaSuccess) return cuda_fail(e, "clear device error word");
    }
    if (word & 1u) return fail(FA512_ERR_TIMEOUT, "a kernel pipeline wait exceeded its bound");
    if (word & 2u) return fail(FA512_ERR_DEVICE_INDEX, "a page index or kv length was out of range");
    if (word & 8u) return fail(FA512_ERR_OUT_OF_PAGES, "more pages were asked for than are free");
    if (word & 4u) return fail(FA512_ERR_UNSUPPORTED, "the dynamic shared-memory window was not 1 KiB aligned");
    return FA512_OK;
}

}  // extern "C"

namespace {

// ------------------------------------------- drafted tokens, cache management

// Most key tiles that a row group of a tree call walks: with a window the
// sinks, the window and the places its rows span, both rounded to boxes of
// `box` positions.
long long tree_tiles(int q_len, int group, int max_kv_len, int window, int n_sinks, int box) {
    const fa512::TreeShape s = fa512::tree_shape(q_len, group);
    const int tile = s.tile;
    const long long all = (static_cast<long long>(max_kv_len) + tile - 1) / tile;
    if (window <= 0) return all;
    // a run's rows span their own tokens; a masked tree's all of its tokens
    const long long span = static_cast<long long>(s.rows) / group + 2;
    const long long tokens = q_len <= fa512::tree_max_nodes() || q_len < span ? q_len : span;
    const long long sinks = (static_cast<long long>(n_sinks) + box - 1) / box * box;
    const long long some = (sinks + window + tokens + box - 1 + tile - 1) / tile;
    return some < all ? some : all;
}

// Whether that many tiles are walked in one piece: a merge costs about 4 us, a
// tile of 128 keys 2 to 3.5 (24 runs of 2 tokens over 164 positions: 20.1 us in
// two pieces, 18.5 in one; with three tiles as many shapes lose as gain).
bool one_piece(const fa512::TreeShape& s, long long tiles) { return tiles <= (s.ctas == 1 ? 2 : 1); }

// Partials of a call with `splits` > 1, in rows: a place for each row and
// segment, or, where that is above 64 MB, two slots a cluster (40 MB at most; 8
// sequences of 4,096 tokens and 32 heads would take 6.5 GB).  Small calls would
// pay for the slots' arithmetic in the merge (47 sequences of 2 tokens 43.2 us
// without them, 43.5 with).
struct TreePartials {
    size_t rows;
    int slot_rows;                  // see TreeParams
    int clusters;
    size_t bytes() const { return round256(rows * kHeadDim * sizeof(float)) + round256(rows * 2 * sizeof(float)); }
};
TreePartials tree_partials(long long batch, int q_len, int n_q_heads, int n_kv_heads, int splits) {
    const fa512::TreeShape s = fa512::tree_shape(q_len, n_q_heads / n_kv_heads);
    const long long in_group = static_cast<long long>(q_len) * (n_q_heads / n_kv_heads);
    TreePartials w;
    w.clusters = sm_count() / s.ctas > 0 ? sm_count() / s.ctas : 1;
    w.rows = static_cast<size_t>(batch) * q_len * n_q_heads * splits;
    w.slot_rows = static_cast<int>(in_group < s.rows ? in_group : s.rows);
    const size_t slots = 2 * static_cast<size_t>(w.clusters) * w.slot_rows;
    if (w.rows * (kHeadDim + 2) * sizeof(float) > (64u << 20) && slots < w.rows) w.rows = slots;
    else w.slot_rows = 0;
    return w;
}

// The partials, and what says where an item's are.
size_t tree_workspace(long long batch, int q_len, int n_q_heads, int n_kv_heads, int splits) {
    const fa512::TreeShape s = fa512::tree_shape(q_len, n_q_heads / n_kv_heads);
    return tree_partials(batch, q_len, n_q_heads, n_kv_heads, splits).bytes() +
           round256(static_cast<size_t>(batch) * s.groups * n_kv_heads * 2 * sizeof(int32_t));
}

// Sizes whose products fit the kernels' counts and grids.
bool tree_size_ok(int batch, int q_len, int group, int n_kv_heads) {
    return batch <= 65535 && n_kv_heads <= 65535 && static_cast<long long>(q_len) * group <= 0x7fffffffLL / 1024;
}

bool tree_shape_ok(int batch, int q_len, int n_q_heads, int n_kv_heads, int max_kv_len, int n_sinks) {
    return batch >= 0 && q_len >= 1 && n_kv_heads >= 1 && n_q_heads >= 1 && n_q_heads % n_kv_heads == 0 &&
           n_q_heads / n_kv_heads <= 128 && tree_size_ok(batch, q_len, n_q_heads / n_kv_heads, n_kv_heads) &&
           max_kv_len >= 0 && n_sinks >= 0;
}

fa512_status tree_call(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                       const int32_t* kv_lens, const int32_t* q_lens, const int32_t* tree_mask, void* out,
                       float* lse, int batch, int q_len, int n_q_heads, int n_kv_heads, int page_size,
                       int num_pages, int max_pages_per_seq, int max_kv_len, float scale, int window,
                       int n_sinks, int num_splits, void* workspace, size_t workspace_bytes, bool fp8,
                       float k_scale, float v_scale, fa512_stream_t stream) {
    g_last_error[0] = 0;
    if (batch < 0) return fail(FA512_ERR_INVALID_ARG, "negative batch");
    if (q_len < 1) return fail(FA512_ERR_INVALID_ARG, "q_len must be >= 1");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
        return fail(FA512_ERR_INVALID_ARG, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)",
                    n_q_heads, n_kv_heads);
    const int G = n_q_heads / n_kv_heads;
    if (G > 128) return fail(FA512_ERR_UNSUPPORTED, "more than 128 query heads per KV head");
    if (tree_mask && q_len > fa512::tree_max_nodes())
        return fail(FA512_ERR_UNSUPPORTED, "a tree_mask covers at most %d tokens", fa512::tree_max_nodes());
    if (!pow2_page(page_size)) return fail(FA512_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(FA512_ERR_INVALID_ARG, "num_pages and max_pages_per_seq must be >= 1");
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL - 256 ||
        static_cast<long long>(max_pages_per_seq) * page_size > 0x7fffffffLL - 256)
        return fail(FA512_ERR_UNSUPPORTED, "page pool or page table too large for int32 key rows");
    if (max_kv_len < 0 || static_cast<long long>(max_kv_len) > static_cast<long long>(max_pages_per_seq) * page_size)
        return fail(FA512_ERR_INVALID_ARG, "max_kv_len outside [0, max_pages_per_seq * page_size]");
    if (num_splits < 0 || num_splits > 1024) return fail(FA512_ERR_INVALID_ARG, "num_splits outside [0, 1024]");
    if (n_sinks < 0) return fail(FA512_ERR_INVALID_ARG, "negative n_sinks");
    if (!(scale == scale) || isinf(scale)) return fail(FA512_ERR_INVALID_ARG, "scale is not finite");
    if (fp8 && (!(k_scale == k_scale) || isinf(k_scale) || !(v_scale == v_scale) || isinf(v_scale)))
        return fail(FA512_ERR_INVALID_ARG, "k_scale and v_scale must be finite");
    if (!tree_size_ok(batch, q_len, G, n_kv_heads)) return fail(FA512_ERR_UNSUPPORTED, "grid too large");
    if (batch == 0) return FA512_OK;
    if (!q || !k_pages || !v_pages || !page_table || !kv_lens || !out)
        return fail(FA512_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return fail(FA512_ERR_INVALID_ARG, "q, pages and out must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_lens) |
         reinterpret_cast<uintptr_t>(q_lens) | reinterpret_cast<uintptr_t>(tree_mask) |
         reinterpret_cast<uintptr_t>(lse)) & 3u)
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays and lse must be 4-byte aligned");
    const fa512::TreeShape shape = fa512::tree_shape(q_len, G);
    const long long tiles = tree_tiles(q_len, G, max_kv_len, window, n_sinks, page_size < 128 ? page_size : 128);
    const long long items = static_cast<long long>(batch) * shape.groups * n_kv_heads;
    if (items > 0x7fffffffLL || items * (tiles > 1 ? tiles : 1) > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "more key tiles than int32 counts");
    const int splits = num_splits > 0           ? num_splits
                       : one_piece(shape, tiles) ? 1
                                                 : fa512_decode_auto_splits_tree(batch, q_len, n_q_heads, n_kv_heads,
                                                                                 max_kv_len, window, n_sinks);
    if (splits > 1) {
        if (static_cast<long long>(batch) * q_len > 65535)
            return fail(FA512_ERR_UNSUPPORTED, "more than 65535 tokens with more than one split");
        const size_t need = tree_workspace(batch, q_len, n_q_heads, n_kv_heads, splits);
        if (!workspace || workspace_bytes < need)
            return fail(FA512_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return fail(FA512_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");

    fa512::TreeParams p;
    memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.q_lens = q_lens;
    p.tree_mask = tree_mask;
    const TreePartials partials = tree_partials(batch, q_len, n_q_heads, n_kv_heads, splits);
    p.clusters = partials.clusters;
    if (splits > 1) {
        char* ws = static_cast<char*>(workspace);
        p.ws_o = reinterpret_cast<float*>(ws);
        p.ws_ml = reinterpret_cast<float*>(ws + round256(partials.rows * kHeadDim * sizeof(float)));
        p.ws_item = reinterpret_cast<int32_t*>(ws + partials.bytes());
        p.slot_rows = partials.slot_rows;
    }
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.batch = batch;
    p.q_len = q_len;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.rows = shape.rows;
    p.row_groups = shape.groups;
    p.max_tiles = static_cast<int>(tiles);
    p.min_range = splits > 1 ? (p.max_tiles + splits - 2) / (splits - 1) : 0;
    p.mask_words = (q_len + 31) / 32;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.len_cap = max_kv_len;
    p.window = window > 0 ? window : 0;
    p.n_sinks = n_sinks;
    p.num_splits = splits;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (fp8) p.scale_log2 *= k_scale;
    p.o_scale = fp8 ? v_scale : 1.f;
    p.err = err;
    const uint64_t eb = fp8 ? 1 : 2;
    const uint64_t dims[3] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(n_kv_heads),
                              static_cast<uint64_t>(num_pages) * page_size};
    const uint64_t strides[2] = {kHeadDim * eb, static_cast<uint64_t>(n_kv_heads) * kHeadDim * eb};
    const uint32_t box[3] = {static_cast<uint32_t>(128 / eb), 1u, static_cast<uint32_t>(page_size < 128 ? page_size : 128)};
    CUtensorMap tmk, tmv;
    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    fa512_status st = encode_map(&tmk, type, CU_TENSOR_MAP_SWIZZLE_128B, k_pages, 3, dims, strides, box);
    if (st != FA512_OK) return st;
    st = encode_map(&tmv, type, CU_TENSOR_MAP_SWIZZLE_128B, v_pages, 3, dims, strides, box);
    if (st != FA512_OK) return st;
    e = fa512::launch_decode_tree(tmk, tmv, p, fp8, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree decode launch");
    return FA512_OK;
}

fa512_status append_call(const void* k_new, const void* v_new, int64_t kb, int64_t kt, int64_t vb, int64_t vt,
                         void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* kv_lens,
                         const int32_t* q_lens, int batch, int q_len, int n_kv_heads, int page_size,
                         int num_pages, int max_pages_per_seq, bool fp8, float k_scale, float v_scale,
                         fa512_stream_t stream) {
    g_last_error[0] = 0;
    if (batch < 0 || q_len < 0) return fail(FA512_ERR_INVALID_ARG, "negative batch or q_len");
    if (n_kv_heads < 1) return fail(FA512_ERR_INVALID_ARG, "n_kv_heads must be >= 1");
    if (!pow2_page(page_size)) return fail(FA512_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(FA512_ERR_INVALID_ARG, "num_pages and max_pages_per_seq must be >= 1");
    if (static_cast<long long>(max_pages_per_seq) * page_size > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "page table too large for int32 positions");
    if ((kb | kt | vb | vt) & 7)
        return fail(FA512_ERR_INVALID_ARG, "strides of k_new and v_new must be multiples of 8 elements");
    if (fp8 && (!(k_scale > 0.f) || isinf(k_scale) || !(v_scale > 0.f) || isinf(v_scale)))
        return fail(FA512_ERR_INVALID_ARG, "k_scale and v_scale must be finite and above 0");
    if (batch > 65535 || static_cast<long long>(q_len) * n_kv_heads > 0x7fffffffLL / 64)
        return fail(FA512_ERR_UNSUPPORTED, "grid too large");
    if (batch == 0 || q_len == 0) return FA512_OK;
    if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !kv_lens)
        return fail(FA512_ERR_INVALID_ARG, "null tensor pointer");
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages))
        return fail(FA512_ERR_INVALID_ARG, "k_new, v_new and pages must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_lens) |
         reinterpret_cast<uintptr_t>(q_lens)) & 3u)
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    fa512::AppendParams p;
    memset(&p, 0, sizeof p);
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.k_batch_stride = kb;
    p.k_token_stride = kt;
    p.v_batch_stride = vb;
    p.v_token_stride = vt;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.q_lens = q_lens;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.batch = batch;
    p.q_len = q_len;
    p.n_kv_heads = n_kv_heads;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.err = err;
    e = fa512::launch_cache_append(p, fp8, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
    return FA512_OK;
}

// Shared checks of the calls that take a whole cache of several layers.
fa512_status cache_shape(int n_layers, int batch, int n_kv_heads, int element_bytes, int page_size,
                         int num_pages, int max_pages_per_seq) {
    if (batch < 0 || n_layers < 0) return fail(FA512_ERR_INVALID_ARG, "negative batch or n_layers");
    if (n_kv_heads < 1 || n_kv_heads > 65535) return fail(FA512_ERR_INVALID_ARG, "n_kv_heads outside [1, 65535]");
    if (element_bytes != 1 && element_bytes != 2)
        return fail(FA512_ERR_INVALID_ARG, "element_bytes must be 1 (E4M3) or 2 (bf16)");
    if (!pow2_page(page_size)) return fail(FA512_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(FA512_ERR_INVALID_ARG, "num_pages and max_pages_per_seq must be >= 1");
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL ||
        static_cast<long long>(max_pages_per_seq) * page_size > 0x7fffffffLL)
        return fail(FA512_ERR_UNSUPPORTED, "page pool or page table too large for int32 rows");
    if (n_layers > 32767) return fail(FA512_ERR_UNSUPPORTED, "more than 32767 layers");
    return FA512_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

extern "C" {

int fa512_decode_auto_splits_tree(int batch, int q_len, int n_q_heads, int n_kv_heads, int max_kv_len,
                                  int window, int n_sinks) {
    if (!tree_shape_ok(batch, q_len, n_q_heads, n_kv_heads, max_kv_len, n_sinks) || batch == 0) return 1;
    if (static_cast<long long>(batch) * q_len > 65535) return 1;   // the merge's grid
    const int G = n_q_heads / n_kv_heads;
    const fa512::TreeShape s = fa512::tree_shape(q_len, G);
    const long long tiles = tree_tiles(q_len, G, max_kv_len, window, n_sinks, 128);
    const long long clusters = sm_count() / s.ctas > 0 ? sm_count() / s.ctas : 1;
    const long long items = static_cast<long long>(batch) * n_kv_heads * s.groups;
    if (items > 0x7fffffffLL || one_piece(s, tiles)) return 1;
    const long long per = (items * tiles + clusters - 1) / clusters;
    if (per <= 0) return 1;
    // the ranges of a batch of this length touch ceil(tiles / per) + 1 of an
    // item's segments at most; a batch with shorter sequences has shorter
    // ranges, so twice as many are allowed
    const long long most = 2 * ((tiles + per - 1) / per) + 1;
    return static_cast<int>(most < tiles + 1 ? (most < 1024 ? most : 1024) : (tiles + 1 < 1024 ? tiles + 1 : 1024));
}

size_t fa512_decode_workspace_bytes_tree(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                         int max_kv_len, int window, int n_sinks, int num_splits) {
    if (!tree_shape_ok(batch, q_len, n_q_heads, n_kv_heads, max_kv_len, n_sinks) || num_splits < 0 ||
        num_splits > 1024)
        return 0;
    const int s = num_splits > 0 ? num_splits
                                 : fa512_decode_auto_splits_tree(batch, q_len, n_q_heads, n_kv_heads,
                                                                 max_kv_len, window, n_sinks);
    if (s == 1 || batch == 0) return 256;
    return tree_workspace(batch, q_len, n_q_heads, n_kv_heads, s);
}

fa512_status fa512_decode_paged_tree(const void* q, const void* k_pages, const void* v_pages,
                                     const int32_t* page_table, const int32_t* kv_lens,
                                     const int32_t* q_lens, const int32_t* tree_mask, void* out, float* lse,
                                     int batch, int q_len, int n_q_heads, int n_kv_heads, int page_size,
                                     int num_pages, int max_pages_per_seq, int max_kv_len, float scale,
                                     int window, int n_sinks, int num_splits, void* workspace,
                                     size_t workspace_bytes, fa512_stream_t stream) {
    return tree_call(q, k_pages, v_pages, page_table, kv_lens, q_lens, tree_mask, out, lse, batch, q_len,
                     n_q_heads, n_kv_heads, page_size, num_pages, max_pages_per_seq, max_kv_len, scale, window,
                     n_sinks, num_splits, workspace, workspace_bytes, false, 1.f, 1.f, stream);
}

fa512_status fa512_decode_paged_tree_fp8(const void* q, const void* k_pages, const void* v_pages,
                                         const int32_t* page_table, const int32_t* kv_lens,
                                         const int32_t* q_lens, const int32_t* tree_mask, void* out,
                                         float* lse, int batch, int q_len, int n_q_heads, int n_kv_heads,
                                         int page_size, int num_pages, int max_pages_per_seq, int max_kv_len,
                                         float scale, float k_scale, float v_scale, int window, int n_sinks,
                                         int num_splits, void* workspace, size_t workspace_bytes,
                                         fa512_stream_t stream) {
    return tree_call(q, k_pages, v_pages, page_table, kv_lens, q_lens, tree_mask, out, lse, batch, q_len,
                     n_q_heads, n_kv_heads, page_size, num_pages, max_pages_per_seq, max_kv_len, scale, window,
                     n_sinks, num_splits, workspace, workspace_bytes, true, k_scale, v_scale, stream);
}

fa512_status fa512_cache_append(const void* k_new, const void* v_new, int64_t k_batch_stride,
                                int64_t k_token_stride, int64_t v_batch_stride, int64_t v_token_stride,
                                void* k_pages, void* v_pages, const int32_t* page_table,
                                const int32_t* kv_lens, const int32_t* q_lens, int batch, int q_len,
                                int n_kv_heads, int page_size, int num_pages, int max_pages_per_seq,
                                fa512_stream_t stream) {
    return append_call(k_new, v_new, k_batch_stride, k_token_stride, v_batch_stride, v_token_stride, k_pages,
                       v_pages, page_table, kv_lens, q_lens, batch, q_len, n_kv_heads, page_size, num_pages,
                       max_pages_per_seq, false, 1.f, 1.f, stream);
}

fa512_status fa512_cache_append_fp8(const void* k_new, const void* v_new, int64_t k_batch_stride,
                                    int64_t k_token_stride, int64_t v_batch_stride, int64_t v_token_stride,
                                    void* k_pages, void* v_pages, const int32_t* page_table,
                                    const int32_t* kv_lens, const int32_t* q_lens, float k_scale,
                                    float v_scale, int batch, int q_len, int n_kv_heads, int page_size,
                                    int num_pages, int max_pages_per_seq, fa512_stream_t stream) {
    return append_call(k_new, v_new, k_batch_stride, k_token_stride, v_batch_stride, v_token_stride, k_pages,
                       v_pages, page_table, kv_lens, q_lens, batch, q_len, n_kv_heads, page_size, num_pages,
                       max_pages_per_seq, true, k_scale, v_scale, stream);
}

fa512_status fa512_cache_compact(void* k_pages, void* v_pages, const int32_t* page_table,
                                 const int32_t* kv_lens, const int32_t* q_lens, const int32_t* accepted,
                                 const int32_t* n_accepted, int32_t* new_kv_lens, int n_layers, int batch,
                                 int q_len, int max_accepted, int n_kv_heads, int element_bytes, int page_size,
                                 int num_pages, int max_pages_per_seq, fa512_stream_t stream) {
    g_last_error[0] = 0;
    fa512_status st = cache_shape(n_layers, batch, n_kv_heads, element_bytes, page_size, num_pages,
                                  max_pages_per_seq);
    if (st != FA512_OK) return st;
    if (q_len < 0 || max_accepted < 0) return fail(FA512_ERR_INVALID_ARG, "negative q_len or max_accepted");
    if (max_accepted > fa512::compact_max_accepted())
        return fail(FA512_ERR_UNSUPPORTED, "max_accepted above %d", fa512::compact_max_accepted());
    if (batch > 65535) return fail(FA512_ERR_UNSUPPORTED, "grid too large");
    if (batch == 0) return FA512_OK;
    if (!kv_lens || !n_accepted || !new_kv_lens || !page_table || (max_accepted > 0 && !accepted) ||
        (n_layers > 0 && (!k_pages || !v_pages)))
        return fail(FA512_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k_pages) || !aligned16(v_pages))
        return fail(FA512_ERR_INVALID_ARG, "pages must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(kv_lens) || misaligned4(q_lens) || misaligned4(accepted) ||
        misaligned4(n_accepted) || misaligned4(new_kv_lens))
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    const size_t nb = static_cast<size_t>(batch) * 4;
    if (overlap(new_kv_lens, nb, kv_lens, nb) || overlap(new_kv_lens, nb, q_lens, nb) ||
        overlap(new_kv_lens, nb, n_accepted, nb) || overlap(new_kv_lens, nb, accepted, nb * max_accepted) ||
        overlap(new_kv_lens, nb, page_table, nb * max_pages_per_seq))
        return fail(FA512_ERR_INVALID_ARG, "new_kv_lens overlaps an input");
    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    fa512::CompactParams p;
    memset(&p, 0, sizeof p);
    p.k_pages = static_cast<uint8_t*>(k_pages);
    p.v_pages = static_cast<uint8_t*>(v_pages);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.q_lens = q_lens;
    p.accepted = accepted;
    p.n_accepted = n_accepted;
    p.new_kv_lens = new_kv_lens;
    p.n_layers = n_layers;
    p.batch = batch;
    p.q_len = q_len;
    p.max_accepted = max_accepted;
    p.row_bytes = n_kv_heads * kHeadDim * element_bytes;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.err = err;
    e = fa512::launch_cache_compact(p, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache compact launch");
    return FA512_OK;
}

fa512_status fa512_cache_fork(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* kv_lens,
                              const int32_t* parents, const int32_t* page_refs, int32_t* new_page_table,
                              int32_t* new_kv_lens, int32_t* new_page_refs, int n_layers, int batch,
                              int n_children, int n_kv_heads, int element_bytes, int page_size, int num_pages,
                              int max_pages_per_seq, fa512_stream_t stream) {
    g_last_error[0] = 0;
    fa512_status st = cache_shape(n_layers, batch, n_kv_heads, element_bytes, page_size, num_pages,
                                  max_pages_per_seq);
    if (st != FA512_OK) return st;
    if (n_children < 0) return fail(FA512_ERR_INVALID_ARG, "negative n_children");
    if (batch > fa512::page_plan_max_batch() || n_children > fa512::page_plan_max_batch())
        return fail(FA512_ERR_UNSUPPORTED, "more than %d sequences", fa512::page_plan_max_batch());
    if (!page_refs || !new_page_refs || (batch > 0 && (!page_table || !kv_lens)) ||
        (n_children > 0 && (!parents || !new_page_table || !new_kv_lens)) ||
        (n_layers > 0 && (!k_pages || !v_pages)))
        return fail(FA512_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k_pages) || !aligned16(v_pages))
        return fail(FA512_ERR_INVALID_ARG, "pages must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(kv_lens) || misaligned4(parents) || misaligned4(page_refs) ||
        misaligned4(new_page_table) || misaligned4(new_kv_lens) || misaligned4(new_page_refs))
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    const size_t row = static_cast<size_t>(max_pages_per_seq) * 4, pool = static_cast<size_t>(num_pages) * 4;
    struct { const void* p; size_t n; } in[] = {{page_table, row * batch}, {kv_lens, 4ull * batch},
                                                {parents, 4ull * n_children}, {page_refs, pool}},
                                        outs[] = {{new_page_table, row * n_children},
                                                  {new_kv_lens, 4ull * n_children}, {new_page_refs, pool}};
    for (auto& o : outs)
        for (auto& i : in)
            if (overlap(o.p, o.n, i.p, i.n) && !(o.p == new_page_refs && i.p == page_refs && o.p == i.p))
                return fail(FA512_ERR_INVALID_ARG, "an output overlaps an input");
    if (overlap(outs[0].p, outs[0].n, outs[1].p, outs[1].n) || overlap(outs[0].p, outs[0].n, outs[2].p, outs[2].n) ||
        overlap(outs[1].p, outs[1].n, outs[2].p, outs[2].n))
        return fail(FA512_ERR_INVALID_ARG, "two outputs overlap");
    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    fa512::PagePlanParams p;
    memset(&p, 0, sizeof p);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.page_refs = page_refs;
    p.parents = parents;
    p.new_table = new_page_table;
    p.new_lens = new_kv_lens;
    p.new_refs = new_page_refs;
    p.batch = batch;
    p.n_new = n_children;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.k_pages = static_cast<uint8_t*>(k_pages);
    p.v_pages = static_cast<uint8_t*>(v_pages);
    p.n_layers = n_layers;
    p.row_bytes = n_kv_heads * kHeadDim * element_bytes;
    p.err = err;
    e = fa512::launch_page_plan(p, true, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache fork launch");
    return FA512_OK;
}

fa512_status fa512_cache_resize(const int32_t* page_table, const int32_t* kv_lens, const int32_t* new_kv_lens,
                                const int32_t* page_refs, int32_t* new_page_table, int32_t* new_page_refs,
                                int batch, int page_size, int num_pages, int max_pages_per_seq,
                                fa512_stream_t stream) {
    g_last_error[0] = 0;
    fa512_status st = cache_shape(0, batch, 1, 2, page_size, num_pages, max_pages_per_seq);
    if (st != FA512_OK) return st;
    if (batch > fa512::page_plan_max_batch())
        return fail(FA512_ERR_UNSUPPORTED, "more than %d sequences", fa512::page_plan_max_batch());
    if (!page_refs || !new_page_refs ||
        (batch > 0 && (!page_table || !kv_lens || !new_kv_lens || !new_page_table)))
        return fail(FA512_ERR_INVALID_ARG, "null pointer");
    if (misaligned4(page_table) || misaligned4(kv_lens) || misaligned4(new_kv_lens) || misaligned4(page_refs) ||
        misaligned4(new_page_table) || misaligned4(new_page_refs))
        return fail(FA512_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    const size_t tb = static_cast<size_t>(max_pages_per_seq) * 4 * batch, pool = static_cast<size_t>(num_pages) * 4,
                 lb = 4ull * batch;
    if ((new_page_table != page_table && overlap(new_page_table, tb, page_table, tb)) ||
        (new_page_refs != page_refs && overlap(new_page_refs, pool, page_refs, pool)) ||
        overlap(new_page_table, tb, kv_lens, lb) || overlap(new_page_table, tb, new_kv_lens, lb) ||
        overlap(new_page_table, tb, page_refs, pool) || overlap(new_page_table, tb, new_page_refs, pool) ||
        overlap(new_page_refs, pool, kv_lens, lb) || overlap(new_page_refs, pool, new_kv_lens, lb) ||
        overlap(new_page_refs, pool, page_table, tb))
        return fail(FA512_ERR_INVALID_ARG, "an output overlaps another array");
    unsigned* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    fa512::PagePlanParams p;
    memset(&p, 0, sizeof p);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.page_refs = page_refs;
    p.next_lens = new_kv_lens;
    p.new_table = new_page_table;
    p.new_refs = new_page_refs;
    p.batch = batch;
    p.n_new = batch;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages_per_seq = max_pages_per_seq;
    p.err = err;
    e = fa512::launch_page_plan(p, false, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cache resize launch");
    return FA512_OK;
}

}  // extern "C"
