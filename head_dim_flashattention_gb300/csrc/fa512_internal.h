// Internal interface between the C ABI (api.cu) and the kernel translation
// units.  Not installed; the public interface is include/fa512.h.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa512 {

struct DecodeParams {
    const __nv_bfloat16* q;        // [batch, q_len, n_q_heads, 512]
    const __nv_bfloat16* k_pages;  // [num_pages, page_size, n_kv_heads, 512]
    const __nv_bfloat16* v_pages;
    // FP8 E4M3 cache (same layout, one byte per element; null for a bf16
    // cache): a key element is k_scale * e4m3, a value element v_scale * e4m3.
    // k_scale is folded into scale_log2, v_scale into o_scale.
    const uint8_t* k8;
    const uint8_t* v8;
    float o_scale;                 // multiplies the split partials O (FP8 cache: v_scale)
    const int32_t* page_table;     // [batch, max_pages_per_seq]
    const int32_t* kv_lens;        // [batch]
    float* ws_o;                   // [batch, q_len, n_q_heads, num_splits, 512] unnormalised O
    float* ws_ml;                  // [batch, q_len, n_q_heads, num_splits, 2] (m in log2 units, l)
    __nv_bfloat16* out;            // [batch, q_len, n_q_heads, 512]
    float* lse;                    // [batch, q_len, n_q_heads] or null
    int batch, n_q_heads, n_kv_heads, group;
    int q_len;                     // query tokens per sequence: its last q_len positions
    int page_size, box_rows, num_pages, max_pages_per_seq;
    int len_cap;                   // min(max_kv_len, max_pages_per_seq * page_size)
    int window;
    int tiles_per_split, num_splits;
    int page_shift;                // page_size = 1 << page_shift
    int groups;                    // kernels over ranges: ranges that the tiles of all sequences are dealt in, tiles_per_split long at least
    float scale_log2;              // scale * log2(e)
    unsigned* err;                 // device error word
    // Selected pages (null: all of the band): [batch, n_kv_heads, n_listed] logical
    // pages in rising order, then -1.  Positions are then counted along the list:
    // position v is slot v % page_size of entry v / page_size.
    const int32_t* listed;
    int n_listed;
};

int decode_smem_bytes();
int decode_tile_positions();
cudaError_t launch_decode(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p,
                          cudaStream_t stream);
// FP8 cache: tmk / tmv map the e4m3 pages as bytes, boxes of
// decode_fp8_box_bytes() head-dim bytes x box_rows positions, no swizzle.
int decode_fp8_box_bytes();
// FP8 cache with q_len * G <= decode_fp8_mma_rows(): the split kernel runs
// decode_fp8_ctas_per_sm() CTAs per SM, one split each.
int decode_fp8_mma_rows();
int decode_fp8_ctas_per_sm();
// The merge kernel takes `rows` (sequence, token, query head) rows in four
// column slices each (128 splits loaded up front) when this is true, else
// whole (32 splits up front).
bool decode_merge_sliced(long long rows);
cudaError_t launch_decode_fp8(const CUtensorMap& tmk, const CUtensorMap& tmv,
                              const DecodeParams& p, cudaStream_t stream);
// Combines the split partials of a kernel that has allowed a dependent launch.
cudaError_t launch_decode_merge(const DecodeParams& p, cudaStream_t stream);

// Kernels over ranges of tiles: a 4-bit cache (bits 4), or listed pages of any (16, 8, 4).
// tmk / tmv: 4 bits, rows of kFp4RowBytes as 32-bit words, boxes of a whole row x
// box_rows positions (min(page_size, decode_ranges_tile())), no swizzle; else boxes of
// 128 bytes x box_rows positions, 128-byte swizzle.  The pages' pointers are unused.
constexpr int kFp4RowBytes = 288;  // 256 bytes of E2M1 pairs, 32 E4M3 scales
int decode_ranges_tile(int bits);  // positions
int decode_ranges_ctas_per_sm();
cudaError_t launch_decode_ranges(const CUtensorMap& tmk, const CUtensorMap& tmv, const DecodeParams& p, int bits,
                                 cudaStream_t stream);

// Bounds of a page's keys, and the pages whose bounds allow the largest products.
struct BoundsParams {
    const uint8_t* k_pages;        // rows of one head: 1024, 512 or kFp4RowBytes bytes
    const int32_t *page_table, *kv_lens, *q_lens;
    __nv_bfloat16* bounds;         // [num_pages, n_kv_heads, 2, 512] smallest, largest
    int batch, q_len, n_kv_heads, page_size, num_pages, max_pages_per_seq;
    unsigned* err;
};
cudaError_t launch_page_bounds(const BoundsParams& p, int element_bits, cudaStream_t stream);

struct SelectParams {
    const __nv_bfloat16* q;        // [batch, q_len, n_q_heads, 512]
    const __nv_bfloat16* bounds;
    const int32_t *page_table, *kv_lens;
    int32_t* selected;             // [batch, n_kv_heads, n_select]
    uint32_t* keys;                // [batch, n_kv_heads, max_pages] ordered like the scores
    int batch, q_len, n_q_heads, n_kv_heads, group;
    int page_size, num_pages, max_pages_per_seq, len_cap;
    int max_pages;                 // pages of len_cap
    int n_select, n_first, n_last;
    unsigned* err;
};
cudaError_t launch_select_pages(const SelectParams& p, cudaStream_t stream);

// Drafted tokens (a tree or a run of them) over a paged cache.
struct TreeParams {
    const __nv_bfloat16* q;        // [batch, q_len, n_q_heads, 512]
    const void* k_pages;           // [num_pages, page_size, n_kv_heads, 512] bf16 or E4M3
    const void* v_pages;
    const int32_t* page_table;     // [batch, max_pages_per_seq]
    const int32_t* kv_lens;        // [batch]
    const int32_t* q_lens;         // [batch] or null: q_len each
    const int32_t* tree_mask;      // [batch, q_len, mask_words] or null: a run of tokens
    // Partials: unnormalised O (512 floats each) and (m, l).  Either a place per
    // row and segment, [batch, q_len, n_q_heads, num_splits], or (slot_rows > 0)
    // a slot of slot_rows rows for the first and for the last segment of each
    // cluster, [clusters, 2, slot_rows]: no other of its segments is a partial.
    float* ws_o;
    float* ws_ml;
    int32_t* ws_item;              // [batch, row_groups, n_kv_heads, 2] segments | cluster step << 16, first cluster
    int slot_rows;
    int clusters;                  // most CTAs (or pairs) of the launch
    __nv_bfloat16* out;            // [batch, q_len, n_q_heads, 512]
    float* lse;                    // [batch, q_len, n_q_heads] or null
    int batch, q_len, n_q_heads, n_kv_heads, group, mask_words;
    int rows, row_groups;          // TreeShape
    int max_tiles;                 // most key tiles of an item
    int min_range;                 // shortest range of tiles that keeps an item to num_splits segments
    int page_size, num_pages, max_pages_per_seq, len_cap;
    int window, n_sinks;
    int num_splits;                // most segments of an item; 1: no partials
    float scale_log2;              // scale * log2(e) (E4M3 cache: * k_scale)
    float o_scale;                 // E4M3 cache: v_scale; else 1
    unsigned* err;
};

int tree_max_nodes();              // most tokens a tree_mask covers
struct TreeShape {
    int rows;                      // rows of a KV head that share a walk over its keys
    int ctas;                      // CTAs that hold them
    int tile;                      // keys per tile
    int groups;                    // row groups of a KV head
};
TreeShape tree_shape(int q_len, int group);
// Both maps: {128 bytes of the head dim, 1 KV head, min(page_size, 128) positions} boxes, 128-byte swizzle.
cudaError_t launch_decode_tree(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, bool fp8,
                               cudaStream_t stream);

struct AppendParams {
    const __nv_bfloat16 *k_new, *v_new;
    long long k_batch_stride, k_token_stride, v_batch_stride, v_token_stride;   // elements
    void *k_pages, *v_pages;
    const int32_t *page_table, *kv_lens, *q_lens;
    float k_scale, v_scale;        // E4M3 and 4-bit caches
    int batch, q_len, n_kv_heads, page_size, num_pages, max_pages_per_seq;
    int page_shift;                // page_size = 1 << page_shift
    unsigned* err;
};
// element_bits: 16 (bf16), 8 (E4M3) or 4 (E2M1 with group scales)
cudaError_t launch_cache_append(const AppendParams& p, int element_bits, cudaStream_t stream);

struct CompactParams {
    uint8_t *k_pages, *v_pages;    // rows of row_bytes (all KV heads of a position)
    const int32_t *page_table, *kv_lens, *q_lens, *accepted, *n_accepted;
    int32_t* new_kv_lens;
    int n_layers, batch, q_len, max_accepted, row_bytes, page_size, num_pages, max_pages_per_seq;
    unsigned* err;
};
int compact_max_accepted();
cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream);

// Fork and resize of a cache's page tables.
struct PagePlanParams {
    const int32_t *page_table, *kv_lens, *page_refs;
    const int32_t* parents;        // fork: [n_new]
    const int32_t* next_lens;      // resize: [batch]
    int32_t *new_table, *new_lens, *new_refs;
    int batch, n_new, page_size, num_pages, max_pages_per_seq;
    // fork: the pages to copy
    uint8_t *k_pages, *v_pages;
    int n_layers, row_bytes;
    unsigned* err;
};
int page_plan_max_batch();
cudaError_t launch_page_plan(const PagePlanParams& p, bool fork, cudaStream_t stream);

struct PrefillParams {
    __nv_bfloat16* out;            // [total_q, n_q_heads, 512]
    float* lse;                    // [n_q_heads, total_q] or null
    int seqlen_q, seqlen_k, q_offset, n_q_heads, n_kv_heads, group;
    int tokens_per_tile;           // query tokens packed per 128-row tile
    int rows_per_tile;             // tokens_per_tile * group (<= 128)
    int num_q_tiles;               // per KV head (contiguous mode)
    int causal, window;
    float scale_log2;              // scale * log2(e)
    unsigned* err;
    int total_q;                   // rows of q / out (contiguous mode: seqlen_q)
    // varlen mode over a paged cache (the contiguous kernel ignores these)
    const int32_t* page_table;     // [batch, max_pages_per_seq]
    const int32_t* cu_seqlens_q;   // [batch + 1]
    const int32_t* seqused_k;      // [batch]
    int batch, max_seqlen_q, max_pairs;
    int page_shift, num_pages, max_pages_per_seq;
    int oob_row;                   // num_pages * page_size: a row past the pool (TMA fills zeros)
    unsigned long long wait_limit_ns;  // bound of each pipeline wait (0: the default, 2 s)
    int test_skip_first_k_load;    // test hook: CTA 0 does not issue its first K load
};

int prefill_smem_bytes();
int prefill_k_box_rows();   // keys per K box (one head-dim chunk of a key tile)
int prefill_v_box_rows();   // keys per V box (one key slice)

// Head dim 256 (the sliding-window local layers): a persistent kernel, one
// cluster of two CTAs per SM pair, each walking a contiguous range of
// (KV head, q-tile pair) items.
constexpr int kMaxPersistentClusters = 128;

struct Prefill256Params {
    __nv_bfloat16* out;            // [seqlen_q, n_q_heads, 256]
    float* lse;                    // [n_q_heads, seqlen_q] or null
    int seqlen_q, seqlen_k, q_offset, n_q_heads, n_kv_heads, group;
    int tokens_per_tile, rows_per_tile, num_q_tiles, n_pairs, n_items;
    int causal, window;
    float scale_log2;
    unsigned* err;
    int n_clusters;
    // items of cluster c: range_start[c], + item_stride, ... below range_start[c + 1]
    int item_stride;
    int range_start[kMaxPersistentClusters + 1];
};

int prefill256_smem_bytes();
int prefill256_k_box_rows();
int prefill256_v_box_rows();
void plan_prefill256(Prefill256Params& p, int n_sm);
cudaError_t launch_prefill256(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                              const CUtensorMap& tmo, const Prefill256Params& p, cudaStream_t stream);

// Sets the text fa512_last_error_message() returns on this thread.
void set_last_error_message(const char* msg);
cudaError_t launch_prefill(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                           const PrefillParams& p, cudaStream_t stream);
int prefill_paged_v_box_rows();   // keys per V box over a paged cache (one page-aligned half tile)
cudaError_t launch_prefill_paged(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                 const PrefillParams& p, cudaStream_t stream);

}  // namespace fa512
