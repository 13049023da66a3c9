/*
 * fa512 -- head-dim-512 FlashAttention forward for GB300 (sm_103a).
 *
 * C ABI of the library.  Plain pointers and sizes only; every device pointer
 * is owned by the caller, the library calls no allocator and never
 * synchronises the stream it is given.  All work is enqueued on `stream`.
 * The library's own device memory is static: a 4-byte error word and the
 * FA512_DECODE_STATIC_SCRATCH_BYTES array of fa512_decode_paged_noalloc,
 * held on every GPU that loads the library until the process exits.  Their
 * device addresses are looked up once per device and kept, so the library
 * must not be used across a device reset (cudaDeviceReset).
 *
 * Operations (page title, then the part of the page that states them):
 *
 *  fa512_prefill -- causal GQA/MQA attention of a chunk of query rows against
 *    the keys before them, with online softmax (running max m, running sum l,
 *    rescaled O) so the [q x k] score matrix never reaches memory.
 *    "Writing a FlashAttention Prefill Kernel for Gemma 4", sections "The
 *    starting point" and "Head dim 512 breaks the textbook"; "A custom
 *    attention kernel for Gemma 4 on the RTX PRO 6000", section "The kernel
 *    in three steps" (query heads that share a KV head are packed into one
 *    tile); pegainfer issue #1051, "Description" (one 8192-row chunk against
 *    everything before it, 32 query heads over 4 KV heads).
 *
 *  fa512_prefill_d256 -- the same for heads of 256 dimensions (the
 *    sliding-window local layers, window 1,024), from a persistent kernel.
 *
 *  fa512_prefill_paged -- the same for a batch of chunks of different
 *    lengths over a paged KV cache (pegainfer issue #1051, "Proposed Plan").
 *
 *  fa512_decode_paged_fp8 -- the same over a cache stored in FP8 E4M3
 *    (vllm-project/flash-attention PR #199, "Summary").
 *
 *  fa512_decode_paged -- one query token per sequence against a paged KV
 *    cache, split over the key sequence (Flash-Decoding): each split writes an
 *    unnormalised (O, m, l) partial and a merge step combines them.
 *    "Flash-Decoding for MQA in CUDA", section "One KV head breaks the
 *    textbook"; vllm-project/flash-attention PR #199, "Performance" table
 *    (q_len 1, 8 query heads over 4 KV heads, head dim 512, page size 64).
 *
 *  fa512_decode_paged_tree, fa512_decode_paged_tree_fp8 -- the drafted tokens
 *    of each sequence, a tree of them or a plain run of any length, against
 *    the cache they were just appended to; with a window, the first n_sinks
 *    positions can stay visible.
 *
 *  fa512_decode_paged_fp4 -- the decode calls over a cache held in 4 bits an
 *    element, filled by fa512_cache_append_fp4.
 *
 *  fa512_cache_page_bounds, fa512_select_pages, fa512_decode_paged_sparse,
 *    _sparse_fp8, _sparse_fp4 -- a decode step that reads only the pages whose
 *    keys can have large products with the queries.
 *
 *  fa512_cache_append, _append_fp8, _compact, _fork, _resize -- the cache
 *    around those calls: writing new rows, moving accepted rows together,
 *    sharing and copying pages between sequences, handing out and taking back
 *    pages by reference counts.  The pages read a cache that a serving system
 *    manages; these have no counterpart there.
 *
 * Numerics: bf16 inputs and outputs, fp32 accumulation and softmax state.
 * LSE is the natural logarithm of sum_j exp(scale * q.k_j) over the visible
 * keys; a row with no visible key gets O = 0 and LSE = -inf
 * (vllm-project/flash-attention PR #199, review item F4).
 *
 * Errors: arguments are validated before anything is enqueued; a rejected
 * call returns a non-zero fa512_status and launches nothing.  A failed launch
 * returns FA512_ERR_CUDA.  Faults that only the device can see (a page index
 * outside the pool, a kv length beyond the page table, a pipeline wait that
 * ran past its bound) are recorded in a device-side error word that
 * fa512_device_status() reads; the kernels skip the offending access instead
 * of trapping.
 */
#ifndef FA512_H
#define FA512_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *fa512_stream_t;

typedef enum {
    FA512_OK = 0,
    FA512_ERR_INVALID_ARG = 1, /* a pointer, size or alignment is unusable      */
    FA512_ERR_UNSUPPORTED = 2, /* well-formed but outside what the kernels do    */
    FA512_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed              */
    FA512_ERR_TIMEOUT = 4,     /* device: a pipeline wait exceeded its bound     */
    FA512_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required     */
    FA512_ERR_DEVICE_INDEX = 6, /* device: page index or kv length out of range  */
    FA512_ERR_OUT_OF_PAGES = 7  /* device: more pages asked for than are free    */
} fa512_status;

/* Head dimension of every tensor this library accepts. */
#define FA512_HEAD_DIM 512

/*
 * fa512_prefill -- attention forward of one prefill chunk (batch 1).
 *
 *   q    [seqlen_q, n_q_heads, 512]  bf16, device, contiguous
 *   k, v [seqlen_k, n_kv_heads, 512] bf16, device, contiguous
 *   out  [seqlen_q, n_q_heads, 512]  bf16, device, written
 *   lse  [n_q_heads, seqlen_q]       fp32, device, written; may be NULL
 *
 * Query row i sits at absolute position q_offset + i.  Query head h reads KV
 * head h / (n_q_heads / n_kv_heads).  Key j is visible to row i iff
 *   (causal == 0 or j <= q_offset + i)  and
 *   (window <= 0 or j > q_offset + i - window)        (window keys incl. own).
 * scale multiplies q.k before the softmax (1/sqrt(512) for Gemma-4 shapes).
 *
 * Requirements: seqlen_q >= 0, seqlen_k >= 0, q_offset >= 0, n_kv_heads >= 1,
 * n_q_heads a multiple of n_kv_heads with G = n_q_heads / n_kv_heads <= 128,
 * every pointer 16-byte aligned.  seqlen_q == 0 is a no-op.
 * Returns FA512_OK once the kernels are enqueued.
 */
fa512_status fa512_prefill(const void *q, const void *k, const void *v, void *out, float *lse,
                           int seqlen_q, int seqlen_k, int q_offset, int n_q_heads,
                           int n_kv_heads, float scale, int causal, int window,
                           fa512_stream_t stream);

/*
 * fa512_prefill_d256 -- the same forward for heads of 256 dimensions, the
 * sliding-window local layers ("A custom attention kernel for Gemma 4 on the
 * RTX PRO 6000", "The deployment": they attend to the last 1,024 tokens with
 * heads of 256 dimensions).
 *
 *   q    [seqlen_q, n_q_heads, 256]  bf16, device, contiguous
 *   k, v [seqlen_k, n_kv_heads, 256] bf16, device, contiguous
 *   out  [seqlen_q, n_q_heads, 256]  bf16, device, written
 *   lse  [n_q_heads, seqlen_q]       fp32, device, written; may be NULL
 *
 * Positions, visibility (causal, window), scale, requirements and errors are
 * those of fa512_prefill; a window of 1024 is the local layers' setting and
 * window <= 0 attends causally (or fully) to every key.
 */
fa512_status fa512_prefill_d256(const void *q, const void *k, const void *v, void *out, float *lse,
                                int seqlen_q, int seqlen_k, int q_offset, int n_q_heads,
                                int n_kv_heads, float scale, int causal, int window,
                                fa512_stream_t stream);

/*
 * fa512_prefill_paged -- attention forward of a batch of prefill chunks
 * (varlen rows) over a paged KV cache.  pegainfer issue #1051, "Proposed
 * Plan" (a varlen paged prefill for head dim 512; the pool paged at the key
 * block, so a block of keys is one copy); vllm-project/flash-attention PR
 * #199, review (call shapes: varlen Q, paged K/V, prefix prefill).
 *
 *   q            [total_q, n_q_heads, 512]              bf16, device
 *   k_pages      [num_pages, page_size, n_kv_heads, 512] bf16, device
 *   v_pages      same shape as k_pages                  bf16, device
 *   page_table   [batch, max_pages_per_seq] int32, device: logical page p of
 *                sequence b is physical page page_table[b * max_pages_per_seq + p]
 *   cu_seqlens_q [batch + 1] int32, device: the chunk of sequence b is rows
 *                cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 of q and out
 *   seqused_k    [batch] int32, device: cached positions of sequence b,
 *                the chunk's own keys included
 *   out          [total_q, n_q_heads, 512] bf16, device, written
 *   lse          [n_q_heads, total_q] fp32, device, written; may be NULL
 *
 * A chunk is the tail of its sequence: row i of a chunk of S rows sits at
 * position seqused_k[b] - S + i, and key j < seqused_k[b] is visible to it
 * under the same causal / window rule as fa512_prefill (a negative position
 * sees no key when causal: O = 0, LSE = -inf).  Only the pages that hold
 * visible positions are read; slots past seqused_k[b] may hold anything
 * (NaN included) without reaching the output.
 *
 * max_seqlen_q is a host-side upper bound of the chunk lengths (it sizes the
 * grid; nothing is read back).  On the device, a chunk longer than
 * max_seqlen_q, seqused_k[b] outside [0, max_pages_per_seq * page_size],
 * cu_seqlens_q not rising within [0, total_q], or a page index outside
 * [0, num_pages) is recorded in the device error word; the offending rows or
 * pages are clipped or read as zeros, never out of bounds.
 *
 * Requirements: page_size 64, 128 or 256 (a page holds whole 64-key half
 * tiles); num_pages, max_pages_per_seq >= 1; n_q_heads a multiple of
 * n_kv_heads with at most 128 query heads per KV head; tensors 16-byte
 * aligned, int32 arrays 4-byte aligned.  batch, total_q or max_seqlen_q == 0
 * is a no-op.
 */
fa512_status fa512_prefill_paged(const void *q, const void *k_pages, const void *v_pages,
                                 const int32_t *page_table, const int32_t *cu_seqlens_q,
                                 const int32_t *seqused_k, void *out, float *lse, int batch,
                                 int total_q, int max_seqlen_q, int n_q_heads, int n_kv_heads,
                                 int page_size, int num_pages, int max_pages_per_seq, float scale,
                                 int causal, int window, fa512_stream_t stream);

/*
 * fa512_decode_paged -- one query token per sequence over a paged KV cache.
 *
 *   q          [batch, n_q_heads, 512]                     bf16, device
 *   k_pages    [num_pages, page_size, n_kv_heads, 512]      bf16, device
 *   v_pages    same shape as k_pages                        bf16, device
 *   page_table [batch, max_pages_per_seq] int32, device: logical page p of
 *              sequence b is physical page page_table[b * max_pages_per_seq + p]
 *   kv_lens    [batch] int32, device: live length of each sequence
 *   out        [batch, n_q_heads, 512] bf16, device, written
 *   lse        [batch, n_q_heads] fp32, device, written; may be NULL
 *
 * The query of sequence b sits at position kv_lens[b] - 1 and sees positions
 * [max(0, kv_lens[b] - window), kv_lens[b]) (window <= 0: all of [0, len)).
 * Only the pages that hold those positions are read.
 *
 * max_kv_len is a host-side upper bound of kv_lens (it sizes the split grid;
 * no value is read back from the device).  kv_lens[b] > max_kv_len is an
 * error recorded on the device; positions past max_kv_len are not read.
 * num_splits: 0 picks fa512_decode_auto_splits(); otherwise 1 <= num_splits
 * <= 1024.  workspace holds the (O, m, l) partials and must be at least
 * fa512_decode_workspace_bytes(batch, n_q_heads, splits) bytes, 256-byte
 * aligned, for the split count actually used.
 *
 * Requirements: batch >= 0, page_size one of 16, 32, 64, 128, 256,
 * n_q_heads a multiple of n_kv_heads with G <= 16, num_pages >= 1,
 * max_kv_len <= max_pages_per_seq * page_size, tensors 16-byte aligned.
 */
fa512_status fa512_decode_paged(const void *q, const void *k_pages, const void *v_pages,
                                const int32_t *page_table, const int32_t *kv_lens, void *out,
                                float *lse, int batch, int n_q_heads, int n_kv_heads,
                                int page_size, int num_pages, int max_pages_per_seq,
                                int max_kv_len, float scale, int window, int num_splits,
                                void *workspace, size_t workspace_bytes,
                                fa512_stream_t stream);

/* Bytes of workspace fa512_decode_paged needs for this shape and split count
 * (num_splits 0 means the automatic choice for max_kv_len).  Returns 0 for an
 * invalid shape. */
size_t fa512_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int page_size,
                                    int max_kv_len, int num_splits);

/*
 * fa512_decode_paged_q -- q_len query tokens per sequence over a paged KV
 * cache: the tokens just appended to each cache (draft tokens being
 * verified, a short chunk), each attending causally to the cache.  The pages
 * list multi-token decode among the next steps of the decode path
 * (vllm-project/flash-attention PR #199, "Notes": varlen Q over a paged
 * cache; "A custom attention kernel for Gemma 4 on the RTX PRO 6000", the
 * draft of 4 tokens).
 *
 *   q    [batch, q_len, n_q_heads, 512] bf16, device
 *   out  [batch, q_len, n_q_heads, 512] bf16, device, written
 *   lse  [batch, q_len, n_q_heads] fp32, device, written; may be NULL
 *   other tensors and arguments as fa512_decode_paged.
 *
 * Query t of sequence b sits at position kv_lens[b] - q_len + t and sees
 * positions [max(0, pos - window + 1), pos] (window <= 0: [0, pos]); a query
 * whose position is negative (kv_lens[b] < q_len) sees nothing and returns
 * O = 0, LSE = -inf.  The workspace must be at least
 * fa512_decode_workspace_bytes_q(batch, q_len, ...) bytes.  Requirements as
 * fa512_decode_paged, plus q_len >= 1 and q_len * (n_q_heads / n_kv_heads)
 * <= 16 (FA512_ERR_UNSUPPORTED otherwise).  q_len = 1 is fa512_decode_paged.
 */
fa512_status fa512_decode_paged_q(const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *page_table, const int32_t *kv_lens, void *out,
                                  float *lse, int batch, int q_len, int n_q_heads, int n_kv_heads,
                                  int page_size, int num_pages, int max_pages_per_seq,
                                  int max_kv_len, float scale, int window, int num_splits,
                                  void *workspace, size_t workspace_bytes,
                                  fa512_stream_t stream);

/* Workspace bytes fa512_decode_paged_q needs (0 for an invalid shape). */
size_t fa512_decode_workspace_bytes_q(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                      int page_size, int max_kv_len, int num_splits);

/*
 * fa512_decode_paged_fp8 -- fa512_decode_paged_q over a paged KV cache
 * stored in FP8 E4M3 (vllm-project/flash-attention PR #199, "Summary": the
 * paged KV cache in FP8; its "Performance" table times the decode shapes
 * with an FP8 cache).
 *
 *   k_pages, v_pages [num_pages, page_size, n_kv_heads, 512] uint8, device:
 *              one OCP E4M3 ("e4m3fn": bias 7, no infinities, S.1111.111
 *              NaN, largest finite 448) byte per element
 *   k_scale, v_scale per-tensor dequantisation scales: key element
 *              k_scale * e4m3(byte), value element v_scale * e4m3(byte)
 *   q, out, lse, positions and every other argument as
 *              fa512_decode_paged_q (q_len >= 1, q_len * G <= 16)
 *   num_splits 0 picks fa512_decode_auto_splits_fp8(); workspace must be
 *              at least fa512_decode_workspace_bytes_fp8() bytes for the
 *              split count used (256-byte aligned).
 *
 * The cache is read as bytes: half the HBM traffic of a bf16 cache.  Every
 * byte is widened exactly (e4m3 -> bf16/fp32) before it meets the bf16
 * query, so the arithmetic is that of fa512_decode_paged_q on the
 * dequantised cache: fp32 accumulation, fp32 softmax state, P rounded to
 * bf16 only on the tensor-core path (q_len * G > 2).  Slots outside the live
 * band are never read (NaN codes there do not reach the output).
 * k_scale and v_scale must be finite (FA512_ERR_INVALID_ARG otherwise).
 */
fa512_status fa512_decode_paged_fp8(const void *q, const void *k_pages, const void *v_pages,
                                    const int32_t *page_table, const int32_t *kv_lens, void *out,
                                    float *lse, int batch, int q_len, int n_q_heads,
                                    int n_kv_heads, int page_size, int num_pages,
                                    int max_pages_per_seq, int max_kv_len, float scale,
                                    float k_scale, float v_scale, int window, int num_splits,
                                    void *workspace, size_t workspace_bytes,
                                    fa512_stream_t stream);

/* Split count chosen when num_splits == 0: enough (batch, KV head, split)
 * work items to fill the current device's SMs about twice, each split at
 * least one page.  Returns 1 when there is nothing to split. */
int fa512_decode_auto_splits(int batch, int n_kv_heads, int page_size, int max_kv_len);

/* Split count fa512_decode_paged_fp8 uses when num_splits == 0.  With
 * q_len * G <= 8 its split kernel runs four CTAs of four warps per SM, one
 * split each, so the choice spreads the keys over four times as many CTAs
 * (at most 128 splits); otherwise it is fa512_decode_auto_splits().  Returns
 * 1 when there is nothing to split. */
int fa512_decode_auto_splits_fp8(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                 int page_size, int max_kv_len);

/* Workspace bytes fa512_decode_paged_fp8 needs for this shape and split
 * count (num_splits 0: fa512_decode_auto_splits_fp8).  0 for an invalid
 * shape. */
size_t fa512_decode_workspace_bytes_fp8(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                        int page_size, int max_kv_len, int num_splits);

/*
 * fa512_decode_paged_noalloc -- fa512_decode_paged without a workspace
 * argument.  (The pages have no counterpart: this is a convenience of the
 * library, not a step of the method.)
 *
 * For callers that cannot call cudaMalloc: code that only receives device
 * pointers for its inputs and outputs from another framework and has no
 * allocator of its own, or that runs where every byte of device memory
 * belongs to a pool it does not control.  The (O, m, l) split partials go to
 * a file-scope device array of FA512_DECODE_STATIC_SCRATCH_BYTES that the
 * library holds on every GPU it is loaded on until the process exits.  The
 * call allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 * routine.
 *
 * Arguments, layouts and errors are those of fa512_decode_paged.  A shape
 * whose partials need more than FA512_DECODE_STATIC_SCRATCH_BYTES
 * (fa512_decode_workspace_bytes) is rejected with FA512_ERR_WORKSPACE before
 * anything is enqueued; lower num_splits or the batch to fit.
 *
 * The first call on a device looks up the array's device address on that
 * device (cudaGetSymbolAddress, with that device current) and keeps it for
 * the life of the process; make that first call before any stream capture.
 * The kept address does not survive a device reset (cudaDeviceReset or a
 * reset of the primary context): do not use the library across one.  All calls share the one array and it
 * keeps the last call's contents; nothing in it has to start at zero, since
 * every split writes its whole partial before the merge reads it.  Calls
 * whose kernels overlap on the GPU (different streams, or different host
 * threads without ordering) race on the array: order them.
 */
#define FA512_DECODE_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)

fa512_status fa512_decode_paged_noalloc(const void *q, const void *k_pages,
                                        const void *v_pages, const int32_t *page_table,
                                        const int32_t *kv_lens, void *out, float *lse,
                                        int batch, int n_q_heads, int n_kv_heads, int page_size,
                                        int num_pages, int max_pages_per_seq, int max_kv_len,
                                        float scale, int window, int num_splits,
                                        fa512_stream_t stream);

/*
 * fa512_decode_paged_tree -- the drafted tokens of each sequence over a paged
 * KV cache that already holds their keys and values.
 *
 *   q          [batch, q_len, n_q_heads, 512] bf16, device
 *   k_pages, v_pages, page_table, kv_lens as fa512_decode_paged
 *   q_lens     [batch] int32, device: drafted tokens of sequence b, its last
 *              q_lens[b] cached positions; NULL: q_len for every sequence
 *   tree_mask  [batch, q_len, ceil(q_len / 32)] int32, device: bit j % 32 of
 *              word j / 32 of row t says that token t sees token j; NULL: a
 *              plain run of tokens (token t sees tokens 0 .. t)
 *   out        [batch, q_len, n_q_heads, 512] bf16, device, written
 *   lse        [batch, q_len, n_q_heads] fp32, device, written; may be NULL
 *
 * With start = kv_lens[b] - q_lens[b], token t's key is cached at position
 * start + t.  Every token sees the positions before start and the tokens its
 * mask names (usually itself and the tokens on its way to the root).  The
 * place of a cached key is its position; the place of token t is start + d,
 * d the number of tokens it sees less one: in a tree, its depth.  With
 * window > 0 a key is visible only if its place is above the token's own
 * place less window, or below n_sinks (the first positions, which stay
 * visible whatever the window).  Rows of tokens from q_lens[b] on, and of
 * tokens whose cached position would be negative, see nothing: O = 0,
 * LSE = -inf.
 *
 * A row is a (token, query head) pair.  Up to 64 rows of a KV head share one
 * pass over its keys in one CTA; more are taken in groups of 128, each on a
 * pair of SMs.  The keys of all sequences are cut into ranges of equal length
 * (or each item's into equal segments), one per CTA or pair, so num_splits is
 * the most segments that one row may be left in (1: no row is split; 0: at
 * most fa512_decode_auto_splits_tree()).  Only
 * pages that hold positions inside the band of some row are read; slots that
 * no row sees may hold anything (NaN included) without reaching the output.
 * A row that sees a score of NaN or +infinity is NaN, as is, over an E4M3
 * cache, a row whose query holds an infinity.
 * Without a mask and sinks the older calls do the same: fa512_decode_paged_q and
 * _fp8 (up to 16 rows) are faster for one sequence with a few tokens,
 * fa512_prefill_paged (bf16, pages of 64 and more) from some hundred rows of a KV
 * head on.  max_kv_len also bounds how evenly the keys are dealt out: give it as
 * tightly as the host knows it.
 * The same inputs give the same bits every time.  out, lse and workspace must
 * not overlap the inputs or one another; calls that may run at the same time
 * need workspaces of their own.
 *
 * workspace must be at least fa512_decode_workspace_bytes_tree() bytes for
 * the split count used, 256-byte aligned; with one split it is not used and
 * may be NULL.
 *
 * Requirements: q_len >= 1 (at most 256 with a tree_mask), page_size one of
 * 16, 32, 64, 128, 256, n_q_heads a multiple of n_kv_heads with G <= 128,
 * num_pages >= 1, max_kv_len <= max_pages_per_seq * page_size, n_sinks >= 0
 * (it only matters with window > 0), batch and n_kv_heads at most 65535, and
 * with more than one split batch * q_len <= 65535.  On the device, kv_lens[b]
 * outside [0, max_kv_len], q_lens[b] outside [0, q_len] and page indices
 * outside the pool are recorded in the error word and clipped or read as
 * zeros.
 */
fa512_status fa512_decode_paged_tree(const void *q, const void *k_pages, const void *v_pages,
                                     const int32_t *page_table, const int32_t *kv_lens,
                                     const int32_t *q_lens, const int32_t *tree_mask, void *out,
                                     float *lse, int batch, int q_len, int n_q_heads,
                                     int n_kv_heads, int page_size, int num_pages,
                                     int max_pages_per_seq, int max_kv_len, float scale,
                                     int window, int n_sinks, int num_splits, void *workspace,
                                     size_t workspace_bytes, fa512_stream_t stream);

/* The same over a cache stored in FP8 E4M3 (as fa512_decode_paged_fp8: a key
 * element is k_scale * e4m3(byte), a value element v_scale * e4m3(byte)). */
fa512_status fa512_decode_paged_tree_fp8(const void *q, const void *k_pages, const void *v_pages,
                                         const int32_t *page_table, const int32_t *kv_lens,
                                         const int32_t *q_lens, const int32_t *tree_mask,
                                         void *out, float *lse, int batch, int q_len,
                                         int n_q_heads, int n_kv_heads, int page_size,
                                         int num_pages, int max_pages_per_seq, int max_kv_len,
                                         float scale, float k_scale, float v_scale, int window,
                                         int n_sinks, int num_splits, void *workspace,
                                         size_t workspace_bytes, fa512_stream_t stream);

/* Split count of the tree calls when num_splits == 0: the segments that the
 * longest sequence's row can be left in when the current device's SMs share
 * the keys of max_kv_len equally, twice over for batches with shorter
 * sequences.  Returns 1 when there is nothing to split. */
int fa512_decode_auto_splits_tree(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                  int max_kv_len, int window, int n_sinks);

/* Workspace bytes of the tree calls for this shape and split count
 * (num_splits 0: the automatic choice); at least 256 for a valid shape, 0
 * for an invalid one.  Whatever the shape, not more than 64 MB and 8 bytes for
 * each (sequence, row group, KV head), with less than 1 KB of rounding. */
size_t fa512_decode_workspace_bytes_tree(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                         int max_kv_len, int window, int n_sinks, int num_splits);

/*
 * fa512_cache_append -- writes the newest tokens' keys and values into the
 * pages of a cache.
 *
 *   k_new, v_new [batch, q_len, n_kv_heads, 512] bf16, device; the heads of a
 *                token are contiguous, sequences and tokens are
 *                k_batch_stride / v_batch_stride and k_token_stride /
 *                v_token_stride elements apart (multiples of 8), so slices of
 *                a fused projection's output need no copy
 *   k_pages, v_pages as fa512_decode_paged, written
 *   kv_lens      [batch] int32, device: cached positions of sequence b, the
 *                new tokens included
 *   q_lens       [batch] int32, device: new tokens of sequence b; NULL: q_len
 *
 * Token t of sequence b goes to position kv_lens[b] - q_lens[b] + t; tokens
 * from q_lens[b] on are padding and are not written.  Nothing else in the
 * pages is touched.  Two positions that share a slot are the caller's error;
 * a slot of a page that several sequences hold is written for all of them (see
 * fa512_cache_resize).
 * On the device, q_lens[b] outside [0, q_len], positions outside
 * [0, max_pages_per_seq * page_size) and page indices outside the pool are
 * recorded in the error word and their rows are not written.
 */
fa512_status fa512_cache_append(const void *k_new, const void *v_new, int64_t k_batch_stride,
                                int64_t k_token_stride, int64_t v_batch_stride,
                                int64_t v_token_stride, void *k_pages, void *v_pages,
                                const int32_t *page_table, const int32_t *kv_lens,
                                const int32_t *q_lens, int batch, int q_len, int n_kv_heads,
                                int page_size, int num_pages, int max_pages_per_seq,
                                fa512_stream_t stream);

/* The same into an FP8 E4M3 cache: the byte of x is the E4M3 value nearest to
 * x / k_scale (x / v_scale), ties to even, values beyond +-448 stored as
 * +-448, NaN as the NaN code.  The scales must be finite and above 0. */
fa512_status fa512_cache_append_fp8(const void *k_new, const void *v_new, int64_t k_batch_stride,
                                    int64_t k_token_stride, int64_t v_batch_stride,
                                    int64_t v_token_stride, void *k_pages, void *v_pages,
                                    const int32_t *page_table, const int32_t *kv_lens,
                                    const int32_t *q_lens, float k_scale, float v_scale,
                                    int batch, int q_len, int n_kv_heads, int page_size,
                                    int num_pages, int max_pages_per_seq, fa512_stream_t stream);

/*
 * fa512_cache_append_fp4 -- the same into a cache held in 4 bits an element.
 *
 *   k_pages, v_pages [num_pages, page_size, n_kv_heads, FA512_FP4_ROW_BYTES]
 *                uint8, device.  The row of a head at a position is 256 bytes of
 *                E2M1 codes, element 2 i in the low half of byte i and element
 *                2 i + 1 in the high half, then 32 E4M3 scales, the one in byte
 *                256 + j for elements 16 j .. 16 j + 15.  An E2M1 code is a sign
 *                bit and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 in the order of its
 *                three lower bits.  Key element = k_scale * scale * code, value
 *                element = v_scale * scale * code.
 *
 * With y = x / k_scale (x / v_scale), the nearest fp32 quotient, the scale of a
 * group is the E4M3 value nearest to max |y| / 6 and a code the E2M1 value
 * nearest to the fp32 quotient y / scale; ties to even, beyond the largest value
 * the largest value.  A group whose scale rounds to 0 (max |y| up to 6 * 2^-10)
 * gets codes 0.  A group that holds a NaN gets the NaN scale and codes 0: all its
 * elements read as NaN.  k_scale and v_scale are finite and above 0; where both are
 * powers of two the call is faster (8 sequences of up to 4,096 tokens, 4 heads: 55 us,
 * else 147), and the choice only matters for what lies outside the scales' range.
 * Other arguments and errors as fa512_cache_append.
 */
#define FA512_FP4_ROW_BYTES 288

fa512_status fa512_cache_append_fp4(const void* k_new, const void* v_new, int64_t k_batch_stride,
                                    int64_t k_token_stride, int64_t v_batch_stride,
                                    int64_t v_token_stride, void* k_pages, void* v_pages,
                                    const int32_t* page_table, const int32_t* kv_lens,
                                    const int32_t* q_lens, float k_scale, float v_scale,
                                    int batch, int q_len, int n_kv_heads, int page_size,
                                    int num_pages, int max_pages_per_seq, fa512_stream_t stream);

/*
 * fa512_decode_paged_fp4 -- fa512_decode_paged_q over a paged KV cache held in 4
 * bits an element, in the rows of fa512_cache_append_fp4: 576 bytes of K and V a
 * position and KV head instead of bf16's 2,048.
 *
 *   k_scale, v_scale per-tensor scales, finite
 *   q, out, lse, positions and every other argument as fa512_decode_paged_q
 *              (q_len >= 1, q_len * G <= 16)
 *   num_splits most pieces that a sequence may be cut into, at most 1024 (the
 *              SMs take equal ranges of the keys of all sequences; 1: whole
 *              sequences); 0 picks fa512_decode_auto_splits_fp4(), which is for
 *              lengths of half of max_kv_len and more.  Give max_kv_len as tightly
 *              as the host knows it; where the lengths are much shorter, or few of
 *              many are long, 1024 spreads the keys over all SMs (64 sequences of
 *              4,096 positions: 101 us with that bound, 511 with 131,072, 117 with
 *              1024) at the price of a larger workspace; workspace
 *              must be at least fa512_decode_workspace_bytes_fp4() bytes,
 *              256-byte aligned, not shared by calls that may run at the same time
 *
 * Codes and group scales are widened exactly, the queries (bf16) scaled by a
 * power of two per row and held in f16, sums are fp32; the softmax weights round
 * to f16: to 11 bits, or, below 2^-16 of the row's largest, within 2^-26 of that,
 * whatever the group scales of their values.  Slots that no row sees may hold anything without reaching the output;
 * a value that is not finite in a slot that one row of a KV head sees may reach
 * the head's other rows.  A row that sees a score of NaN or +infinity is NaN.  The
 * same inputs give the same bits every time.  batch * q_len is at most 65535, and
 * so is n_kv_heads; num_pages * page_size and max_pages_per_seq * page_size are
 * below 2^31 - 4096, batch * max_kv_len is at most 2^34.
 */
fa512_status fa512_decode_paged_fp4(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* page_table, const int32_t* kv_lens, void* out,
                                    float* lse, int batch, int q_len, int n_q_heads,
                                    int n_kv_heads, int page_size, int num_pages,
                                    int max_pages_per_seq, int max_kv_len, float scale,
                                    float k_scale, float v_scale, int window, int num_splits,
                                    void* workspace, size_t workspace_bytes,
                                    fa512_stream_t stream);

/* num_splits of fa512_decode_paged_fp4 when it is 0; 1 when there is nothing to
 * split. */
int fa512_decode_auto_splits_fp4(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                 int page_size, int max_kv_len);

/* Workspace bytes fa512_decode_paged_fp4 needs for this shape and split count
 * (num_splits 0: the automatic choice).  0 for an invalid shape. */
size_t fa512_decode_workspace_bytes_fp4(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                        int page_size, int max_kv_len, int num_splits);

/*
 * fa512_cache_page_bounds -- the smallest and the largest key element of each
 * channel, of the pages that hold the newest tokens.
 *
 *   k_pages      [num_pages, page_size, n_kv_heads, 512] bf16 (element_bits 16)
 *                or E4M3 (8), or [..., FA512_FP4_ROW_BYTES] bytes (4), device
 *   page_table   [batch, max_pages_per_seq], kv_lens [batch] int32, device
 *   q_lens       [batch] int32, device: newest tokens of sequence b; NULL: q_len
 *   bounds       [num_pages, n_kv_heads, 2, 512] bf16, device, written: smallest,
 *                largest
 *
 * The pages of positions kv_lens[b] - q_lens[b] .. kv_lens[b] - 1 are read, up to
 * position kv_lens[b] - 1, and their bounds written; no others.  Of a coded cache
 * the bounds are those of what is stored, without the tensor scale; they are
 * exact.  A channel with a NaN has NaN bounds.  Call it after each append (with
 * the same kv_lens and q_lens), after fa512_cache_compact (with the new lengths)
 * and, with a q_len of 1, after fa512_cache_fork.  A page that several sequences
 * hold gets its bounds from each call that names it: give it no sequence that
 * ends inside a page that others hold beyond.
 * On the device, q_lens[b] outside [0, q_len], kv_lens[b] below it or beyond the
 * page table and page indices outside the pool are recorded in the error word
 * and skipped.
 */
fa512_status fa512_cache_page_bounds(const void* k_pages, const int32_t* page_table,
                                     const int32_t* kv_lens, const int32_t* q_lens, void* bounds,
                                     int batch, int q_len, int n_kv_heads, int element_bits,
                                     int page_size, int num_pages, int max_pages_per_seq,
                                     fa512_stream_t stream);

/*
 * fa512_select_pages -- the pages that a sparse decode step reads.
 *
 *   q          [batch, q_len, n_q_heads, 512] bf16, device
 *   bounds     [num_pages, n_kv_heads, 2, 512] bf16, device
 *   page_table, kv_lens, max_kv_len as fa512_decode_paged_q
 *   selected   [batch, n_kv_heads, n_select] int32, device, written: logical pages
 *              of the sequence in rising order, then -1
 *
 * The score of page p for a KV head is the largest, over its query rows (token,
 * query head), of sum_d max(q_d lo_d, q_d hi_d): with lo and hi the page's bounds,
 * no product of the row with a key of the page is larger.  Selected are the
 * n_first first and the n_last last pages of the sequence, and of the others
 * those with the largest scores, equal ones by their number, n_select in all; of
 * a sequence with no more pages, all.  (The page that is filling and those of
 * drafted tokens are among the last: n_last counts them.)  Rows whose position
 * kv_lens[b] - q_len + t is negative are left out.  A page with a bound that is
 * not finite comes before all others; one whose index lies outside the pool
 * comes last and is recorded in the error word.  A NaN in a row that counts makes
 * all scores of its KV head equal.
 *
 * Sums are fp32 in a fixed order (channels c and c + 256, then c % 8 by halves,
 * then c / 8 by halves), so the choice is the same for every launch shape.
 *
 * Requirements: q_len * G <= 16, page_size one of 16, 32, 64, 128, 256, n_first +
 * n_last <= n_select; workspace of fa512_select_workspace_bytes() bytes, 256-byte
 * aligned, not shared by calls that may run at the same time.
 */
fa512_status fa512_select_pages(const void* q, const void* bounds, const int32_t* page_table,
                                const int32_t* kv_lens, int32_t* selected, int batch, int q_len,
                                int n_q_heads, int n_kv_heads, int page_size, int num_pages,
                                int max_pages_per_seq, int max_kv_len, int n_select, int n_first,
                                int n_last, void* workspace, size_t workspace_bytes,
                                fa512_stream_t stream);

/* Workspace bytes of fa512_select_pages; 0 for an invalid shape. */
size_t fa512_select_workspace_bytes(int batch, int n_kv_heads, int page_size, int max_kv_len);

/*
 * fa512_decode_paged_sparse -- fa512_decode_paged_q over some pages of each
 * sequence.
 *
 *   selected   [batch, n_kv_heads, n_selected] int32, device: the logical pages
 *              that the rows of a KV head see, rising, then -1
 *   other tensors and arguments as fa512_decode_paged_q
 *
 * Query t of sequence b sits at position kv_lens[b] - q_len + t and sees the
 * positions up to its own that lie in a selected page.  Only those pages are
 * read.  A row that sees nothing returns O = 0, LSE = -inf.
 * Entries that do not rise, follow a -1 or lie outside the sequence's pages are
 * recorded in the error word; nothing is read out of bounds for them, but the
 * outputs of their (sequence, KV head) mean nothing.
 *
 * num_splits and workspace as fa512_decode_paged_fp4: 0 picks
 * fa512_decode_auto_splits_sparse(), the workspace holds at least
 * fa512_decode_workspace_bytes_sparse() bytes.  Slots that no row sees, and
 * scores and values that are not finite, as there; weights too over coded caches,
 * over bf16 they round to bf16.
 * n_selected >= 1; n_selected * page_size, num_pages * page_size and
 * max_pages_per_seq * page_size are below 2^31 - 4096, batch * q_len and n_kv_heads
 * at most 65535, batch times the positions of a list at most 2^34.
 */
fa512_status fa512_decode_paged_sparse(const void* q, const void* k_pages, const void* v_pages,
                                       const int32_t* page_table, const int32_t* kv_lens,
                                       const int32_t* selected, void* out, float* lse, int batch,
                                       int q_len, int n_q_heads, int n_kv_heads, int page_size,
                                       int num_pages, int max_pages_per_seq, int n_selected,
                                       int max_kv_len, float scale, int num_splits, void* workspace,
                                       size_t workspace_bytes, fa512_stream_t stream);

/* The same over a cache in FP8 E4M3 (as fa512_decode_paged_fp8). */
fa512_status fa512_decode_paged_sparse_fp8(const void* q, const void* k_pages, const void* v_pages,
                                           const int32_t* page_table, const int32_t* kv_lens,
                                           const int32_t* selected, void* out, float* lse, int batch,
                                           int q_len, int n_q_heads, int n_kv_heads, int page_size,
                                           int num_pages, int max_pages_per_seq, int n_selected,
                                           int max_kv_len, float scale, float k_scale, float v_scale,
                                           int num_splits, void* workspace, size_t workspace_bytes,
                                           fa512_stream_t stream);

/* The same over a cache in 4 bits (as fa512_decode_paged_fp4). */
fa512_status fa512_decode_paged_sparse_fp4(const void* q, const void* k_pages, const void* v_pages,
                                           const int32_t* page_table, const int32_t* kv_lens,
                                           const int32_t* selected, void* out, float* lse, int batch,
                                           int q_len, int n_q_heads, int n_kv_heads, int page_size,
                                           int num_pages, int max_pages_per_seq, int n_selected,
                                           int max_kv_len, float scale, float k_scale, float v_scale,
                                           int num_splits, void* workspace, size_t workspace_bytes,
                                           fa512_stream_t stream);

/* Split count and workspace bytes of the sparse calls; element_bits 16 (bf16), 8
 * (E4M3) or 4.  1 and 0 for an invalid shape. */
int fa512_decode_auto_splits_sparse(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                    int element_bits, int page_size, int n_selected,
                                    int max_kv_len);
size_t fa512_decode_workspace_bytes_sparse(int batch, int q_len, int n_q_heads, int n_kv_heads,
                                           int element_bits, int page_size, int n_selected,
                                           int max_kv_len, int num_splits);

/*
 * fa512_cache_compact -- after a verification step: moves the accepted
 * tokens' rows together, in all layers of a cache.
 *
 *   k_pages, v_pages [n_layers, num_pages, page_size, n_kv_heads, 512] of
 *                element_bytes 1 (E4M3) or 2 (bf16), or rows of
 *                FA512_FP4_ROW_BYTES bytes instead (FA512_ELEMENT_FP4), device,
 *                written
 *   kv_lens      [batch] int32, device: cached positions, the q_lens[b]
 *                (NULL: q_len) drafted tokens included
 *   accepted     [batch, max_accepted] int32, device: the accepted tokens of
 *                sequence b in rising order, each in [0, q_lens[b])
 *   n_accepted   [batch] int32, device: how many
 *   new_kv_lens  [batch] int32, device, written: start + n_accepted[b], with
 *                start = kv_lens[b] - q_lens[b]; must not overlap the inputs
 *
 * The row of token accepted[b, i] moves to position start + i.  Rows behind
 * the new length keep what they held.  A sequence whose entries do not rise
 * inside [0, q_lens[b]), whose n_accepted[b] is outside
 * [0, min(max_accepted, q_lens[b])] or whose lengths are impossible is
 * recorded in the error word; it is left as it is, its new length kv_lens[b].
 * A row that would move from or to a page outside the pool is recorded too and
 * stays where it is; the sequence's other rows move and its new length is the
 * usual one.  max_accepted is at most 1024.
 */
#define FA512_ELEMENT_FP4 (-4)

fa512_status fa512_cache_compact(void *k_pages, void *v_pages, const int32_t *page_table,
                                 const int32_t *kv_lens, const int32_t *q_lens,
                                 const int32_t *accepted, const int32_t *n_accepted,
                                 int32_t *new_kv_lens, int n_layers, int batch, int q_len,
                                 int max_accepted, int n_kv_heads, int element_bytes,
                                 int page_size, int num_pages, int max_pages_per_seq,
                                 fa512_stream_t stream);

/*
 * fa512_cache_fork -- replaces the sequences of a cache by children of them
 * (beam search, several samples of one prompt, dropped sequences), in all
 * layers at once.
 *
 *   k_pages, v_pages as fa512_cache_compact, written where pages are copied
 *   page_table   [batch, max_pages_per_seq], kv_lens [batch] int32, device
 *   parents      [n_children] int32, device: the sequence child c continues
 *   page_refs    [num_pages] int32, device: how many sequences (and other
 *                holders) refer to each page; 0 is free
 *   new_page_table [n_children, max_pages_per_seq], new_kv_lens [n_children],
 *   new_page_refs [num_pages] int32, device, written; new_page_refs may be
 *                page_refs itself, the other two must not overlap the inputs; no two of
 *                the three may overlap
 *
 * A sequence of n positions holds its first ceil(n / page_size) entries.
 * Child c shares the pages of parents[c].  A last page that is only partly
 * filled goes to the first child of its parent, whoever else holds it; every
 * other child gets a free page of its own with the filled rows copied, the
 * lowest free pages in the order of the children.  Table entries that a child
 * does not hold are -1.
 * The counts lose one for each entry the old sequences held and gain one for
 * each the children hold; pages whose count comes to 0 are free, also within
 * this call.  When the free pages do not suffice, the children without one
 * get -1 there and FA512_ERR_OUT_OF_PAGES is recorded in the error word.
 * Parents outside [0, batch), lengths outside the table and page indices
 * outside the pool are recorded too: such a child is empty, such a length is
 * clipped, such a page is -1 in the new table and not counted.
 *
 * batch and n_children are at most 8192.
 */
fa512_status fa512_cache_fork(void *k_pages, void *v_pages, const int32_t *page_table,
                              const int32_t *kv_lens, const int32_t *parents,
                              const int32_t *page_refs, int32_t *new_page_table,
                              int32_t *new_kv_lens, int32_t *new_page_refs, int n_layers,
                              int batch, int n_children, int n_kv_heads, int element_bytes,
                              int page_size, int num_pages, int max_pages_per_seq,
                              fa512_stream_t stream);

/*
 * fa512_cache_resize -- gives each sequence the pages of its new length and
 * takes back those behind it.
 *
 *   page_table [batch, max_pages_per_seq], kv_lens [batch], new_kv_lens
 *   [batch], page_refs [num_pages] int32, device
 *   new_page_table, new_page_refs: like page_table and page_refs, written;
 *                each may be its input itself
 *
 * Sequence b holds its first ceil(kv_lens[b] / page_size) entries before and
 * ceil(new_kv_lens[b] / page_size) after the call.  Entries that it gives up
 * become -1 and the count of their page falls by one; then the entries that
 * it gains get the lowest pages whose count is 0, in the order of (sequence,
 * entry), with a count of 1.  All other entries behind the new length are -1.
 * Pages of a full pool, bad lengths and bad pages as fa512_cache_fork.
 * new_kv_lens 0 ends a sequence.  batch is at most 8192.
 *
 * The counts say how many hold a page, not which of its rows.  A sequence that
 * is shortened to inside a page that others hold too (it was whole when a fork
 * shared it) keeps that page, and appending to the sequence then would write
 * over their rows.  To let it grow, fork it into two children: the second has
 * a page of its own with its rows, and the first is ended with a length of 0.
 */
fa512_status fa512_cache_resize(const int32_t *page_table, const int32_t *kv_lens,
                                const int32_t *new_kv_lens, const int32_t *page_refs,
                                int32_t *new_page_table, int32_t *new_page_refs, int batch,
                                int page_size, int num_pages, int max_pages_per_seq,
                                fa512_stream_t stream);

/*
 * fa512_test_prefill_missing_load -- test hook, not a step of the method.
 * (The pages have no counterpart: it exists so that tests can drive the
 * kernels' bounded waits, which ordinary inputs never exhaust.)
 *
 * The same launch as fa512_prefill with the same arguments, except that
 * (a) every pipeline wait of the kernel is bounded by wait_limit_ns instead
 * of the default 2 s, and (b) the first CTA pair's even CTA does not issue
 * its first K tile load, so that pair's waits for it run into the bound.
 * The pair then records FA512_ERR_TIMEOUT in the device error word, drains
 * the MMAs it issued, frees its tensor memory and returns; CTAs that start
 * after the record skip their work.  The rows of the pair (and of skipped
 * CTAs) are left unwritten.  The device stays usable: read the status with
 * fa512_device_status(stream, 1) (which also clears it) before the next call.
 *
 * wait_limit_ns must lie in [1e6, 2e9] and seqlen_k must be >= 1
 * (FA512_ERR_INVALID_ARG otherwise); other errors as for fa512_prefill.
 */
fa512_status fa512_test_prefill_missing_load(const void *q, const void *k, const void *v,
                                             void *out, float *lse, int seqlen_q, int seqlen_k,
                                             int q_offset, int n_q_heads, int n_kv_heads,
                                             float scale, int causal, int window,
                                             uint64_t wait_limit_ns, fa512_stream_t stream);

/* Reads and optionally clears the device-side error word after
 * synchronising `stream`.  Returns FA512_OK, FA512_ERR_TIMEOUT,
 * FA512_ERR_DEVICE_INDEX, FA512_ERR_OUT_OF_PAGES or FA512_ERR_CUDA. */
fa512_status fa512_device_status(fa512_stream_t stream, int clear);

/* Static, human-readable name of a status code. */
const char *fa512_status_string(fa512_status status);

/* Detail of the last error returned on the calling thread (static storage,
 * overwritten by the next failing call). */
const char *fa512_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* FA512_H */
