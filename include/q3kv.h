/*
 * q3kv -- speculative-verify attention over a 3-bit, Walsh-Hadamard-rotated,
 * paged KV cache.  C ABI of the shared library libq3kv.so (sm_103a).
 *
 * Source of the method: the "Quasar" (q27) engine wiki --
 *   - "turbo3 3-bit KV cache" bullet and the "KV cache" stack bullet: K and V
 *     are WHT-rotated and stored as 3-bit codes in fixed-size blocks,
 *     symmetric for K and V, per slot;
 *   - "Self-speculation as the whole design": all drafted tokens of a step are
 *     checked in one shared-KV verify pass;
 *   - "Width-12 verify": up to 12 tokens per step (this library takes up to 16);
 *   - "Continuous batching": several slots go through one fused round.
 * The pages give no bit-level codec and no kernel for this GPU.  The codec
 * here is this library's own (head_dim 256; y = H x in float32 with H the
 * orthonormal Sylvester-Hadamard matrix; 8 blocks of 32; per block an fp16
 * scale s = absmax/3.5 and codes q = clamp(rint(y/s + 3.5), 0, 7); value
 * (q - 3.5) s; 112 bytes per vector).  Queries are rotated by the same H; the
 * output is rotated back, so callers see ordinary attention outputs.
 *
 * Conventions for every call:
 *   - Return value: Q3KV_OK (0) or a negative Q3KV_ERR_* code.  Nothing is
 *     launched when an argument check fails.
 *   - Device-side problems (a page id outside [0, num_pages), a length beyond
 *     the slot's page table, a non-finite input, an fp16 scale overflow) never
 *     trap: the kernel ORs a Q3KV_STATUS_* bit into *d_status and skips the
 *     offending unit.  d_status may be NULL to ignore them.
 *   - All device work is asynchronous on the given stream.  Pointers prefixed
 *     d_ are device pointers; h_ are host pointers.  The library allocates no
 *     device memory: the caller owns the pool, page tables, lengths, inputs,
 *     outputs, workspace and status word.
 *   - Lengths are owned by the caller.  Rolling back rejected drafts is a
 *     smaller length on the next call; stale records are overwritten by the
 *     next append.
 */
#ifndef Q3KV_H
#define Q3KV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define Q3KV_API __attribute__((visibility("default")))
#else
#define Q3KV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define Q3KV_FORMAT_VERSION 1   /* bumps when the record or page layout changes */

/* error codes (return values) */
#define Q3KV_OK                      0
#define Q3KV_ERR_INVALID_ARG        -1
#define Q3KV_ERR_UNSUPPORTED        -2
#define Q3KV_ERR_OUT_OF_PAGES       -3
#define Q3KV_ERR_WORKSPACE_TOO_SMALL -4
#define Q3KV_ERR_CUDA               -5
#define Q3KV_ERR_SLOT_RANGE         -6
#define Q3KV_ERR_HOST_MEMORY        -7   /* host allocation of the page allocator failed */

/* device status bits (*d_status) */
#define Q3KV_STATUS_NONFINITE_INPUT  1
#define Q3KV_STATUS_SCALE_OVERFLOW   2
#define Q3KV_STATUS_BAD_PAGE         4
#define Q3KV_STATUS_BAD_LENGTH       8
#define Q3KV_STATUS_TIMEOUT         16   /* a bounded wait inside a kernel gave up */
#define Q3KV_STATUS_RANGE           32   /* tensor-core leg: a block scale above 5458
                                            (its exact fp16 dequantisation needs
                                            12 s in fp16 range) */
#define Q3KV_STATUS_BAD_TOKEN       64   /* a token id outside [0, vocab), or biases not in
                                            ascending order of their tokens */

/* input dtypes */
#define Q3KV_F32   0
#define Q3KV_BF16  1

/* verify implementations */
#define Q3KV_IMPL_AUTO  0   /* the fastest one that supports the shape          */
#define Q3KV_IMPL_FMA   1   /* CUDA-core fp32 FMA flash-decode (reference leg)   */
#define Q3KV_IMPL_MMA   2   /* tcgen05 tensor-core leg (fp16 hi/lo operand pairs,
                               fp32 accumulation); needs block scales <= 5458   */

/* Shape of one cache pool.  Supported: head_dim 256, page_size 256,
 * num_q_heads = 8 * num_kv_heads (GQA group of 8), num_kv_heads >= 1. */
typedef struct q3kv_cache_desc {
    int32_t num_layers;
    int32_t num_kv_heads;
    int32_t num_q_heads;
    int32_t head_dim;    /* 256 */
    int32_t page_size;   /* 256 */
    int32_t num_pages;
} q3kv_cache_desc;

/* Library and layout versions. */
Q3KV_API int q3kv_version(void);
Q3KV_API int q3kv_format_version(void);

/* Text of an error code (static string, never NULL). */
Q3KV_API const char* q3kv_strerror(int err);

/* Text of the last CUDA failure behind a Q3KV_ERR_CUDA return on the calling
 * host thread (static string, never NULL). */
Q3KV_API const char* q3kv_last_cuda_error(void);

/* Bytes of a pool for desc:
 *   num_pages * num_layers * num_kv_heads * 2 * page_size * 112.
 * Pool layout: the 112-byte record of (page, layer, kv_head, kv in {0:K, 1:V},
 * row = position % 256) starts at
 *   ((((page*num_layers + layer)*num_kv_heads + kv_head)*2 + kv)*256 + row)*112.
 * Record: 24 little-endian uint32 code words (three per 32-element block; in
 * block b, element e < 30 is pair m = e/2, half = e%2, in word 3b + m/5 at bit
 * 16*half + 3*(m%5); element 30 keeps code bit k in bit 15 of word 3b+k and
 * element 31 in bit 31), then 8 fp16 scales.  The pool must be 16-byte aligned. */
Q3KV_API int q3kv_pool_bytes(const q3kv_cache_desc* desc, size_t* bytes);

/* ---- host page allocator (no device work) --------------------------------
 * Source: per-slot KV of the "turbo3 3-bit KV cache" bullet, and the
 * PagedAttention paragraph of the prefix-reuse section (a pool of fixed-size
 * blocks).  Pages are 256 positions.  The allocator owns only host state. */
typedef struct q3kv_allocator q3kv_allocator;

/* Create an allocator over page ids [0, num_pages) for num_slots slots whose
 * page-table rows hold max_pages_per_slot entries.  *out receives the handle.
 * Q3KV_ERR_HOST_MEMORY if its host arrays cannot be allocated (no C++
 * exception leaves any call of this library). */
Q3KV_API int q3kv_allocator_create(int32_t num_pages, int32_t num_slots, int32_t max_pages_per_slot,
                          q3kv_allocator** out);
Q3KV_API void q3kv_allocator_destroy(q3kv_allocator* a);

/* Make slot hold pages for n_positions positions (ceil(n/256) pages), taking
 * new pages from the free list.  Writes the slot's page ids into the caller's
 * host row h_page_table_row[0 .. *n_pages_out) (length max_pages_per_slot;
 * entries past the count are set to -1).  Never shrinks.  All or nothing: on
 * Q3KV_ERR_OUT_OF_PAGES or Q3KV_ERR_HOST_MEMORY nothing changes. */
Q3KV_API int q3kv_alloc_pages(q3kv_allocator* a, int32_t slot, int64_t n_positions,
                     int32_t* h_page_table_row, int32_t* n_pages_out);

/* Return all pages of slot to the free list. */
Q3KV_API int q3kv_free_slot(q3kv_allocator* a, int32_t slot);

/* Free pages left. */
Q3KV_API int q3kv_free_pages(const q3kv_allocator* a, int32_t* n_free);

/* ---- shared pages: forks, copies on write, trimming, compaction -------------------
 * Source: the same PagedAttention paragraph (blocks are immutable once full, so
 * requests with one prefix can hold the same blocks).  A page may be held by several slots; it
 * returns to the free list when the last of them lets it go.  These calls only keep the books
 * (no device work): q3kv_copy_pages moves the bytes.  Each writes a page-table row as
 * q3kv_alloc_pages does, and changes nothing when it returns an error. */

/* The row of a slot as it is now. */
Q3KV_API int q3kv_slot_pages(const q3kv_allocator* a, int32_t slot, int32_t* h_page_table_row, int32_t* n_pages_out);

/* Make dst_slot, which must hold no page, share the pages of src_slot's first n_positions
 * positions (Q3KV_ERR_INVALID_ARG if dst_slot holds pages or src_slot fewer). */
Q3KV_API int q3kv_fork_slot(q3kv_allocator* a, int32_t src_slot, int32_t dst_slot, int64_t n_positions,
                     int32_t* h_page_table_row, int32_t* n_pages_out);

/* Before slot writes positions [first_position, first_position + n_positions): make it hold
 * pages up to there (as q3kv_alloc_pages) and own those of the range alone.  A page of the range
 * that another slot holds too is replaced by a fresh one.  Only the page that the range begins
 * inside keeps earlier positions: where that one is replaced, h_copy = {old page, new page,
 * number of positions to copy}, for q3kv_copy_pages before the write and before any call that
 * reads the new row; else h_copy = {-1, -1, 0}.  Positions behind the range in a replaced page
 * are lost to this slot (a write at position n is an append to a slot of length n). */
Q3KV_API int q3kv_write_pages(q3kv_allocator* a, int32_t slot, int64_t first_position, int64_t n_positions,
                     int32_t* h_page_table_row, int32_t* n_pages_out, int32_t* h_copy);

/* Let go of the pages behind the first n_positions positions (after a rollback or an eviction). */
Q3KV_API int q3kv_trim_slot(q3kv_allocator* a, int32_t slot, int64_t n_positions, int32_t* h_page_table_row,
                     int32_t* n_pages_out);

/* Move held pages from the highest ids to the lowest free ones, at most max_moves of them, and
 * list them: page h_src[i] becomes page h_dst[i].  No destination is another move's source or
 * destination.  Every row that held a moved page changes (q3kv_slot_pages). */
Q3KV_API int q3kv_compact_pages(q3kv_allocator* a, int32_t max_moves, int32_t* h_src, int32_t* h_dst,
                     int32_t* n_moves_out);

/* ---- quantise-append --------------------------------------------------------
 * Source: the "turbo3 3-bit KV cache" bullet of the "Quasar" (q27) wiki (each
 * step's K and V are WHT-rotated and stored as 3-bit blocks in the slot's
 * cache) and the PagedAttention paragraph of its prefix-reuse section (the
 * attention KV is an append-only log addressed by position).
 * Encodes new raw K and V head vectors and writes their records.  Slot b
 * appends d_n_new[b] tokens at positions [d_slot_len[b], d_slot_len[b] +
 * d_n_new[b]); token t of slot b is input row d_row_offsets[b] + t.
 *   k, v           device, [rows, num_kv_heads, 256], dtype f32 or bf16,
 *                  unrotated; rows = d_row_offsets[num_slots]
 *   d_page_table   device int32 [num_slots, max_pages_per_slot]
 *   d_slot_len     device int32 [num_slots], positions before the append
 *   d_n_new        device int32 [num_slots], 0 allowed
 *   d_row_offsets  device int32 [num_slots + 1]
 *   max_n_new      host bound on d_n_new[b] (sizes the launch; larger device
 *                  values set Q3KV_STATUS_BAD_LENGTH and are skipped)
 * A record whose page id is out of range is skipped with Q3KV_STATUS_BAD_PAGE. */
Q3KV_API int q3kv_append(void* stream, const q3kv_cache_desc* desc, void* d_pool,
                const int32_t* d_page_table, int32_t max_pages_per_slot,
                const int32_t* d_slot_len, const int32_t* d_n_new, const int32_t* d_row_offsets,
                int32_t num_slots, int32_t max_n_new, int32_t layer,
                const void* k, const void* v, int32_t dtype, int32_t* d_status);

/* ---- verify attention ------------------------------------------------------
 * Source: "Self-speculation as the whole design" (the step's drafts are
 * checked in one pass over the shared KV, causal among themselves), "Width-12
 * verify" (a few to a dozen query tokens per slot) and "Continuous batching"
 * (ragged slots in one launch) of the "Quasar" (q27) wiki.
 * For slot b with L_b = d_ctx_len[b] positions already in the cache (the new
 * tokens appended) and T_b = d_n_q[b] query tokens, query token t in [0, T_b)
 * of q head h attends to positions [0, L_b - T_b + t] of kv head h / 8:
 *   out = H softmax((H q) . k_hat / 16) v_hat        (float32 output)
 *   q      device [rows, num_q_heads, 256], f32 or bf16, unrotated;
 *          token t of slot b is row d_q_offsets[b] + t
 *   out    device float32, same indexing as q
 *   max_ctx_len, max_n_q   host bounds of d_ctx_len and d_n_q (size the
 *          launch); max_n_q <= 16
 *   impl   Q3KV_IMPL_*;  split_positions: positions per split-K unit
 *          (multiple of 256; 0 = chosen from the shape and the GPU)
 *   workspace, workspace_bytes: device scratch of at least
 *          q3kv_workspace_bytes(...) bytes for the same arguments (split
 *          partials and, for the tensor-core leg, the rotated queries; no
 *          initial contents needed).  Calls that share one
 *          workspace must not overlap on the GPU.
 * Slots with T_b == 0 produce nothing.  T_b > L_b or L_b beyond the slot's
 * page table sets Q3KV_STATUS_BAD_LENGTH and the slot's rows are left as they
 * were. */
Q3KV_API int q3kv_workspace_bytes(const q3kv_cache_desc* desc, int32_t num_slots, int64_t max_ctx_len,
                         int32_t max_n_q, int32_t impl, int32_t split_positions, size_t* bytes);

Q3KV_API int q3kv_verify_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- verify attention with fixed scratch (no workspace argument) -----------
 * The pages have no counterpart to this call; it exists for callers that
 * cannot provide a device workspace (another allocator owns all device memory,
 * a serving loop that must not allocate once running, a binding that only
 * receives device pointers).  Same arguments and results as q3kv_verify_attn,
 * minus the workspace: the split-K scratch comes from one array of
 * Q3KV_NOALLOC_SCRATCH_BYTES in the library's own device memory, which every
 * GPU that loads the library holds until the process exits.  The call
 * allocates nothing.
 *   - A call that needs more scratch than the limit (q3kv_workspace_bytes for
 *     the same arguments) returns Q3KV_ERR_WORKSPACE_TOO_SMALL and launches
 *     nothing.
 *   - The first call on a device looks up the array's device address for that
 *     device (cudaGetSymbolAddress, with that device current) and caches it;
 *     make that first call before any stream capture.  The cached address is
 *     kept for the life of the process: do not use this call on a device
 *     after cudaDeviceReset, which may reload the library's device memory at
 *     another address.
 *   - All calls share the one array: calls that overlap on the GPU (other
 *     streams, other host threads) race and may return wrong results.  The
 *     array keeps the last call's contents; the call needs no initial
 *     contents. */
#define Q3KV_NOALLOC_SCRATCH_BYTES (16u << 20)
Q3KV_API int q3kv_verify_attn_noalloc(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out,
                     int32_t impl, int32_t split_positions, int32_t* d_status);

/* ---- prefill attention over the 3-bit cache --------------------------------------
 * Source: the "turbo3 3-bit KV cache" bullet of the "Quasar" (q27) wiki (the
 * cache serves decode, verify and batched prefill) and the prefill follow-ons
 * bullet (a prefill-attention kernel).  A prefill is the verify step with many
 * new tokens: append them with q3kv_append, then q3kv_prefill_attn computes
 * the same causal attention as q3kv_verify_attn (new token t of slot b sees
 * positions [0, ctx_len - n_new + t]) for up to 8192 new tokens per slot.
 * Arguments, layout, workspace contract, errors and status bits are those of
 * q3kv_verify_attn, with d_n_new / max_n_new in place of d_n_q / max_n_q and
 * the workspace sized by q3kv_prefill_workspace_bytes.  Each CTA of the
 * tensor-core leg reads only the positions its rows can see. */
Q3KV_API int q3kv_prefill_workspace_bytes(const q3kv_cache_desc* desc, int32_t num_slots, int64_t max_ctx_len,
                         int32_t max_n_new, int32_t impl, int32_t split_positions, size_t* bytes);
Q3KV_API int q3kv_prefill_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_new, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_new, int32_t layer,
                     const void* q, int32_t dtype, float* out,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- fp8 E4M3 comparison cache ------------------------------------------------
 * The format the pages' server uses by default ("KV cache" stack bullet of the
 * "Quasar" (q27) wiki): K and V stored as fp8 E4M3 with a scale-free,
 * saturating conversion and no rotation.  It exists here to measure what the
 * 3-bit cache buys: 512 bytes per (position, kv head) against 224.
 *   - Record: 256 E4M3 bytes (dims in order) per head vector; pages, page
 *     tables, lengths and allocator exactly as the 3-bit cache, with 256-byte
 *     records in place of 112-byte ones.
 *   - Conversion: round to nearest (ties to even mantissa); magnitudes above
 *     448 and infinities to +-448; NaN stays NaN and, like an infinity, sets
 *     Q3KV_STATUS_NONFINITE_INPUT.
 *   - Verify: out = softmax(q . k / 16) v over the decoded values (no
 *     rotation), on the tensor-core leg only (impl AUTO or MMA; FMA returns
 *     Q3KV_ERR_UNSUPPORTED).  Its workspace is q3kv_workspace_bytes(...) with
 *     the same arguments.
 * Arguments, ownership, errors and status bits are those of q3kv_pool_bytes,
 * q3kv_append and q3kv_verify_attn. */
Q3KV_API int q3kv_fp8_pool_bytes(const q3kv_cache_desc* desc, size_t* bytes);
Q3KV_API int q3kv_fp8_append(void* stream, const q3kv_cache_desc* desc, void* d_pool, const int32_t* d_page_table,
                    int32_t max_pages_per_slot, const int32_t* d_slot_len, const int32_t* d_n_new,
                    const int32_t* d_row_offsets, int32_t num_slots, int32_t max_n_new, int32_t layer,
                    const void* k, const void* v, int32_t dtype, int32_t* d_status);
Q3KV_API int q3kv_fp8_verify_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- turbo5k-style cache: 5-bit Lloyd-Max K, 3-bit V ----------------------------
 * Source: the turbo5k bullet of the "Quasar" (q27) wiki's stack list: 5-bit K
 * with 32 Lloyd-Max centroids over the same WHT rotation, 82-byte K blocks per
 * 128 dims, and the 3-bit V -- the pages' fix for the 3-bit cache's tail
 * errors.  This library's reading:
 *   - K: y = H x (the 3-bit codec's rotation); per 128-dim half an fp16 scale
 *     s = root mean square of y (float32 squares summed within each run of 8
 *     elements from its first, then over runs pairwise); v = y / s (IEEE
 *     float32), code = the number of the 31 float32 midpoints of the float32
 *     Lloyd-Max centroids of N(0, 1) below v (s == 0: code 16); value c_code s.
 *   - K record, 164 bytes: bytes 0..127 the low nibbles of the 256 codes (two
 *     per byte, even element low), 128..159 their 5th bits (element d at bit
 *     d % 8 of byte 128 + d / 8), 160..163 the two fp16 scales.
 *   - V record: the 3-bit codec's 112 bytes.
 *   - Pool: per (page, layer, kv head) 256 K records then 256 V records:
 *     ((page * L + layer) * H + head) * 70,656 + row * 164 (K), or
 *     + 41,984 + row * 112 (V).  Pages, page tables, lengths, allocator as the
 *     3-bit cache.
 *   - Verify: both legs (impl AUTO = the tensor-core leg, which reads K_hat =
 *     centroid * s rounded to float32 and split into fp16 hi/lo, within 2^-22
 *     of the exact value, and flags Q3KV_STATUS_RANGE for a K scale above
 *     20,000); the workspace is q3kv_workspace_bytes(...) with the same impl.
 * Arguments, ownership, errors and status bits as q3kv_pool_bytes,
 * q3kv_append and q3kv_verify_attn. */
Q3KV_API int q3kv_t5k_pool_bytes(const q3kv_cache_desc* desc, size_t* bytes);
Q3KV_API int q3kv_t5k_append(void* stream, const q3kv_cache_desc* desc, void* d_pool, const int32_t* d_page_table,
                    int32_t max_pages_per_slot, const int32_t* d_slot_len, const int32_t* d_n_new,
                    const int32_t* d_row_offsets, int32_t num_slots, int32_t max_n_new, int32_t layer,
                    const void* k, const void* v, int32_t dtype, int32_t* d_status);
Q3KV_API int q3kv_t5k_verify_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- greedy acceptance and commit ------------------------------------------
 * Source: "Quasar" (q27) wiki -- the sampler paragraph of "Serving" and the
 * "Model tool protocol" bullet (greedy speculative decode is the default), and
 * the prefix-cache discussion (attention rows below the point where the drafts
 * diverge are append-only and stay valid in place: a rejected draft is undone
 * by shortening the length, and the next append overwrites its rows).
 *
 * Slot b's verify step had T_b = d_n_q[b] query tokens: t_0 (the last committed
 * token) then drafts d_1 .. d_{T_b - 1}, at rows d_q_offsets[b] + j of logits
 * and d_tokens (the same row indexing as q3kv_verify_attn); logits row j
 * predicts the token after query token j.  With g_j the argmax of row j (the
 * lowest vocabulary index among equal maxima):
 *   a    = number of leading drafts with d_{j+1} == g_j      (0 <= a <= T_b - 1)
 *   next = g_a                     (the correction, or the bonus token if a = T_b - 1)
 *   committed = ctx_len - (T_b - 1 - a)   (keeps t_0 and the accepted drafts)
 * Outputs per slot: d_n_accepted[b] = a, d_next_token[b] = next,
 * d_committed_len[b] = committed.  A slot with T_b == 0 gets (0, -1, ctx_len).
 *   logits   device [num_rows, vocab], f32 or bf16 (dtype); num_rows bounds
 *            the rows of all slots (sizes the launch; rows past the slots'
 *            rows are read but unused)
 *   d_ctx_len   cache length of each slot after the step's append; may be the
 *            same array as d_committed_len (in-place commit)
 *   workspace   device scratch of at least q3kv_accept_workspace_bytes(num_rows,
 *            vocab) bytes, 8-byte aligned, no initial contents needed; calls
 *            sharing it must not overlap on the GPU
 * Errors: Q3KV_ERR_INVALID_ARG / _UNSUPPORTED (num_rows > 65535, max_n_q > 16)
 * / _WORKSPACE_TOO_SMALL before any launch.  On the device, T_b > max_n_q,
 * T_b > ctx_len or rows past num_rows set Q3KV_STATUS_BAD_LENGTH and give the
 * slot (0, -1, ctx_len); a NaN logit sets Q3KV_STATUS_NONFINITE_INPUT (its
 * row's argmax is then unspecified).  Asynchronous on the stream. */
Q3KV_API int q3kv_accept_workspace_bytes(int32_t num_rows, int32_t vocab, size_t* bytes);   /* either call */
Q3KV_API int q3kv_accept_greedy(void* stream, const void* logits, int32_t dtype, int32_t vocab,
                       const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                       int32_t num_slots, int32_t num_rows, int32_t max_n_q, const int32_t* d_ctx_len,
                       int32_t* d_n_accepted, int32_t* d_next_token, int32_t* d_committed_len,
                       void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- sampled acceptance ------------------------------------------------------
 * Source: "Quasar" (q27) wiki, "Model tool protocol" bullet: temperature > 0
 * routes to sampled speculative decode with Gumbel-max sampling and
 * rejection-sampled acceptance, seeded and reproducible.  This call's reading
 * (without the top-p nucleus; see q3kv_accept_sample_nucleus): the drafts are point masses
 * (a deterministic drafter), p_j = softmax(logits row j / temperature), and
 *   draft d_{j+1} is accepted iff d_uniforms[row j] < p_j(d_{j+1});
 *   at the first rejected row a, next = argmax over x != d_{a+1} of
 *     logits_a[x] / temperature + G(row, x)   (a sample of p_a without the
 *     rejected token, i.e. the residual of the rejection rule);
 *   if every draft is accepted, next = the same argmax over all x of the last
 *     row (the bonus token);
 *   G(row, x) = -log(-log U), U = ((z >> 41) + 0.5) / 2^23, z = output number
 *     row * 2^32 + x of the SplitMix64 stream seeded with `seed` (rows are
 *     global logits rows).
 * Same arguments, outputs, workspace and errors as q3kv_accept_greedy, plus:
 *   temperature  > 0 and finite (else Q3KV_ERR_INVALID_ARG)
 *   d_uniforms   device float [num_rows], values in [0, 1): row j's uniform
 *                tests the draft that follows query token j (the caller draws
 *                them; the last row of a slot is unused)
 * The probabilities and keys are computed in float32; results equal the float64
 * definition except where a uniform or a key lies within rounding of a tie. */
Q3KV_API int q3kv_accept_sample(void* stream, const void* logits, int32_t dtype, int32_t vocab,
                       const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                       int32_t num_slots, int32_t num_rows, int32_t max_n_q, const int32_t* d_ctx_len,
                       float temperature, const float* d_uniforms, uint64_t seed,
                       int32_t* d_n_accepted, int32_t* d_next_token, int32_t* d_committed_len,
                       void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- sampled acceptance with the top-p nucleus ---------------------------------
 * Source: the same "Model tool protocol" bullet (sampled speculative decode
 * filters with a top-p nucleus before the Gumbel-max draw and the rejection
 * test) and the sampler paragraph of "Serving" (the nucleus is taken on the
 * temperature-scaled distribution).  Reading: the nucleus of row j is
 * {x : logits_j[x] >= l*}, l* the largest logit of the row whose tokens at or
 * above it carry at least top_p of p_j = softmax(logits_j / temperature) (all
 * tokens tied with the cut are kept); q_j = p_j restricted to the nucleus and
 * renormalised.  Then exactly q3kv_accept_sample's rule with q_j for p_j: draft
 * d_{j+1} is accepted iff d_uniforms[row j] < q_j(d_{j+1}) (0 outside the
 * nucleus), and the residual / bonus argmax of logits / temperature + G runs
 * over the nucleus only (without the rejected token).
 *   top_p   in (0, 1]; 1 gives q3kv_accept_sample's result (else
 *           Q3KV_ERR_INVALID_ARG)
 * The cut is found by a radix select over the logits' order (masses summed
 * in 2^-40 fixed point, so the search is deterministic); results equal the
 * float64 definition except where top_p, a uniform or a key lies within
 * rounding of a tie.  Same arguments, outputs, workspace and errors as
 * q3kv_accept_sample. */
Q3KV_API int q3kv_accept_sample_nucleus(void* stream, const void* logits, int32_t dtype, int32_t vocab,
                       const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                       int32_t num_slots, int32_t num_rows, int32_t max_n_q, const int32_t* d_ctx_len,
                       float temperature, float top_p, const float* d_uniforms, uint64_t seed,
                       int32_t* d_n_accepted, int32_t* d_next_token, int32_t* d_committed_len,
                       void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- rotary positions with several axes ------------------------------------------
 * Rotates the step's query and key rows by their positions before the append
 * and the verify.  The pages have no counterpart (their engine rotates inside
 * its own projections); the call is here because after an eviction a cache row
 * is no longer a position, so positions are given explicitly, and because rows
 * of images and video carry one position per axis (time, height, width).
 *
 * The first rotary_dim of the 256 dims are rotary_dim / 2 pairs.  Pair i turns
 * by the angle a_i = position[axis_i] * f_i:
 *   (x, y) -> (x cos a_i - y sin a_i, x sin a_i + y cos a_i)
 * in float32, rounded once to the output type; the other dims are copied.
 *   - Pairs: dims (i, i + rotary_dim / 2), or (2i, 2i + 1) with
 *     Q3KV_ROPE_ADJACENT.
 *   - Axes: sections[a] pairs belong to axis a (their sum is rotary_dim / 2), in
 *     runs, or dealt in turn with Q3KV_ROPE_DEAL_AXES (pair 0 to axis 0, pair 1
 *     to axis 1, ..; an axis that has all its pairs is passed over).
 *   - Frequencies: f_i = theta^(-i / (rotary_dim / 2)), or with
 *     Q3KV_ROPE_AXIS_FREQS theta^(-k / sections[a]) for the k-th pair of axis a.
 * A plan holds each pair's frequency as a 64-bit fixed-point fraction of a turn,
 * so position * turns[i] is exact modulo whole turns for every int32 position
 * (float32 angles lose whole digits beyond a few thousand positions); the turns of
 * q3kv_rope_plan_init are within 2^-53 of a turn, a double's roundings.  It is a
 * plain host struct; a caller may fill turns[] itself (scaled frequencies):
 * turns[i] = round(f_i / (2 pi) * 2^64). */
#define Q3KV_ROPE_ADJACENT   1
#define Q3KV_ROPE_DEAL_AXES  2
#define Q3KV_ROPE_AXIS_FREQS 4
#define Q3KV_ROPE_MAX_AXES   4

typedef struct q3kv_rope_config {
    double theta;                            /* > 1, finite                                */
    int32_t rotary_dim;                      /* 16 .. 256, a multiple of 16                */
    int32_t num_axes;                        /* 1 .. 4                                     */
    int32_t sections[Q3KV_ROPE_MAX_AXES];    /* pairs of each axis (0 allowed)             */
    int32_t flags;                           /* Q3KV_ROPE_*                                */
    int32_t reserved;                        /* 0                                          */
} q3kv_rope_config;

typedef struct q3kv_rope_plan {
    uint64_t turns[128];                     /* pair i: 2^-64 turns per position           */
    uint8_t axis[128];                       /* pair i: its axis                           */
    int32_t rotary_dim;
    int32_t num_axes;
    int32_t flags;
    int32_t reserved;
} q3kv_rope_plan;

/* Fills *plan (host only, no device work).  Q3KV_ERR_INVALID_ARG for a config
 * outside the ranges above. */
Q3KV_API int q3kv_rope_plan_init(const q3kv_rope_config* config, q3kv_rope_plan* plan);

/* q_in / q_out [num_rows, num_q_heads, 256] and k_in / k_out [num_rows,
 * num_kv_heads, 256], all of one dtype.  The heads of a row are contiguous; rows
 * lie *_stride elements apart (so q and k may be slices of one projection's
 * output).  An output may be its input (same pointer and stride); its rows may
 * interleave with other operands' but not share a byte with them
 * (Q3KV_ERR_INVALID_ARG).  num_q_heads or num_kv_heads may be 0 (its
 * pointers are then unused).  d_positions int32 [num_rows, num_axes], any values.
 * Q3KV_ERR_INVALID_ARG for pointers that are not 16-byte aligned or strides that
 * are below heads * 256 or not multiples of 16 bytes. */
Q3KV_API int q3kv_rope(void* stream, const q3kv_rope_plan* plan, const int32_t* d_positions, int32_t num_rows,
              const void* q_in, int64_t q_in_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
              const void* k_in, int64_t k_in_stride, void* k_out, int64_t k_out_stride, int32_t num_kv_heads,
              int32_t dtype);

/* ---- verify and prefill attention with the softmax statistic ---------------------
 * As q3kv_verify_attn, q3kv_prefill_attn, q3kv_fp8_verify_attn and
 * q3kv_t5k_verify_attn, and the same bits in out, plus
 *   lse   device float32 [rows, num_q_heads]: log of the sum over the visible
 *         positions of e^(q . k_hat / 16) (natural log), the statistic that
 *         q3kv_attn_mass needs; rows of skipped slots are left as they were. */
Q3KV_API int q3kv_verify_attn_lse(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out, float* lse,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);
Q3KV_API int q3kv_prefill_attn_lse(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_new, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_new, int32_t layer,
                     const void* q, int32_t dtype, float* out, float* lse,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);
Q3KV_API int q3kv_fp8_verify_attn_lse(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out, float* lse,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);
Q3KV_API int q3kv_t5k_verify_attn_lse(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, float* out, float* lse,
                     int32_t impl, int32_t split_positions,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- attention mass ------------------------------------------------------------
 * The attention weight each cached position received, summed over the query
 * heads of its kv head and accumulated over steps: what an eviction goes by.
 * The pages have no counterpart (their slots never evict).  For slot b with
 * L = d_ctx_len[b] and T = d_n_q[b] query tokens (the slot's last T positions),
 * every kv head g and every position j in [0, L):
 *   mass[b, g, j] = decay * old + sum over tokens t with j <= L - T + t and the 8
 *                   query heads h of g of e^(q_th . k_hat_j / 16 - lse[t, h])
 * where old = mass[b, g, j] for j < L - T and 0 for the step's own positions
 * (they have no history; what a rolled-back draft left there is dropped).  After
 * an acceptance, call it with the committed lengths and n_accepted + 1 tokens:
 * lse and the query rows of the kept tokens are unchanged by the rollback.
 *   q, dtype, d_q_offsets   as in q3kv_verify_attn (the same unrotated queries)
 *   lse      float32 [rows, num_q_heads], as q3kv_verify_attn_lse stores it; a
 *            row whose lse or whose queries are not finite (a query of 2^92 or
 *            more counts as that) contributes nothing and sets
 *            Q3KV_STATUS_NONFINITE_INPUT; the other rows' weights do not change
 *   decay    in [0, 1]; with 0 the old values are not read (they may be anything)
 *   d_mass   float32 [num_slots, num_kv_heads, mass_stride], updated in place;
 *            entries at or past L and slots with T == 0 are left as they were;
 *            mass_stride >= max_ctx_len.  It must not overlap the other buffers.
 * max_n_q <= 16.  T > max_n_q, T > L, L > max_ctx_len or L beyond the slot's page
 * table set Q3KV_STATUS_BAD_LENGTH and leave the slot's mass as it was.  Positions
 * of a page whose id is out of range keep decay * old and set
 * Q3KV_STATUS_BAD_PAGE.  Sums run in a fixed order: equal inputs give equal bits.
 * The cache's scales must be finite and non-negative, as an append without
 * Q3KV_STATUS_SCALE_OVERFLOW leaves them. */
Q3KV_API int q3kv_attn_mass(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, const float* lse, float decay,
                     float* d_mass, int64_t mass_stride, int32_t* d_status);
Q3KV_API int q3kv_fp8_attn_mass(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, const float* lse, float decay,
                     float* d_mass, int64_t mass_stride, int32_t* d_status);
Q3KV_API int q3kv_t5k_attn_mass(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, const float* lse, float decay,
                     float* d_mass, int64_t mass_stride, int32_t* d_status);

/* ---- eviction by attention mass --------------------------------------------------
 * Brings each slot down to a budget of positions: per (layer, slot, kv head) the
 * last n_recent positions, the first n_sink, and the positions between them with
 * the largest mass (the lowest position on equal masses) are kept, and their
 * records are compacted, in ascending order of position, into the pages of
 * another page table.  The attention calls go by order only, so a slot continues
 * with the destination row of pages and the new length (keys carry their rotary
 * positions); the source pages can then be freed.
 * With L = d_ctx_len[b] and n = min(L, d_budget[b]): if n_recent + n_sink > n, the
 * recent positions are kept first, then the sinks.
 *   layers    [layer, layer + num_call_layers): every layer of a slot must be
 *             evicted before its old pages are freed
 *   d_mass    float32 [num_call_layers, num_slots, num_kv_heads, mass_stride],
 *             mass_stride >= max_ctx_len; a NaN counts as less than everything
 *             and sets Q3KV_STATUS_NONFINITE_INPUT
 *   d_budget  int32 [num_slots]; 0 or less leaves the slot out: only
 *             d_new_len[b] = d_ctx_len[b] is written
 *   d_dst_page_table  int32 [num_slots, dst_max_pages_per_slot]: ceil(n / 256)
 *             pages per slot, each used once in this call and part of no slot's
 *             source pages
 *   d_kept    int32 [num_call_layers, num_slots, num_kv_heads, max_budget]: the kept
 *             positions, ascending (entries past n are left as they were)
 *   d_mass_out  float32, same layout, the kept positions' masses; may be NULL
 *   d_new_len int32 [num_slots]: n; may be the array d_ctx_len or d_budget
 * d_kept, d_mass_out and d_mass must not overlap one another, nor d_new_len the
 * lengths or budgets in any other way (Q3KV_ERR_INVALID_ARG).
 * With a max_budget as large as the lengths to come, a layer of d_mass_out is the
 * d_mass of the next q3kv_attn_mass calls, without a copy: its mass_stride is
 * max_budget, and entries past n are not read before that call has written them.
 * d_budget[b] > max_budget, L < 0, L > max_ctx_len, L beyond the slot's page table
 * or n beyond its destination pages set Q3KV_STATUS_BAD_LENGTH and leave the slot
 * out.  A record whose source or destination page id is out of range is skipped
 * with Q3KV_STATUS_BAD_PAGE.  No workspace. */
Q3KV_API int q3kv_evict(void* stream, const q3kv_cache_desc* desc, void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, int32_t num_slots, int64_t max_ctx_len,
                     const int32_t* d_budget, int32_t max_budget, int32_t n_sink, int32_t n_recent,
                     int32_t layer, int32_t num_call_layers, const float* d_mass, int64_t mass_stride,
                     const int32_t* d_dst_page_table, int32_t dst_max_pages_per_slot,
                     int32_t* d_kept, float* d_mass_out, int32_t* d_new_len, int32_t* d_status);
Q3KV_API int q3kv_fp8_evict(void* stream, const q3kv_cache_desc* desc, void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, int32_t num_slots, int64_t max_ctx_len,
                     const int32_t* d_budget, int32_t max_budget, int32_t n_sink, int32_t n_recent,
                     int32_t layer, int32_t num_call_layers, const float* d_mass, int64_t mass_stride,
                     const int32_t* d_dst_page_table, int32_t dst_max_pages_per_slot,
                     int32_t* d_kept, float* d_mass_out, int32_t* d_new_len, int32_t* d_status);
Q3KV_API int q3kv_t5k_evict(void* stream, const q3kv_cache_desc* desc, void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, int32_t num_slots, int64_t max_ctx_len,
                     const int32_t* d_budget, int32_t max_budget, int32_t n_sink, int32_t n_recent,
                     int32_t layer, int32_t num_call_layers, const float* d_mass, int64_t mass_stride,
                     const int32_t* d_dst_page_table, int32_t dst_max_pages_per_slot,
                     int32_t* d_kept, float* d_mass_out, int32_t* d_new_len, int32_t* d_status);

/* ---- acceptance of sampled drafts --------------------------------------------------
 * Source: the same "Model tool protocol" bullet as q3kv_accept_sample, for a
 * drafter that samples: draft d_{j+1} was drawn from the distribution
 * q_j = draft_probs row j, and the step's output has to follow the target
 * p_j = softmax(logits row j / temperature).
 *   draft d_{j+1} is accepted iff u_j q_j(d_{j+1}) < p_j(d_{j+1}),  u_j = d_uniforms[row j]
 *   (for u_j uniform in [0, 1): with probability min(1, p / q));
 *   at the first rejected row a, next = argmax over x with r(x) > 0 of
 *     r(x) / E(row, x),  r = max(p_a - q_a, 0),  E = -log U
 *   (a sample of the normalised r: the smallest of exponential clocks E / r rings
 *   first); if r is 0 everywhere, and for the bonus token of a slot whose drafts
 *   were all accepted, the same argmax with p in place of r;
 *   U(row, x) as in q3kv_accept_sample (equal keys: the lowest index).
 * Same arguments, outputs and errors as q3kv_accept_sample, plus:
 *   temperature   log2(e) / temperature must be finite in float32 (4.3e-39 is, 4.2e-39
 *                 is not: Q3KV_ERR_INVALID_ARG), and temperature below 3e38
 *   draft_probs   device [num_rows, vocab] of draft_dtype (f32 or bf16), the same row
 *                 indexing as logits (a slot's last row is unused); values >= 0, taken
 *                 as they are (not renormalised)
 *   d_accept_prob float [num_rows] or NULL: min(1, p_j(d_{j+1}) / q_j(d_{j+1})) in the
 *                 row of every tested draft (1 or 0 for q = 0: whether p > 0), other
 *                 rows left as they were -- what a draft-depth controller goes by;
 *                 it must not overlap d_uniforms (Q3KV_ERR_INVALID_ARG)
 *   workspace     at least q3kv_accept_draft_workspace_bytes(...) bytes, 16-byte
 *                 aligned, no initial contents needed; calls sharing it must not
 *                 overlap on the GPU
 * A draft token outside [0, vocab) is rejected with acceptance probability 0.  A
 * logit of -inf is a token of probability 0; a NaN or +inf logit sets
 * Q3KV_STATUS_NONFINITE_INPUT, and so does a NaN, infinite or negative draft
 * probability where one is read (the slot's results are then unspecified but in
 * range).  A row whose logits are all -inf has p = 0 everywhere: its draft is
 * rejected, and next is then -1. */
Q3KV_API int q3kv_accept_draft_workspace_bytes(int32_t num_slots, int32_t num_rows, int32_t vocab, size_t* bytes);
Q3KV_API int q3kv_accept_draft(void* stream, const void* logits, int32_t dtype, int32_t vocab,
                       const void* draft_probs, int32_t draft_dtype,
                       const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                       int32_t num_slots, int32_t num_rows, int32_t max_n_q, const int32_t* d_ctx_len,
                       float temperature, const float* d_uniforms, uint64_t seed,
                       int32_t* d_n_accepted, int32_t* d_next_token, int32_t* d_committed_len,
                       float* d_accept_prob, void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- block-scaled 8-bit cache ----------------------------------------------------------
 * Beside the scale-free E4M3 cache of the "KV cache" stack bullet (whose pages measured scales per
 * row to buy nothing for that engine's models): E4M3 codes with one scale for each block of 16
 * positions of a kv head, K and V apart, so that large values do not saturate and small ones
 * keep their digits.  Not rotated.
 *   scale   2^e with the smallest e in [-64, 64] for which no |x| of the block exceeds 448 2^e
 *           (-64 for a block of zeros)
 *   code    E4M3 of x 2^-e, to nearest even, magnitudes above 448 (and infinities) to 448
 * A block grows by appends: its scale is the larger of the one it has and the one that the new rows
 * ask for, and if it grows the earlier rows' codes are rewritten for it (each by the rounding of
 * code 2^(old e - new e), exact but for codes that become subnormal).  A block's first row starts
 * it afresh; a rollback leaves its scale.
 * Pool: per (page, layer, kv_head, kv) a unit of 65,600 bytes at
 *   (((page*num_layers + layer)*num_kv_heads + kv_head)*2 + kv) * 65600:
 * the code of row r = position % 256 and dim d is byte
 *   ((r/8)*16 + d/16)*128 + (r%8)*16 + d%16,
 * and the 16 blocks' scales are float32 at byte 65536 + 4*(r/16).  16-byte aligned.
 * Arguments, status bits and errors of q3kv_bs8_append are those of q3kv_append
 * (SCALE_OVERFLOW: a finite value above 448 2^64, which saturates; BAD_LENGTH: also a negative row
 * offset).  The pool must not overlap another operand (Q3KV_ERR_INVALID_ARG where the call can see it: not the
 * ends of k and v).  A NaN in K is a NaN code; one in V is a zero there and a NaN code in K at the same position
 * and dim, so that queries that see the position come out as NaN and no others do. */
Q3KV_API int q3kv_bs8_pool_bytes(const q3kv_cache_desc* desc, size_t* bytes);
Q3KV_API int q3kv_bs8_append(void* stream, const q3kv_cache_desc* desc, void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_slot_len, const int32_t* d_n_new, const int32_t* d_row_offsets,
                     int32_t num_slots, int32_t max_n_new, int32_t layer,
                     const void* k, const void* v, int32_t dtype, int32_t* d_status);

/* Verify attention over it, with q3kv_verify_attn's arguments and masks but for:
 *   out     of q's dtype (float32 or bf16), same indexing as q
 *   impl    Q3KV_IMPL_AUTO = Q3KV_IMPL_MMA: the tensor-core leg; Q3KV_IMPL_FMA: the CUDA-core leg
 *           (float32 arithmetic)
 *   d_workspace   at least q3kv_bs8_workspace_bytes(...) bytes, 16-byte aligned, no initial
 *           contents needed; its size is the same for every call on a device.  Calls that share
 *           one must not overlap on the GPU.
 * A slot with T_b > L_b, L_b above max_ctx_len or beyond its page table, T_b above max_n_q or a
 * negative offset sets Q3KV_STATUS_BAD_LENGTH and its rows are left as they were.  Positions of
 * a page out of range count as hidden (Q3KV_STATUS_BAD_PAGE); a row that sees nothing is 0.  A
 * query row that is not finite gives NaN; scores have to stay within float32.  The tensor-core leg
 * keeps weights times V's block scales in float32: V blocks of a context whose scales lie more than
 * 2^90 apart may lose weights.  Neither out nor the workspace may overlap another operand
 * (Q3KV_ERR_INVALID_ARG where the call can see it: not the ends of q and out). */
Q3KV_API int q3kv_bs8_workspace_bytes(const q3kv_cache_desc* desc, int32_t num_slots, int64_t max_ctx_len,
                     int32_t max_n_q, int32_t impl, size_t* bytes);
Q3KV_API int q3kv_bs8_verify_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool,
                     const int32_t* d_page_table, int32_t max_pages_per_slot,
                     const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                     int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer,
                     const void* q, int32_t dtype, void* out, int32_t impl,
                     void* d_workspace, size_t workspace_bytes, int32_t* d_status);

/* ---- copies of pages ---------------------------------------------------------------------
 * Copies n pages, all layers: page d_src[i] of the source pool to page d_dst[i] of the destination
 * pool, or its first d_rows[i] positions (0..256; d_rows NULL: all).  Positions behind them keep
 * what the destination held (block-scaled cache: so do their codes, while the scale of a block
 * that begins before d_rows[i] is copied).
 *   desc            the cache's shape; num_pages of the source pool
 *   d_dst_pool, dst_num_pages   may be the source pool (dst_num_pages = desc->num_pages);
 *                   pools that overlap otherwise are refused, and
 *                   so are lists within the destination pool
 *   n               at most 4096 (Q3KV_ERR_UNSUPPORTED above)
 * All pairs are copied as if at once.  A pair with a page out of range, or whose destination is
 * another pair's destination or (in one pool) source, sets Q3KV_STATUS_BAD_PAGE and is skipped; a row count
 * outside 0..256 sets Q3KV_STATUS_BAD_LENGTH likewise.  A page copied to itself stays. */
Q3KV_API int q3kv_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool,
                     int32_t dst_num_pages, const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows,
                     int32_t n, int32_t* d_status);
Q3KV_API int q3kv_fp8_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool,
                     int32_t dst_num_pages, const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows,
                     int32_t n, int32_t* d_status);
Q3KV_API int q3kv_t5k_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool,
                     int32_t dst_num_pages, const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows,
                     int32_t n, int32_t* d_status);
Q3KV_API int q3kv_bs8_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool,
                     int32_t dst_num_pages, const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows,
                     int32_t n, int32_t* d_status);

/* ---- token counts and logits --------------------------------------------------------------
 * What runs between the model's logits and the acceptance ("Serving", sampler paragraph; "Model
 * tool protocol": constrained tool calls): penalties for repeated tokens, biases, grammar masks.
 *
 * d_counts int16 [num_slots, counts_stride], one word per vocabulary entry and slot: bits 0..14
 * how often the token was generated (stays at 32767), bit 15 set if the prompt holds it.  A new
 * slot's words are zeroed by the caller.  counts_stride: entries per slot, a multiple of 8, at
 * least vocab (at most 2^28); d_counts 16-byte aligned.
 *
 * q3kv_count_tokens adds slot b's tokens d_tokens[d_offsets[b] .. + d_n[b]) (prompt = 0: one per
 * occurrence; 1: marks them as the prompt's).  d_tokens holds num_tokens; max_n bounds d_n[b].
 * A range outside it sets Q3KV_STATUS_BAD_LENGTH and skips the slot; a token outside [0, vocab)
 * sets Q3KV_STATUS_BAD_TOKEN and is skipped.  After a step the committed tokens are the step's
 * t_0 .. t_a: d_offsets = d_q_offsets, d_n = n_accepted + 1.  d_counts overlapping an input is refused. */
Q3KV_API int q3kv_count_tokens(void* stream, int16_t* d_counts, int64_t counts_stride, int32_t vocab,
                     const int32_t* d_tokens, int64_t num_tokens, const int32_t* d_offsets, const int32_t* d_n,
                     int32_t num_slots, int32_t max_n, int32_t prompt, int32_t* d_status);

/* Slot b's row j is row d_q_offsets[b] + j of logits [num_rows, vocab], j < d_n_q[b] <= max_n_q <= 16;
 * it comes after the step's tokens t_0 .. t_j (d_tokens, same indexing), which d_counts does not
 * hold yet.  With c = count + #{i <= j : t_i = x}, in float32, for every token x of the row:
 *   y = l;  if c > 0 or the prompt holds x:  y = y > 0 ? y / repetition : y * repetition
 *     (the quotient as the product with 1 / repetition, which has to be a normal number)
 *   if c > 0:  y = y - frequency c - presence
 *   y = y + bias(x);  where the row's mask bit is 0:  y = -inf
 * and out = y rounded to the logits' dtype (f32 or bf16).
 *   out            [num_rows, vocab]; may be logits itself (then rows change in place), must not overlap
 *                  any other operand.  Rows of no slot are left as they were; two slots share none.
 *   d_counts       or NULL: only the step's tokens count
 *   d_repetition, d_frequency, d_presence   float [num_slots], each or NULL (1, 0, 0)
 *   d_bias_offsets int32 [num_slots + 1] or NULL; slot b's biases are entries
 *                  [d_bias_offsets[b], d_bias_offsets[b + 1]) of d_bias_tokens (ascending, each once)
 *                  and d_bias_values, which hold num_biases entries
 *   d_mask         int32 [num_rows, ceil(vocab / 32)] or NULL: bit x % 32 of word x / 32 is 1 where x is
 *                  allowed.  A row that allows nothing is -inf everywhere.
 * A slot whose rows are not within num_rows, or a range of biases outside num_biases, sets
 * Q3KV_STATUS_BAD_LENGTH (the slot, or its biases, are skipped).  A step token or a bias token
 * outside [0, vocab), or a bias token not above the one before it, sets Q3KV_STATUS_BAD_TOKEN
 * and is skipped; of several biases that are then left for one token the last counts. */
Q3KV_API int q3kv_process_logits(void* stream, const void* logits, void* out, int32_t dtype, int32_t vocab,
                     const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                     int32_t num_slots, int32_t num_rows, int32_t max_n_q,
                     const int16_t* d_counts, int64_t counts_stride, const float* d_repetition,
                     const float* d_frequency, const float* d_presence,
                     const int32_t* d_bias_offsets, const int32_t* d_bias_tokens, const float* d_bias_values,
                     int32_t num_biases, const int32_t* d_mask, int32_t* d_status);

#ifdef __cplusplus
}
#endif
#endif /* Q3KV_H */
