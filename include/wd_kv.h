/*
 * wd_kv.h - paged cache of keys and values held in 4 bits (MXFP4), the
 * attention that reads it, and the operations on its pages: the half of a
 * decode step that stands next to the MoE layer of wd_moe.h.
 *
 * Format (OCP Microscaling Formats (MX) v1.0, MXFP4): every 32 channels of one
 * token and one head are 32 E2M1 codes (sign, 2 exponent bits, 1 mantissa bit:
 * 0, .5, 1, 1.5, 2, 3, 4, 6) and one E8M0 scale byte (2^(s-127); 255 = NaN).
 * A block with largest magnitude a gets s = floor(log2 a) - 2 + 127, clamped to
 * [0, 254]; 127 if a = 0; 255 if any value is not finite.  Elements are rounded to
 * nearest even and saturate at 6; the sign bit is kept.
 *
 * Pool: uint8 [num_pages][layers][kv_heads][page_size / 16][group], a group
 * being 16 tokens of one head in the order in which the tensor-core fragments
 * of the attention kernel want them (a fragment of 8 tokens is one contiguous,
 * conflict-free shared-memory read).  With nb = min(4, head_dim / 32) blocks to
 * a slab and slabs = head_dim / 32 / nb, a group is
 *
 *   K codes  [slabs][16 tokens][4 t][nb][4 bytes]   channel 32*nb*slab + 32c + 8t + n
 *   V codes  [slabs][2 halves][8 g][4 i][2 j][nb][2 bytes]
 *            channel 32*nb*slab + 32c + 4g + n, token 8*half + 2i + j
 *   K scales [16 tokens][head_dim / 32]
 *   V scales [16 tokens][head_dim / 32]
 *
 * where nibble n of a run is the low (n even) or high half of byte n / 2.  That
 * is 136 bytes per token and head for K and V at head_dim 128, against 512 in
 * BF16.  All layers of a page are contiguous, so a page moves as one block.
 *
 * Bookkeeping, all int32 device memory:
 *   table   [slots][columns]  the pages of the sequence in each slot, in order;
 *                             -1 beyond its last page
 *   lengths [slots]           its tokens; slot s holds ceil(lengths[s] / page_size) pages
 *   refs    [num_pages]       how many table entries name the page; 0 = free
 * A page that several sequences share is always full: forking copies the last,
 * partly filled page.  Pages are handed out lowest index first, so every result
 * is the same from run to run.
 *
 * A decode step: wd_kv_reserve adds the new tokens' places to the sequences,
 * then for each layer wd_kv_append (or wd_kv_append_rotated) writes their keys and values and
 * wd_kv_attention reads.  Both take the new tokens as a batch of `entries`
 * sequences: entry b is slot seqs[b] (NULL: slot b) and owns tokens
 * [q_start[b], q_start[b+1]) of the tensors (NULL: token b alone); its n new
 * tokens are the last n of the sequence, at positions lengths - n .. lengths - 1.
 *
 * As in wd_moe.h every call is asynchronous on `stream`, allocates nothing,
 * checks its arguments on the host before any launch, and finds its scratch in a
 * workspace that calls on different streams must not share.  What only the
 * device can see is range-checked there: a slot, page id or position out of
 * range is skipped and raises a bit of the workspace's error flag.  Lengths grow by wd_kv_reserve and
 * change by wd_kv_fork alone: a caller who lowers one keeps the pages behind the new end taken, and may write into a
 * page that another sequence shares.
 */
#ifndef WD_KV_H_
#define WD_KV_H_

#include <stddef.h>
#include <stdint.h>

#include "wd_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wd_kv_dtype { WD_KV_BF16 = 0, WD_KV_FP16 = 1, WD_KV_FP32 = 2 } wd_kv_dtype;

/* Limits of one call's batch. */
#define WD_KV_MAX_ENTRIES 4096
#define WD_KV_MAX_TOKENS (1 << 20)

typedef struct wd_kv_cache {
  void* pool;       /* 16-byte aligned */
  int32_t* table;   /* [slots][columns] */
  int32_t* lengths; /* [slots] */
  int32_t* refs;    /* [num_pages] */
  void* workspace;  /* 256-byte aligned, initialised by wd_kv_workspace_init */
  size_t workspace_bytes;
  int32_t num_pages; /* 1 .. 2^24 */
  int32_t slots;     /* 1 .. 65536 */
  int32_t columns;   /* 1 .. 2^20 */
  int32_t page_size; /* 16, 32, 64, 128 or 256 tokens */
  int32_t layers;    /* 1 .. 1024 */
  int32_t kv_heads;  /* 1 .. 256 */
  int32_t head_dim;  /* 64, 128 or 256 */
} wd_kv_cache;

/* Bits of the error flag (wd_kv_read_error_flag). */
#define WD_KV_FLAG_BAD_INDEX 1  /* a slot, page id, length or q_start entry out of range was skipped */
#define WD_KV_FLAG_TIMEOUT 2    /* a bounded wait ran out: that call's output is invalid */
#define WD_KV_FLAG_NO_PAGES 4   /* a request was refused for want of free pages */

/* Bytes of one page; 0 for dimensions that wd_kv_cache does not allow. */
WD_API size_t wd_kv_page_bytes(int layers, int kv_heads, int head_dim, int page_size);

/* Bytes of workspace that a cache of these dimensions needs (`workspace` and
 * the other pointers are not looked at); 0 for invalid dimensions. */
WD_API size_t wd_kv_workspace_size(const wd_kv_cache* cache);

/* Set up the error flag, the counters and the constants of the workspace.  Call once
 * after allocating it. */
WD_API wd_status wd_kv_workspace_init(const wd_kv_cache* cache, wd_stream_t stream);

/* Copy the error flag to `*flag` and clear it; SYNCHRONISES `stream`.  Returns
 * WD_ERR_PIPELINE_TIMEOUT, WD_ERR_OUT_OF_PAGES or WD_ERR_BAD_INDEX for the
 * first of these bits that is set, else WD_OK.  A timeout makes the output of the call that ran into it
 * invalid and leaves the calls behind it, and the cache, as they are; this call then also
 * sets the workspace's counters to zero again. */
WD_API wd_status wd_kv_read_error_flag(const wd_kv_cache* cache, wd_stream_t stream, int* flag);

/* Make room for counts[i] >= 0 more tokens at the end of the sequence in slot
 * seqs[i] (NULL: slot i): pages are added to its table and its length grows.
 * Requests are served in order, the lowest free pages first; request i is
 * refused (ok[i] = 0, nothing changed) if its pages and those that the requests
 * before it asked for exceed the free pages, if it exceeds `columns`, if the slot
 * is out of range or appears earlier in the call.  `ok` int32 [n] (may be NULL). */
WD_API wd_status wd_kv_reserve(const wd_kv_cache* cache, const int32_t* seqs,
                               const int32_t* counts, int n, int32_t* ok, wd_stream_t stream);

/* Quantise the keys and values of `tokens` new tokens and write them into one
 * layer of the cache.  k, v: [tokens, kv_heads, head_dim] of `dtype` with
 * the given strides in elements (channels contiguous).  k_out, v_out (both or
 * neither; contiguous, same dtype): the values that the cache now holds for
 * them.  Tokens of no entry are left alone.  Two tokens at one place: either wins. */
WD_API wd_status wd_kv_append(const wd_kv_cache* cache, int layer, const void* k, const void* v,
                              wd_kv_dtype dtype, int64_t k_stride_token, int64_t k_stride_head,
                              int64_t v_stride_token, int64_t v_stride_head, void* k_out,
                              void* v_out, const int32_t* seqs, const int32_t* q_start,
                              int entries, int tokens, wd_stream_t stream);

/* The same, with the rotation of queries and keys by their positions: channels x1, x2 of a pair i of the
 * token at position p become
 *
 *   x1 c - x2 s,   x2 c + x1 s,   c = cos_sin[p][i],  s = cos_sin[p][rot / 2 + i]
 *
 * for the pairs of the first `rot` channels of each head: channels i and i + rot / 2, or 2i and 2i + 1 if
 * `paired`; the others stay.  cos_sin: FP32 [positions, rot], 16-byte aligned, rot a multiple of 16 up to head_dim.
 * Products and sums are rounded to FP32 one by one, keys are quantised from that, queries rounded
 * once to their type.  q: [tokens, q_heads, head_dim] of `dtype` with the given strides (NULL, with q_out:
 * keys and values alone; q_heads up to 4096); q_out: contiguous, and may be q where that is.  Tokens at positions that cos_sin does not
 * have are skipped and raise WD_KV_FLAG_BAD_INDEX. */
WD_API wd_status wd_kv_append_rotated(const wd_kv_cache* cache, int layer, const void* q, const void* k,
                                      const void* v, wd_kv_dtype dtype, int64_t q_stride_token,
                                      int64_t q_stride_head, int q_heads, int64_t k_stride_token,
                                      int64_t k_stride_head, int64_t v_stride_token,
                                      int64_t v_stride_head, void* q_out, void* k_out, void* v_out,
                                      const float* cos_sin, int positions, int rot, int paired,
                                      const int32_t* seqs, const int32_t* q_start, int entries,
                                      int tokens, wd_stream_t stream);

/* Attention of the new tokens' queries over one layer of the cache.
 * q: [tokens, q_heads, head_dim] BF16 or FP16 with the given strides in
 * elements; q_heads a multiple of kv_heads, query head h reading key head
 * h / (q_heads / kv_heads).  The query at position p sees the keys at
 * positions max(0, p - window + 1) .. p (window 0: from 0 on):
 *
 *   out[t, h] = sum_j softmax_j(scale * q . k_j) v_j,   lse[t, h] = log sum_j exp(scale * q . k_j)
 *
 * out: [tokens, q_heads, head_dim] contiguous, q's type; lse: FP32 [tokens,
 * q_heads] or NULL.  A query that sees nothing gets zeros and -inf.  What is
 * not seen never enters the result, whatever its bytes; keys of a page id out of range are not
 * seen.  max_q: the most tokens an entry has, a hint for the tile (0: not known: `tokens` is
 * taken for it).  scale > 0.  Tokens of no entry are not written.
 *
 * Numbers: sums are FP32, probabilities are rounded to FP16 once, and any finite keys and values of the
 * cache give a finite result while the logits are FP32 numbers and |q| scale is below 2^114.  A query's
 * channels below 2^-31 of its largest lose bits; so do values 2^126 times smaller than another one that a row
 * sees in the same 32 channels. */
WD_API wd_status wd_kv_attention(const wd_kv_cache* cache, int layer, const void* q,
                                 wd_kv_dtype dtype, int64_t q_stride_token, int64_t q_stride_head,
                                 int q_heads, void* out, float* lse, const int32_t* seqs,
                                 const int32_t* q_start, int entries, int tokens, int max_q,
                                 float scale, int window, wd_stream_t stream);

/* Slot dst[i] becomes a fork of the sequence that slot src[i] holds before the
 * call, for all i at once (a beam search step passes its parents as src): whole
 * pages are shared, a partly filled last page is copied into a free page, and
 * what dst[i] held before is released.  src[i] = -1 (or src NULL) frees dst[i];
 * src[i] = dst[i] leaves it as it is.  New pages come from those free before the
 * call, lowest first, in order of i; a request that they do not suffice for, a
 * slot out of range, a last page to copy that is out of range, or a dst that appears
 * earlier in the call is refused (ok[i] = 0, dst[i] unchanged).  `ok` int32 [n] (may be NULL); n <= slots. */
WD_API wd_status wd_kv_fork(const wd_kv_cache* cache, const int32_t* src, const int32_t* dst,
                            int n, int32_t* ok, wd_stream_t stream);

/* Release the sequences in these slots (wd_kv_fork with no source). */
WD_API wd_status wd_kv_free(const wd_kv_cache* cache, const int32_t* seqs, int n,
                            wd_stream_t stream);

/* Move the live pages to the front of the pool: with m pages live, the k-th
 * live page at or above m moves into the k-th free page below m.  table_out
 * (like table) and refs_out (like refs) receive the bookkeeping after the move;
 * both NULL: the cache's own are rewritten.  With tables of their own, the old table
 * stays valid until a freed page is written again, since no page is moved onto
 * a live one.  page_map int32 [num_pages] (may be NULL): where each page went,
 * -1 for a free one. */
WD_API wd_status wd_kv_compact(const wd_kv_cache* cache, int32_t* table_out, int32_t* refs_out,
                               int32_t* page_map, wd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WD_KV_H_ */
