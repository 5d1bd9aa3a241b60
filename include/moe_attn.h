/*
 * moe_attn.h - C ABI of the attention-side operators that a decoder layer runs
 * next to the MoE layer of moe.h, for one NVIDIA GB300 (sm_103a): rotary
 * positions, a paged key/value cache held in 8 bits with a scale for each
 * block of tokens and head, and attention over that cache, for prompts and
 * for single tokens, with an optional sliding window and first tokens that
 * stay visible.  Part of libmoe.so.
 *
 * Conventions are those of moe.h: device pointers (16-byte aligned) owned by
 * the caller, work enqueued on `stream` (cudaStream_t as void*) without
 * synchronising, arguments checked on the host before any launch, no CPU
 * fallback, one handle used by one thread and one stream at a time.  Tensor
 * pointers that the CUDA driver does not know as device or mapped pinned
 * memory are refused with MOE_ERR_INVALID_ARG.  Calls work on the device that
 * was current when the cache's handle was made, rotary positions on that of
 * their tensors, whichever is current at the call; `stream` belongs to that
 * device (NULL: its default stream), device memory of another one is refused.
 */
#ifndef MOE_ATTN_H_
#define MOE_ATTN_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Rotary positions -----------------------------------------------------
 *
 * Pair i of a head (0 <= i < rot_dim / 2) at position p is turned by the
 * angle p * inv_freq[i] radians:
 *   (a, b) -> amplitude * (a cos - b sin, a sin + b cos)
 * with (a, b) = elements (i, i + rot_dim/2) of the head, or (2i, 2i + 1) when
 * interleaved; elements from rot_dim on are copied.  Frequencies are the
 * caller's, so every scaling of them for long contexts fits.  An angle is
 * kept as a 64-bit fraction of a turn per position, whose product with the
 * position wraps and is rounded to 32 bits: together off by less than 2^-31
 * turns at every int32 position (negative ones turn backwards) for frequencies
 * below 2^38; sine and cosine are fp32 ones of that angle.
 *
 * moe_rope_create: rot_dim a multiple of 16 in [16, 256]; inv_freq: rot_dim/2
 *   finite doubles on the host, copied; amplitude finite.  Host only.
 * moe_rope_apply: rotates the tokens of q and, when k is not NULL, of k, in
 *   one launch.  x and y: [n_tokens] rows of n_heads * head_dim elements,
 *   x_stride and y_stride elements apart (multiples of 16 bytes, at least
 *   n_heads * head_dim; they let q and k be parts of one projection's rows).
 *   y == x with equal strides rotates in place; otherwise x and y must not
 *   overlap.  head_dim: a multiple of 16, rot_dim <= head_dim <= 256.
 *   positions: [n_tokens] int32 on the device.  n_tokens == 0 is a no-op.
 *   Arithmetic in fp32, one rounding to dtype.
 * Messages of both go to moe_last_error(NULL). */
typedef struct moe_rope moe_rope_t;
typedef struct {
  const void* x;
  void* y;
  int n_heads;
  int64_t x_stride; /* elements between tokens */
  int64_t y_stride;
} moe_rope_tensor_t;

moe_status_t moe_rope_create(int rot_dim, const double* inv_freq, float amplitude,
                             int interleaved, moe_rope_t** out);
moe_status_t moe_rope_apply(const moe_rope_t* r, const moe_rope_tensor_t* q,
                            const moe_rope_tensor_t* k, int head_dim, moe_dtype_t dtype,
                            const int32_t* positions, int n_tokens, void* stream);
void moe_rope_destroy(moe_rope_t* r);

/* ---- The cache ------------------------------------------------------------
 *
 * Keys and values are e4m3 codes in pages of page_size tokens:
 *   k, v              [n_pages][n_kv_heads][page_size][head_dim] bytes
 *   k_scale, v_scale  [n_pages][n_kv_heads] fp32
 * A value is code * scale of its page and head (the scale's block).  The
 * storage is the caller's, borrowed for the handle's lifetime; pages may hold
 * anything before they are written.  Pages that the caller fills itself take
 * any scale >= 0 and any code but NaN; attend counts a value scale below 2^-64
 * (which write never makes) as 2^-64, so that a value is off by less than 2^-55.
 * A scale that is negative, NaN or infinite in a page that attend reads sets bit 2
 * of moe_kv_device_status; the rows that see the page are not valid then.
 *
 * A batch describes the tokens of one call.  Sequence b holds kv_len[b] tokens
 * (those of this call included); its last cu_q[b+1] - cu_q[b] tokens are the
 * call's, in rows cu_q[b] .. cu_q[b+1] - 1 of the call's tensors; page_table[b]
 * [t / page_size] is the page of token t.  These arrays live on the device, so
 * that a captured graph can be replayed with other lengths.  The host passes
 * bounds: n_tokens rows in all, max_q_len new tokens and max_kv_len cached
 * tokens of any sequence (a launch is sized for them).  Tokens at positions
 * below 0 (more new tokens than the sequence's length: an idle slot) are
 * skipped by write and read and see nothing in causal attend; without causal
 * they see every cached token, as all rows do.
 * A batch whose device arrays break the bounds (cu_q not ascending within
 * [0, n_tokens], lengths above the bounds, a needed page id outside
 * [0, n_pages)) sets bit 1 of moe_kv_device_status; the sequence's work that
 * needs them is left out, nothing out of bounds is read or written.  Rows of a
 * result that no sequence covers, or whose sequence has such an offset or length,
 * keep what they held; where a page id was bad, attend's rows that need the page
 * are written, but not valid.
 * write: no two sequences of a batch may write to one page. */
typedef struct moe_kv moe_kv_t;
typedef struct {
  int n_q_heads;  /* a multiple of n_kv_heads */
  int n_kv_heads; /* 1 .. 256 */
  int head_dim;   /* 64 or 128 */
  int page_size;  /* 16, 32, 64 or 128 */
  int n_pages;
  int max_seqs;   /* bounds of every batch: 1 .. 65535 */
  int max_tokens;
  int max_kv_len;
} moe_kv_config_t;
typedef struct {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
} moe_kv_store_t;
typedef struct {
  int n_seqs;
  int n_tokens;
  int max_q_len;
  int max_kv_len;
  int table_stride;          /* entries of a row of page_table */
  const int32_t* cu_q;       /* [n_seqs + 1] */
  const int32_t* kv_len;     /* [n_seqs] */
  const int32_t* page_table; /* [n_seqs][table_stride] */
} moe_kv_batch_t;

/* Checks cfg (MOE_ERR_UNSUPPORTED) and that the store's arrays lie in device
 * memory and hold the bytes that cfg implies, allocates the workspace: what the
 * largest call within cfg can use, at most 70 MB for heads of 64 and 137 MB for
 * heads of 128. */
moe_status_t moe_kv_create(const moe_kv_config_t* cfg, const moe_kv_store_t* store,
                           moe_kv_t** out);
size_t moe_kv_workspace_bytes(const moe_kv_config_t* cfg); /* 0 if cfg is invalid */
const char* moe_kv_last_error(const moe_kv_t* h);          /* NULL: moe_last_error(NULL) */
void moe_kv_destroy(moe_kv_t* h); /* device synchronise, then free; NULL is ignored */

/* Quantises the batch's new keys and values into their pages.  k, v: [n_tokens]
 * rows of n_kv_heads * head_dim, k_stride and v_stride elements apart
 * (multiples of 16 bytes).  A block's scale is the smallest power of two
 * s >= 2^-64 with |x| <= 448 s for all its tokens, so no bit is lost in the
 * scaling; code = x / s rounded to the nearest even e4m3.  When tokens join a
 * page that holds earlier tokens of the sequence and need a larger scale, the
 * earlier codes are re-encoded (exact, but for values below 2^-6 of the new
 * scale).  NaN is stored as 0 and infinities as +-448 s (s from the finite
 * values); both set bit 2 of moe_kv_device_status. */
moe_status_t moe_kv_write(moe_kv_t* h, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, moe_dtype_t dtype, const moe_kv_batch_t* batch,
                          void* stream);

/* The batch's new tokens as values: k_out, v_out [n_tokens][n_kv_heads][head_dim]
 * of dtype (either may be NULL).  Rows of skipped tokens are set to 0. */
moe_status_t moe_kv_read(moe_kv_t* h, void* k_out, void* v_out, moe_dtype_t dtype,
                         const moe_kv_batch_t* batch, void* stream);

/* Attention of the batch's new tokens over the cache (write them first):
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * over the tokens j of the row's sequence that it sees, with the keys and
 * values of kv head h / (n_q_heads / n_kv_heads).  With i the row's place in
 * its sequence's new tokens and P = kv_len - (number of new tokens) + i its
 * position, j is seen when 0 <= j < kv_len and
 *   causal == 0, or j <= P and (window == 0 or j > P - window or j < sinks).
 * A row that sees nothing gets 0 (and lse -inf).  window >= 0 and sinks >= 0
 * need causal != 0 when they are not 0.  q, out: [n_tokens][n_q_heads]
 * [head_dim] bf16, not overlapping, q_stride elements between q's tokens; lse: [n_tokens]
 * [n_q_heads] fp32 natural logarithms of the softmax denominators, or NULL.
 * n_tokens * n_q_heads is below 2^31 (MOE_ERR_UNSUPPORTED). */
typedef struct {
  float scale; /* finite, its product with log2 e too; usually head_dim ^ -0.5 */
  int causal;
  int window;
  int sinks;
} moe_kv_mask_t;
moe_status_t moe_kv_attend(moe_kv_t* h, const void* q, int64_t q_stride, void* out, float* lse,
                           const moe_kv_mask_t* mask, const moe_kv_batch_t* batch, void* stream);

/* Copies the handle's device error word to *flags (synchronous) and clears it;
 * MOE_ERR_CUDA when it was not 0.  Bit 0: a bounded wait gave up (the call's
 * outputs are not valid); bit 1: a batch broke its bounds; bit 2: NaN or
 * infinity was written to the cache, or attend met a scale that is negative, NaN
 * or infinite. */
moe_status_t moe_kv_device_status(moe_kv_t* h, int32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H_ */
