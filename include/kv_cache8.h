/*
 * kv_cache8.h -- C ABI of the live 8-bit KV cache: writing new tokens into its
 * pages, reading them back, and attention over it.
 *
 * The page codec of kv_codec.h encodes 16-bit pages for offload.  This is the
 * cache that an engine serves from: K and V stay in 8 bits on the device, new
 * tokens are quantised as they are written, and attention reads the codes
 * themselves.
 *
 * A LAYER is four device arrays:
 *     k, v              E4M3 codes, one byte a value, in pages of block_tokens
 *                       tokens; [page, token, head, D] or [page, head, token, D]
 *                       by the registered strides (in bytes)
 *     k_scale, v_scale  FP32 [num_blocks][num_kv_heads]: a page's values of a
 *                       head are code * scale
 * A scale is a power of two 2^e, -60 <= e <= 119: E4M3 is a floating-point
 * format, so a power of two costs no precision, codes are x / scale without a
 * rounding of the quotient, and codes rewritten under a larger scale are the
 * codes of the same values unless they fall below the format's normal range.
 *
 * A BATCH names the sequences of a step: block tables, lengths, and how many of
 * each sequence's last tokens are "new".  The same batch serves the write of
 * the new tokens and the attention of their queries; the rows of the 16-bit
 * tensors (k, v, q, out: [n_new, heads, D] by strides) are the new tokens of
 * sequence 0, then those of sequence 1, and so on.  Tokens of sequence s hold
 * positions 0 .. lens[s] - 1; its new ones are the last cu_new[s + 1] -
 * cu_new[s] of these.  A new row whose position would be negative (an idle slot
 * of a padded batch: length 0 with one row) is not written, reads as zeros and
 * attends to nothing.
 *
 * Threading and streams: as for kv_codec.h.  A handle is immutable; every call
 * only enqueues work on the caller's stream (no synchronisation, no allocation)
 * and can be captured into a CUDA graph; all buffers belong to the caller.  The
 * launch depends on the batch's host fields alone, lengths and tables are read
 * on the device: a captured step may be replayed with other lengths and tables
 * in the same arrays.
 *
 * All functions return KV_OK (0) or a negative KV_ERR_* code of kv_codec.h
 * (kv_codec_strerror describes them) and never abort.
 */
#ifndef KV_CACHE8_H
#define KV_CACHE8_H

#include <stddef.h>
#include <stdint.h>

#include "kv_codec.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_CACHE8_ABI_VERSION 1u
#define KV_CACHE8_MAX_SEQS 65535u

/* bits of kv_cache8_batch.errors */
#define KV_CACHE8_BAD_PAGE 1u /* a token's table entry is no page of the cache, or past the table's row:
                                 the token is not written, reads as zeros, is not attended to */
#define KV_CACHE8_STALLED 2u  /* a wait inside the attention kernel ran out (of a sequence whose output is then
                                 unspecified; untold where errors is NULL); never seen in a sound run */

/* Registered once per cache.  Strides are in bytes (= codes), the value stride
 * is 1, and every stride is a multiple of 16. */
typedef struct kv_cache8_geometry {
  uint32_t abi_version;   /* KV_CACHE8_ABI_VERSION */
  uint32_t struct_size;   /* sizeof(kv_cache8_geometry) */
  uint32_t dtype;         /* KV_DT_*: the type of new keys and values, queries and outputs */
  uint32_t head_dim;      /* 32, 64, 128 or 256 */
  uint32_t num_kv_heads;  /* 1 .. 4096 */
  uint32_t num_q_heads;   /* a multiple of num_kv_heads, at most 64 times it: query heads
                             h * G .. h * G + G - 1 read KV head h */
  uint32_t block_tokens;  /* tokens per page, 1 .. 32768 */
  uint32_t reserved;      /* 0 */
  uint64_t num_blocks;    /* pages, below 2^31 */
  int64_t stride_block;
  int64_t stride_token;
  int64_t stride_head;
} kv_cache8_geometry;

typedef struct kv_cache8_layer {
  void* k;        /* 16-byte aligned device memory */
  void* v;
  float* k_scale; /* [num_blocks][num_kv_heads] */
  float* v_scale;
} kv_cache8_layer;

typedef struct kv_cache8_batch {
  uint32_t struct_size;     /* sizeof(kv_cache8_batch) */
  uint32_t n_seqs;          /* <= KV_CACHE8_MAX_SEQS */
  uint32_t n_new;           /* rows of the 16-bit tensors = cu_new[n_seqs] (n_seqs without cu_new) */
  uint32_t max_new;         /* the most new tokens of a sequence, 0 = not known */
  uint32_t max_len;         /* the longest length, 0 = table_width * block_tokens.  max_new and
                               max_len choose how the work is split; a sequence beyond them is
                               served all the same, slower */
  uint32_t table_width;     /* entries of a table row */
  int64_t table_stride;     /* entries between table rows */
  const int32_t* tables;    /* device: page of tokens [i T, (i + 1) T) of sequence s at s * table_stride + i */
  const int32_t* lens;      /* device [n_seqs]: tokens held, the new ones among them */
  const int32_t* cu_new;    /* device [n_seqs + 1], ascending from 0; NULL: one new token each (which attention
                               then takes for granted, and is faster for) */
  uint32_t* errors;         /* device [n_seqs] or NULL: KV_CACHE8_* bits are or-ed in */
} kv_cache8_batch;

/* A tensor [n_new, heads, D] of the registered dtype: 16-byte aligned device
 * memory, strides in elements, multiples of 8, the value stride 1. */
typedef struct kv_cache8_rows {
  void* data;
  int64_t stride_row;
  int64_t stride_head;
} kv_cache8_rows;

typedef struct kv_cache8_s* kv_cache8_t;

/* Validate a geometry and build the handle (host only).  On error *out is NULL. */
int kv_cache8_create(const kv_cache8_geometry* geometry, kv_cache8_t* out);
int kv_cache8_destroy(kv_cache8_t cache);

/* Quantise the batch's new tokens into their pages.  For each page and head that
 * gets tokens, with A the largest finite magnitude among them:
 *     e = the smallest e with A <= 448 * 2^e, within [-60, 119];
 *     scale = 2^e where the page's first token is new, else max(scale held, 2^e)
 *     code = E4M3(x / scale), to nearest even; beyond the range (infinities) it
 *     saturates to +-448, NaN stays NaN.
 * When the scale grows, the codes of the page's earlier tokens are rewritten
 * under the new one (E4M3(code * old / new)).  Pages written by one call must not
 * be shared between its sequences (a shared prefix ends at a page boundary);
 * codes past a sequence's length stay as they are. */
int kv_cache8_write(kv_cache8_t cache, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                    const kv_cache8_rows* k, const kv_cache8_rows* v, void* stream);

/* The batch's new tokens back in 16 bits: code * scale rounded to nearest even,
 * saturating to the dtype's largest value.  (With lens as new counts this is the
 * whole of every sequence.) */
int kv_cache8_read(kv_cache8_t cache, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                   const kv_cache8_rows* k, const kv_cache8_rows* v, void* stream);

#define KV_CACHE8_CAUSAL 1u /* flags of kv_cache8_attend */

/* Attention of the batch's new tokens over their sequences.  A query at position
 * p sees key j < lens when (CAUSAL) j <= p and (window > 0) j > p - window.
 *     z_j = scale * q . k_j;  lse = log(sum_j exp(z_j));  out = sum_j exp(z_j - lse) v_j
 * over the keys it sees.  A row that sees none gets out = 0 and lse = -infinity.
 *   q, out     [n_new, num_q_heads, D]; out may not overlap q
 *   lse        FP32 [n_new][num_q_heads], or NULL
 *   scale      0 selects 1 / sqrt(head_dim); otherwise finite and positive
 *   workspace  workspace_bytes >= kv_cache8_attend_workspace(...) bytes of device
 *              memory, 16-byte aligned, ZERO-FILLED before its first use (each
 *              call leaves it fit for the next, whatever batch or cache that is
 *              for); calls that may run at the same time need workspaces of
 *              their own.  NULL when 0 bytes are wanted.
 * Products accumulate in FP32; maxima, sums and the joining of split ranges are
 * FP32, and the sum (lse) knows nothing of V.  The weights of V times its pages'
 * scales are rounded to FP16: by 2^-11 of each at most, as much as the rounding of an
 * FP16 output; those below 2^-25 of the row's largest weight times the largest scale
 * of V that it sees, by 2^-36 of that.  (So where a page's scale is 2^25 times
 * another's, the small page's part of an output is held to 2^-36 of what the large
 * page could give.)  The result does not depend on timing. */
int kv_cache8_attend(kv_cache8_t cache, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                     const kv_cache8_rows* q, const kv_cache8_rows* out, float* lse, float scale,
                     uint32_t window, uint32_t flags, void* workspace, uint64_t workspace_bytes,
                     void* stream);

/* Workspace bytes of kv_cache8_attend for a batch's host fields (n_seqs, n_new,
 * max_new, max_len, table_width and whether cu_new is NULL). */
int kv_cache8_attend_workspace(kv_cache8_t cache, const kv_cache8_batch* batch, uint64_t* bytes);

uint32_t kv_cache8_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KV_CACHE8_H */
