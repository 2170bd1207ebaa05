/*
 * kv_cache16.h -- C ABI of the live 16-bit KV cache: appending new tokens to its
 * pages with the position rotation on the way, and attention over it.
 *
 * These are the engine's own FP16/BF16 pages, in the layouts that the page codec of
 * kv_codec.h encodes for offload and restores.  A LAYER is two pointers into device
 * memory, to the first K and the first V value; pages of block_tokens tokens lie by
 * the registered strides (in elements) from there:
 *     [page, token, head, D] and [page, head, token, D], K and V apart, or
 *     [page, head, token, 2 D] packed: v = k + D, stride_token = 2 D.
 *
 * Batches, rows and rotations are those of kv_cache8.h: one batch serves the append of
 * a step's new tokens and the attention of their queries, over 16-bit and 8-bit layers.
 * Threading, streams, graphs and errors are as described there too: a handle is
 * immutable, calls only enqueue work, lengths and tables are read on the device, and
 * every function returns KV_OK (0) or a negative KV_ERR_* code.
 */
#ifndef KV_CACHE16_H
#define KV_CACHE16_H

#include "kv_cache8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV_CACHE16_ABI_VERSION 1u

/* Registered once per cache.  Strides are in elements, the value stride is 1, and every
 * stride is a multiple of 8. */
typedef struct kv_cache16_geometry {
  uint32_t abi_version;   /* KV_CACHE16_ABI_VERSION */
  uint32_t struct_size;   /* sizeof(kv_cache16_geometry) */
  uint32_t dtype;         /* KV_DT_*: the type of the pages, of new keys and values, queries and outputs */
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
} kv_cache16_geometry;

typedef struct kv_cache16_layer {
  void* k;                /* 16-byte aligned device memory */
  void* v;
} kv_cache16_layer;

typedef struct kv_cache16_s* kv_cache16_t;

/* Validate a geometry and build the handle (host only).  On error *out is NULL. */
int kv_cache16_create(const kv_cache16_geometry* geometry, kv_cache16_t* out);
int kv_cache16_destroy(kv_cache16_t cache);

/* The batch's new tokens into their pages: keys turned by their positions (rotation NULL:
 * as they are), values as they are; a turned value is rounded once, to nearest even.  q and
 * q_out as for kv_cache8_append.  A token whose page is none, or whose position is
 * negative, is not written (its queries are turned all the same, or become 0).  No two
 * new tokens of a call may lie in the same place of a page (a shared prefix ends before
 * them), and k, v and q lie outside the pages. */
int kv_cache16_append(kv_cache16_t cache, const kv_cache16_layer* layer, const kv_cache8_batch* batch,
                      const kv_cache8_rows* k, const kv_cache8_rows* v, const kv_cache8_rotation* rotation,
                      const kv_cache8_rows* q, const kv_cache8_rows* q_out, void* stream);

/* Attention of the batch's new tokens over their sequences, by the definition, the masks
 * (flags KV_CACHE8_CAUSAL, window) and the arguments of kv_cache8_attend.  Made for few new
 * tokens a sequence (one, or some drafted ones); more are served too, 16 rows (tokens x query
 * heads of a group) at a time, each reading its keys anew.  The work is split evenly over the
 * GPU by the lengths found on the device; parts of a row are joined in a fixed order, so the
 * result does not depend on timing.
 * Products accumulate in FP32; maxima, sums and joins are FP32.  The weights of V go into
 * the product as 16-bit terms, three of BF16 or two of FP16, which together hold them to
 * 2^-24 (BF16) or 2^-22 (FP16; to 2^-36 of the row's largest weight at worst).
 * What a row does not see, or what lies in a page past its sequence's length, does not reach
 * it, NaN and infinities included.  What it sees does: a NaN or +inf among its scores leaves
 * it no finite output, an infinity or NaN in V none of that dim.  A key whose score is -inf
 * weighs 0 (times an infinity or NaN of its value: NaN); a row whose scores are all -inf gets
 * what a row that sees no key gets. */
int kv_cache16_attend(kv_cache16_t cache, const kv_cache16_layer* layer, const kv_cache8_batch* batch,
                      const kv_cache8_rows* q, const kv_cache8_rows* out, float* lse, float scale,
                      uint32_t window, uint32_t flags, void* workspace, uint64_t workspace_bytes,
                      void* stream);

/* Workspace bytes of kv_cache16_attend (16-byte aligned device memory, zero-filled before its
 * first use, not shared by calls that may run at the same time); the same for every
 * batch with new tokens, so one workspace serves a cache for good. */
int kv_cache16_attend_workspace(kv_cache16_t cache, const kv_cache8_batch* batch, uint64_t* bytes);

uint32_t kv_cache16_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KV_CACHE16_H */
