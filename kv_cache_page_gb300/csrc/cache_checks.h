// cache_checks.h -- what the host sides of the paged caches (8-bit and 16-bit) check of a
// call: page layouts, reachable and aligned pointers, batches, rows, rotations, outputs.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "cache8_internal.h"

namespace kvc {

// Whether the kernels can reach ptr (pageable host memory is refused, as for
// the codec's buffers).
inline int accessible(const void* ptr) {
  if (!ptr) return KV_OK;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
    cudaGetLastError();
    return KV_ERR_CUDA;
  }
  return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged ? KV_OK : KV_ERR_NOT_ACCESSIBLE;
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// The geometry part of p (zeroed by the caller) from a registered page layout; strides in values of `bytes` bytes.
inline int set_pages(C8Params& p, uint32_t dtype, uint32_t D, uint32_t H, uint32_t HQ, uint32_t T, uint64_t blocks,
                     int64_t sb, int64_t st, int64_t sh, uint32_t bytes) {
  if (dtype != KV_DT_FP16 && dtype != KV_DT_BF16) return KV_ERR_INVALID_ARG;
  if (D != 32 && D != 64 && D != 128 && D != 256) return KV_ERR_UNSUPPORTED_HEAD_DIM;
  if (H == 0 || H > 4096 || HQ == 0 || HQ % H || HQ / H > 64) return KV_ERR_INVALID_ARG;
  if (T == 0 || T > 32768 || blocks == 0 || blocks > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  if (sb <= 0 || st <= 0 || sh <= 0) return KV_ERR_LAYOUT_MISMATCH;
  if ((sb | st | sh) & (16 / bytes - 1)) return KV_ERR_MISALIGNED;
  // the smaller of the three strides steps over a value row, each next one over the extent of those before
  struct {
    uint64_t stride, n;
  } d[3] = {{(uint64_t)sh, H}, {(uint64_t)st, T}, {(uint64_t)sb, blocks}};
  std::sort(d, d + 3, [](const auto& a, const auto& b) { return a.stride != b.stride ? a.stride < b.stride : a.n < b.n; });
  const uint64_t most = (uint64_t(1) << 62) / bytes;
  uint64_t span = D;
  for (const auto& x : d) {
    if (x.n <= 1) {
      if (bytes > 1 && x.stride > most) return KV_ERR_LAYOUT_MISMATCH;  // (never stepped over, but turned into bytes)
      continue;
    }
    if (x.stride < span || x.stride > most / (x.n - 1)) return KV_ERR_LAYOUT_MISMATCH;
    span += x.stride * (x.n - 1);
    if (span > most) return KV_ERR_LAYOUT_MISMATCH;
  }
  p.dtype = dtype;
  p.D = D;
  p.H = H;
  p.HQ = HQ;
  p.G = HQ / H;
  p.T = T;
  p.num_blocks = (uint32_t)blocks;
  p.sb = sb * bytes;
  p.st = st * bytes;
  p.sh = sh * bytes;
  p.st2 = 2 * p.st;
  // n / T for n < 2^31 by the round-up method (Granlund and Montgomery, PLDI 1994)
  while ((1u << p.t_shift) < p.T) ++p.t_shift;
  p.t_magic = (uint32_t)((((uint64_t(1) << p.t_shift) - p.T) << 32) / p.T + 1);
  return KV_OK;
}

inline int check_batch_fields(const C8Params& p, const kv_cache8_batch* b) {
  if (!b) return KV_ERR_INVALID_ARG;
  if (b->struct_size != sizeof(kv_cache8_batch)) return KV_ERR_ABI;
  if (b->n_seqs > KV_CACHE8_MAX_SEQS || b->n_new > 0x7fffffffu / p.G) return KV_ERR_INVALID_ARG;
  if (!b->cu_new && b->n_new != b->n_seqs) return KV_ERR_INVALID_ARG;
  if (b->n_seqs == 0 && b->n_new != 0) return KV_ERR_INVALID_ARG;
  return KV_OK;
}

inline int set_batch(C8Params& p, const kv_cache8_batch* b) {
  int rc = check_batch_fields(p, b);
  if (rc != KV_OK) return rc;
  if (!b->lens || (!b->tables && b->table_width) || b->table_stride < 0) return KV_ERR_INVALID_ARG;
  if (b->n_seqs > 1 && b->table_stride < (int64_t)b->table_width) return KV_ERR_INVALID_ARG;
  if (misaligned(b->tables, 4) || misaligned(b->lens, 4) || misaligned(b->cu_new, 4) || misaligned(b->errors, 4))
    return KV_ERR_MISALIGNED;
  for (const void* x : {(const void*)b->tables, (const void*)b->lens, (const void*)b->cu_new, (const void*)b->errors})
    if ((rc = accessible(x)) != KV_OK) return rc;
  p.n_seqs = b->n_seqs;
  p.n_new = b->n_new;
  p.table_width = b->table_width;
  p.table_stride = b->table_stride;
  p.tables = b->tables;
  p.lens = b->lens;
  p.cu = b->cu_new;
  p.errors = b->errors;
  return KV_OK;
}

inline int set_rows(const kv_cache8_rows* r, uint16_t*& data, int64_t& row, int64_t& head) {
  if (!r || !r->data) return KV_ERR_INVALID_ARG;
  if (misaligned(r->data, 16) || ((r->stride_row | r->stride_head) & 7)) return KV_ERR_MISALIGNED;
  if (r->stride_row < 0 || r->stride_head < 0) return KV_ERR_LAYOUT_MISMATCH;
  data = static_cast<uint16_t*>(r->data);
  row = r->stride_row;
  head = r->stride_head;
  return accessible(r->data);
}

// A rotation of the append calls; p.R stays 0 without one.
inline int set_rotation(AppendParams& p, const kv_cache8_rotation* t) {
  if (!t) return KV_OK;
  if (t->struct_size != sizeof(kv_cache8_rotation)) return KV_ERR_ABI;
  if (t->dim == 0 || t->dim > p.D || t->dim % 16 || t->positions == 0 || t->positions > 0x7fffffffu ||
      (t->flags & ~KV_CACHE8_NEIGHBOURS) || !t->cos || !t->sin)
    return KV_ERR_INVALID_ARG;
  if (t->stride < 0 || (t->positions > 1 && t->stride < (int64_t)(t->dim / 2))) return KV_ERR_LAYOUT_MISMATCH;
  if (misaligned(t->cos, 16) || misaligned(t->sin, 16) || (t->stride & 3)) return KV_ERR_MISALIGNED;
  for (const void* x : {(const void*)t->cos, (const void*)t->sin}) {
    const int rc = accessible(x);
    if (rc != KV_OK) return rc;
  }
  p.cos = t->cos;
  p.sin = t->sin;
  p.rot_stride = t->stride;
  p.R = t->dim;
  p.positions = t->positions;
  p.neighbours = t->flags & KV_CACHE8_NEIGHBOURS;
  return KV_OK;
}

// Outputs: rows and heads must not overlap.
inline int check_out(const C8Params& p, const kv_cache8_rows* r, uint32_t heads) {
  const int64_t D = p.D;
  const bool rows = p.n_new <= 1, one = heads <= 1;
  if (!one && r->stride_head < D) return KV_ERR_LAYOUT_MISMATCH;
  if (!rows && r->stride_row < D) return KV_ERR_LAYOUT_MISMATCH;
  if (rows || one) return KV_OK;
  const bool fits = r->stride_row >= r->stride_head * (int64_t)(heads - 1) + D ||
                    r->stride_head >= r->stride_row * (int64_t)(p.n_new - 1) + D;
  return fits ? KV_OK : KV_ERR_LAYOUT_MISMATCH;
}

// Queries that an append call turns: both or none, and only with a rotation.
inline int set_queries(AppendParams& p, const kv_cache8_rows* q, const kv_cache8_rows* q_out) {
  if (!q && !q_out) return KV_OK;
  if (!q || !q_out || !p.R) return KV_ERR_INVALID_ARG;
  uint16_t* in = nullptr;
  int rc = set_rows(q, in, p.q_row, p.q_head);
  if (rc != KV_OK) return rc;
  p.q = in;
  if ((rc = set_rows(q_out, p.q_out, p.q_out_row, p.q_out_head)) != KV_OK) return rc;
  return check_out(p, q_out, p.HQ);
}

}  // namespace kvc
