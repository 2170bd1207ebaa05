// cache16_host.cpp -- the C ABI of the live 16-bit KV cache: validation.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "cache_checks.h"
#include "kv_cache16.h"

struct kv_cache16_s {
  kvc::C8Params p;  // geometry part, filled at create
};

namespace {

using kvc::accessible;
using kvc::C16Params;
using kvc::C8Params;
using kvc::check_batch_fields;
using kvc::check_out;
using kvc::misaligned;
using kvc::set_batch;
using kvc::set_rows;

int set_layer(C8Params& p, const kv_cache16_layer* y) {
  if (!y || !y->k || !y->v) return KV_ERR_INVALID_ARG;
  if (misaligned(y->k, 16) || misaligned(y->v, 16)) return KV_ERR_MISALIGNED;
  for (const void* x : {(const void*)y->k, (const void*)y->v}) {
    const int rc = accessible(x);
    if (rc != KV_OK) return rc;
  }
  p.k = static_cast<uint8_t*>(y->k);
  p.v = static_cast<uint8_t*>(y->v);
  return KV_OK;
}

uint32_t tile_rows(const C8Params& p, const kv_cache8_batch* b) { return !b->cu_new && p.G <= 8u ? 8u : kvc::kStepRows; }

// Tickets, and two partial results (maximum, sum and D sums of each row) of every CTA.
uint64_t workspace_bytes_of(const C8Params& p) {
  return kvc::kTickets * 4u + kvc::kC16Ctas * 2ull * kvc::kStepRows * (p.D + 2u) * 4u;
}

}  // namespace

extern "C" {

uint32_t kv_cache16_abi_version(void) { return KV_CACHE16_ABI_VERSION; }

static_assert(sizeof(kv_cache16_geometry) == 64 && sizeof(kv_cache16_layer) == 16, "public structures");

int kv_cache16_create(const kv_cache16_geometry* g, kv_cache16_t* out) {
  if (!out) return KV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!g) return KV_ERR_INVALID_ARG;
  if (g->abi_version != KV_CACHE16_ABI_VERSION || g->struct_size != sizeof(kv_cache16_geometry)) return KV_ERR_ABI;
  if (g->reserved) return KV_ERR_INVALID_ARG;
  C8Params p;
  std::memset(&p, 0, sizeof(p));
  const int rc = kvc::set_pages(p, g->dtype, g->head_dim, g->num_kv_heads, g->num_q_heads, g->block_tokens, g->num_blocks,
                                g->stride_block, g->stride_token, g->stride_head, 2);
  if (rc != KV_OK) return rc;
  kv_cache16_s* h = new (std::nothrow) kv_cache16_s;
  if (!h) return KV_ERR_INVALID_ARG;
  h->p = p;
  *out = h;
  return KV_OK;
}

int kv_cache16_destroy(kv_cache16_t h) {
  if (!h) return KV_ERR_INVALID_ARG;
  delete h;
  return KV_OK;
}

int kv_cache16_append(kv_cache16_t h, const kv_cache16_layer* layer, const kv_cache8_batch* batch,
                      const kv_cache8_rows* k, const kv_cache8_rows* v, const kv_cache8_rotation* rotation,
                      const kv_cache8_rows* q, const kv_cache8_rows* q_out, void* stream) {
  if (!h) return KV_ERR_INVALID_ARG;
  kvc::AppendParams p;  // per-call copy: the handle stays immutable
  std::memset(&p, 0, sizeof(p));
  static_cast<C8Params&>(p) = h->p;
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(k, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(v, p.b, p.b_row, p.b_head)) != KV_OK ||
      (rc = kvc::set_rotation(p, rotation)) != KV_OK || (rc = kvc::set_queries(p, q, q_out)) != KV_OK)
    return rc;
  return kvc::launch_c16_append(p, stream);
}

int kv_cache16_attend_workspace(kv_cache16_t h, const kv_cache8_batch* batch, uint64_t* bytes) {
  if (!h || !bytes) return KV_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check_batch_fields(h->p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new) *bytes = workspace_bytes_of(h->p);
  return KV_OK;
}

int kv_cache16_attend(kv_cache16_t h, const kv_cache16_layer* layer, const kv_cache8_batch* batch,
                      const kv_cache8_rows* q, const kv_cache8_rows* out, float* lse, float scale, uint32_t window,
                      uint32_t flags, void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!h || (flags & ~KV_CACHE8_CAUSAL)) return KV_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || !std::isfinite(scale)) return KV_ERR_INVALID_ARG;
  C16Params p;
  std::memset(&p, 0, sizeof(p));
  static_cast<C8Params&>(p) = h->p;
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(q, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(out, p.b, p.b_row, p.b_head)) != KV_OK ||
      (rc = check_out(p, out, p.HQ)) != KV_OK)
    return rc;
  if (misaligned(lse, 4) || misaligned(workspace, 16)) return KV_ERR_MISALIGNED;
  if ((rc = accessible(lse)) != KV_OK || (rc = accessible(workspace)) != KV_OK) return rc;
  if (!workspace || workspace_bytes < workspace_bytes_of(p)) return KV_ERR_INVALID_ARG;
  p.lse = lse;
  const double s = scale != 0.0f ? (double)scale : 1.0 / std::sqrt((double)p.D);
  p.scale_log2 = (float)(s * 1.44269504088896340736);
  if (!(p.scale_log2 > 0.0f) || !std::isfinite(p.scale_log2)) return KV_ERR_INVALID_ARG;
  p.window = window;
  p.causal = flags & KV_CACHE8_CAUSAL;
  p.tile_rows = tile_rows(p, batch);
  while ((1u << p.g_shift) < p.G) ++p.g_shift;  // as for n / T
  p.g_magic = (uint32_t)((((uint64_t(1) << p.g_shift) - p.G) << 32) / p.G + 1);
  p.tickets = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(p.tickets + kvc::kTickets);

  // the most jobs and keys that the batch may have
  const uint64_t reach = std::min<uint64_t>((uint64_t)p.table_width * p.T, 0x7fff0000u);
  uint64_t keys = batch->max_len ? std::min<uint64_t>(batch->max_len, reach) : reach;
  if (window) keys = std::min<uint64_t>(keys, (uint64_t)window + (batch->max_new ? batch->max_new : p.n_new));
  const uint64_t tiles = !p.cu ? (uint64_t)p.n_seqs * ((p.G + p.tile_rows - 1u) / p.tile_rows)
                               : (uint64_t)p.n_new * p.G / p.tile_rows + p.n_seqs;
  return kvc::launch_c16_attend(p, tiles * p.H, keys, stream);
}

}  // extern "C"
