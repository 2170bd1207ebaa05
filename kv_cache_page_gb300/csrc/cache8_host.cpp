// cache8_host.cpp -- the C ABI of the live 8-bit KV cache: validation of
// geometries, layers, batches and rows, and the choice of how attention's work is
// split.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "cache8_internal.h"
#include "cache_checks.h"

struct kv_cache8_s {
  kvc::C8Params p;  // geometry part filled at create
};

namespace {

using kvc::accessible;
using kvc::C8Params;
using kvc::check_batch_fields;
using kvc::check_out;
using kvc::misaligned;
using kvc::set_batch;
using kvc::set_rows;

int set_layer(C8Params& p, const kv_cache8_layer* y) {
  if (!y || !y->k || !y->v || !y->k_scale || !y->v_scale) return KV_ERR_INVALID_ARG;
  if (misaligned(y->k, 16) || misaligned(y->v, 16) || misaligned(y->k_scale, 4) || misaligned(y->v_scale, 4))
    return KV_ERR_MISALIGNED;
  for (const void* x : {(const void*)y->k, (const void*)y->v, (const void*)y->k_scale, (const void*)y->v_scale}) {
    const int rc = accessible(x);
    if (rc != KV_OK) return rc;
  }
  p.k = static_cast<uint8_t*>(y->k);
  p.v = static_cast<uint8_t*>(y->v);
  p.k_scale = y->k_scale;
  p.v_scale = y->v_scale;
  return KV_OK;
}

// Pages that a sequence's new tokens touch number at most floor(c / T) + 2;
// one new token touches one.
uint32_t page_units(const C8Params& p) {
  return p.cu ? p.n_new / p.T + 2u * p.n_seqs : p.n_seqs;
}

struct Split {
  uint32_t units, per_seq, splits, chunk, warps;
  uint64_t bytes;
};

// Sequences of more than this many rows (new tokens x query heads of a group) go to
// the prompt kernel, the others to the step kernel.  The prompt kernel is several times
// faster when its CTAs (256 rows of a KV head) fill the GPU, but does not split keys: below
// 16 of them it is the slower one (one sequence over 10240 tokens, 4 query heads to each of
// 8 KV heads, D = 128: 20 new tokens 169 us against the step kernel's 31, 64 new 186 against 88).
// The bound does not know the number of keys: 128 new tokens over 131072 make 16 CTAs, 2.46 ms.
uint32_t step_most(const C8Params& p, const kv_cache8_batch* b) {
  return (uint64_t)b->n_new * p.G / kvc::kPromptRows * p.H < 16u ? 512u : 64u;
}

bool has_prompts(const C8Params& p, const kv_cache8_batch* b) {
  if (!b->cu_new || p.D > 128) return false;
  const uint64_t most = b->max_new ? std::min(b->max_new, b->n_new) : b->n_new;
  return most * p.G > step_most(p, b);
}
// A single sequence's count is the total.
bool has_steps(const C8Params& p, const kv_cache8_batch* b) {
  return !has_prompts(p, b) || b->n_seqs > 1 || (uint64_t)b->n_new * p.G <= step_most(p, b);
}

// Row tiles of the step kernel and the ranges their keys are split into, from the
// batch's host fields alone.
Split step_split(const C8Params& p, const kv_cache8_batch* b, uint32_t window) {
  Split s;
  const uint32_t tiles1 = (p.G + kvc::kStepRows - 1) / kvc::kStepRows;
  s.per_seq = !b->cu_new ? tiles1 : has_prompts(p, b) ? step_most(p, b) / kvc::kStepRows : 0u;
  s.units = s.per_seq ? b->n_seqs * s.per_seq : 0u;
  if (b->cu_new) {  // found by cu_new where that leaves fewer units without rows
    const uint32_t by_cu = (uint32_t)((uint64_t)b->n_new * p.G / kvc::kStepRows) + b->n_seqs;
    if (!s.per_seq || by_cu < s.units) s.per_seq = 0u, s.units = by_cu;
  }
  const uint64_t reach = std::min<uint64_t>((uint64_t)b->table_width * p.T, 0x7fff0000u);
  uint64_t keys = b->max_len ? std::min<uint64_t>(b->max_len, reach) : reach;
  if (window) keys = std::min<uint64_t>(keys, (uint64_t)window + kvc::kStepRows + 15u);
  keys = std::max<uint64_t>(keys, 16u);
  // (next to prompts: single tokens, most likely)
  const uint64_t jobs = std::max<uint64_t>((uint64_t)(has_prompts(p, b) ? b->n_seqs * tiles1 : s.units) * p.H, 1u);
  const uint64_t all = std::max<uint64_t>((uint64_t)s.units * p.H, 1u);
  const uint32_t big = p.D == 256 ? 8u : 12u;
  uint64_t chunk;
  if (b->n_seqs == 1 || jobs * ((keys + 32 * big - 1) / (32 * big)) <= kvc::kC8Sms) {
    // one sequence, or so little work that every CTA has an SM of its own: CTAs of as many warps as an
    // SM holds, which join their warps in shared memory and leave few ranges to join through memory
    s.warps = big;
    chunk = std::max<uint64_t>((keys * jobs + kvc::kC8Sms - 1) / kvc::kC8Sms, 32u * big);
  } else {
    // Smaller CTAs, whose starts and ends hide behind each other.  A range costs its CTA some 4 us besides
    // its keys, so it has 384 keys at least; and the lengths may be far below the bound, so the more jobs there
    // are the more ranges each resident CTA gets on average (64 sequences of 100 to 8192 tokens, 8 heads, D = 128:
    // ranges of 1200 keys 72 us, 2300 75, 4096 84, 512 84).  Where there are jobs enough to fill the GPU twice
    // these are balance enough (256 sequences of 1000 to 2000 tokens: whole 150 us, ranges of 1024 169, in one
    // run; whole 139 now).
    s.warps = 4;
    const uint64_t slots = (uint64_t)kvc::kC8Sms * (p.D == 256 ? 2 : 3);
    chunk = jobs >= 2 * slots ? keys : std::max<uint64_t>(keys * jobs / (2 * slots + 5 * jobs), 384u);
  }
  chunk = (chunk + 31u) & ~31ull;
  s.splits = (uint32_t)std::min<uint64_t>((keys + chunk - 1) / chunk, kvc::kMaxSplits);
  // (jobs are below 2 x 456 where there is more than one range, and units at most four times as many)
  if (all > kvc::kTickets) s.splits = 1u;
  if (window) s.splits = std::min(s.splits, step_split(p, b, 0).splits);  // the workspace is sized without one
  s.chunk = (uint32_t)chunk;
  s.bytes = s.splits > 1 ? kvc::kTickets * 4u + all * s.splits * (kvc::kStepRows * (p.D + 2ull) * 4u) : 0u;
  return s;
}

}  // namespace

extern "C" {

uint32_t kv_cache8_abi_version(void) { return KV_CACHE8_ABI_VERSION; }

static_assert(sizeof(kv_cache8_geometry) == 64 && sizeof(kv_cache8_batch) == 64 && sizeof(kv_cache8_rows) == 24 &&
                  sizeof(kv_cache8_layer) == 32 && sizeof(kv_cache8_rotation) == 40,
              "public structures");

int kv_cache8_create(const kv_cache8_geometry* g, kv_cache8_t* out) {
  if (!out) return KV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!g) return KV_ERR_INVALID_ARG;
  if (g->abi_version != KV_CACHE8_ABI_VERSION || g->struct_size != sizeof(kv_cache8_geometry)) return KV_ERR_ABI;
  if (g->reserved) return KV_ERR_INVALID_ARG;
  C8Params p;
  std::memset(&p, 0, sizeof(p));
  const int rc = kvc::set_pages(p, g->dtype, g->head_dim, g->num_kv_heads, g->num_q_heads, g->block_tokens, g->num_blocks,
                                g->stride_block, g->stride_token, g->stride_head, 1);
  if (rc != KV_OK) return rc;
  kv_cache8_s* h = new (std::nothrow) kv_cache8_s;
  if (!h) return KV_ERR_INVALID_ARG;
  p.stv = (int64_t)(512 / p.D) * p.st;
  h->p = p;
  *out = h;
  return KV_OK;
}

int kv_cache8_destroy(kv_cache8_t h) {
  if (!h) return KV_ERR_INVALID_ARG;
  delete h;
  return KV_OK;
}

int kv_cache8_write(kv_cache8_t h, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                    const kv_cache8_rows* k, const kv_cache8_rows* v, void* stream) {
  if (!h) return KV_ERR_INVALID_ARG;
  C8Params p = h->p;  // per-call copy: the handle stays immutable
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(k, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(v, p.b, p.b_row, p.b_head)) != KV_OK)
    return rc;
  p.n_units = page_units(p);
  return kvc::launch_c8_write(p, stream);
}

int kv_cache8_append(kv_cache8_t h, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                     const kv_cache8_rows* k, const kv_cache8_rows* v, const kv_cache8_rotation* rotation,
                     const kv_cache8_rows* q, const kv_cache8_rows* q_out, void* stream) {
  if (!h) return KV_ERR_INVALID_ARG;
  if (!rotation) return q || q_out ? KV_ERR_INVALID_ARG : kv_cache8_write(h, layer, batch, k, v, stream);
  kvc::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  static_cast<C8Params&>(p) = h->p;
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(k, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(v, p.b, p.b_row, p.b_head)) != KV_OK ||
      (rc = kvc::set_rotation(p, rotation)) != KV_OK || (rc = kvc::set_queries(p, q, q_out)) != KV_OK)
    return rc;
  p.n_units = page_units(p);
  return kvc::launch_c8_append(p, stream);
}

int kv_cache8_read(kv_cache8_t h, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                   const kv_cache8_rows* k, const kv_cache8_rows* v, void* stream) {
  if (!h) return KV_ERR_INVALID_ARG;
  C8Params p = h->p;
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(k, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(v, p.b, p.b_row, p.b_head)) != KV_OK ||
      (rc = check_out(p, k, p.H)) != KV_OK || (rc = check_out(p, v, p.H)) != KV_OK)
    return rc;
  p.n_units = page_units(p);
  return kvc::launch_c8_read(p, stream);
}

int kv_cache8_attend_workspace(kv_cache8_t h, const kv_cache8_batch* batch, uint64_t* bytes) {
  if (!h || !bytes) return KV_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = check_batch_fields(h->p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if (has_steps(h->p, batch)) *bytes = step_split(h->p, batch, 0).bytes;  // a window never needs more
  return KV_OK;
}

int kv_cache8_attend(kv_cache8_t h, const kv_cache8_layer* layer, const kv_cache8_batch* batch,
                     const kv_cache8_rows* q, const kv_cache8_rows* out, float* lse, float scale, uint32_t window,
                     uint32_t flags, void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!h || (flags & ~KV_CACHE8_CAUSAL)) return KV_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || !std::isfinite(scale)) return KV_ERR_INVALID_ARG;
  C8Params p = h->p;
  int rc = check_batch_fields(p, batch);
  if (rc != KV_OK) return rc;
  if (batch->n_new == 0) return KV_OK;
  if ((rc = set_batch(p, batch)) != KV_OK || (rc = set_layer(p, layer)) != KV_OK ||
      (rc = set_rows(q, p.a, p.a_row, p.a_head)) != KV_OK || (rc = set_rows(out, p.b, p.b_row, p.b_head)) != KV_OK ||
      (rc = check_out(p, out, p.HQ)) != KV_OK)
    return rc;
  if (misaligned(lse, 4) || misaligned(workspace, 16)) return KV_ERR_MISALIGNED;
  if ((rc = accessible(lse)) != KV_OK || (rc = accessible(workspace)) != KV_OK) return rc;
  p.lse = lse;
  const double s = scale != 0.0f ? (double)scale : 1.0 / std::sqrt((double)p.D);
  p.scale_log2 = (float)(s * 1.44269504088896340736);
  if (!(p.scale_log2 > 0.0f) || !std::isfinite(p.scale_log2)) return KV_ERR_INVALID_ARG;
  p.window = window;
  p.causal = flags & KV_CACHE8_CAUSAL;
  const bool prompts = has_prompts(p, batch), steps = has_steps(p, batch);
  Split sp = {};
  if (steps) sp = step_split(p, batch, window);
  if (sp.bytes && (!workspace || workspace_bytes < sp.bytes)) return KV_ERR_INVALID_ARG;
  if (prompts) {
    p.n_units = (uint32_t)((uint64_t)p.n_new * p.G / kvc::kPromptRows) + p.n_seqs;
    p.min_rows = step_most(p, batch) + 1;
    p.max_rows = 0xffffffffu;
    if ((rc = kvc::launch_c8_prompt(p, stream)) != KV_OK || !steps) return rc;
  }
  p.n_units = sp.units;
  p.per_seq = sp.per_seq;
  p.splits = sp.splits;
  p.chunk = sp.chunk;
  p.step_warps = sp.warps;
  p.rows8 = !p.cu && p.G <= 8 ? 1u : 0u;  // (a hint of few new tokens is not enough: counts are read on the device)
  p.min_rows = 1;
  p.max_rows = prompts ? step_most(p, batch) : 0xffffffffu;
  if (sp.bytes) {
    p.tickets = static_cast<uint32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(p.tickets + kvc::kTickets);
  }
  return kvc::launch_c8_step(p, stream);
}

}  // extern "C"
