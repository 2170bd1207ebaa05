// cache8_page.cuh -- what the kernels that write 8-bit pages share: a warp's page and
// head, and the rule of a page's scale.
#pragma once
#include "cache8_common.cuh"

namespace kvc {

constexpr int kExpMin = -60, kExpMax = 119;

// The smallest 2^e with amax <= 448 * 2^e.  448 = 1.75 * 2^8: with amax = f 2^k,
// 1 <= f < 2, e is k - 8 for f <= 1.75, else k - 7.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int k = (int)(b >> 23) - 127;
  int e = k - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kExpMin), kExpMax);  // amax = 0 and FP32 subnormals have k = -127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Where a warp works: role, head, page and the range of its tokens.
struct PageJob {
  C8Seq q;
  uint32_t role, roles, head;  // first role and how many
  int32_t page;       // index within the sequence
  int32_t t0, t1;     // tokens of the page that are new
  int32_t id;         // page id, -1: none
  int64_t row0;       // row of token 0 of the page (negative where it has none)
};

// All but the page id; false where the warp has no work.
__device__ __forceinline__ bool page_find(const C8Params& p, uint32_t warp, PageJob& j) {
  const uint32_t per = p.both_roles ? p.H : 2u * p.H;
  const uint32_t u = warp / per, r = warp - u * per;
  if (u >= p.n_units) return false;
  j.role = r >= p.H ? 1u : 0u;
  j.roles = p.both_roles ? 2u : 1u;
  j.head = r - j.role * p.H;
  j.q = c8_find(p, u, 1u, p.T, 2u, p.cu ? 0u : 1u);
  const int32_t T = (int32_t)p.T;
  j.page = (int32_t)(c8_div_t(p, (uint32_t)max(j.q.start, 0)) + j.q.unit);
  const int64_t first = (int64_t)j.page * T;
  j.t0 = (int32_t)max((int64_t)max(j.q.start, 0) - first, (int64_t)0);
  j.t1 = (int32_t)min((int64_t)j.q.len - first, (int64_t)T);
  j.row0 = (int64_t)j.q.row + (first - j.q.start);
  j.id = -1;
  return j.q.n_new > 0;
}

__device__ __forceinline__ bool page_job(const C8Params& p, uint32_t warp, PageJob& j) {
  if (!page_find(p, warp, j)) return false;
  if (j.t0 < j.t1) {
    j.id = c8_page(p, j.q.s, (uint32_t)j.page);
    if (j.id < 0 && j.role == 0u && j.head == 0u && (threadIdx.x & 31u) == 0u) c8_error(p, j.q.s, KV_CACHE8_BAD_PAGE);
  }
  return true;
}

// The scale that a page held: an ordinary load, because the same kernel stores there
// (this warp alone, what it makes of the value; so the load needs no other order).
__device__ __forceinline__ float ld_held_f32(const float* ptr) {
  KVC_GUARD(ptr, 4, return 0.0f);
  float v;
  asm("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(ptr));
  return v;
}

}  // namespace kvc
