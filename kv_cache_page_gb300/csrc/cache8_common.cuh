// cache8_common.cuh -- what the kernels of the live 8-bit KV cache share: the
// map from launch units to sequences, page lookups, number formats.
#pragma once
#include <atomic>

#include "cache8_internal.h"
#include "device_common.cuh"

namespace kvc {

#ifdef KVC_BOUNDS_CHECK
inline void dbg_rows(DbgRanges& r, const void* base, int64_t row, int64_t head, const C8Params& p, uint32_t heads) {
  if (base && p.n_new)
    dbg_add(r, base, 2ull * ((uint64_t)row * (p.n_new - 1u) + (uint64_t)head * (heads - 1u) + p.D));
}
inline void dbg_ranges(DbgRanges& r, const C8Params& p) {
  const uint64_t last = (uint64_t)p.sb * (p.num_blocks - 1u) + (uint64_t)p.st * (p.T - 1u) +
                        (uint64_t)p.sh * (p.H - 1u) + p.D;
  dbg_add(r, p.k, dbg_slot_bytes(last));
  dbg_add(r, p.v, dbg_slot_bytes(last));
  dbg_add(r, p.k_scale, 4ull * p.num_blocks * p.H);
  dbg_add(r, p.v_scale, 4ull * p.num_blocks * p.H);
  dbg_add(r, p.tables, 4ull * ((uint64_t)p.table_stride * (p.n_seqs - 1u) + p.table_width));
  dbg_add(r, p.lens, 4ull * p.n_seqs);
  if (p.cu) dbg_add(r, p.cu, 4ull * (p.n_seqs + 1u));
  if (p.errors) dbg_add(r, p.errors, 4ull * p.n_seqs);
  const uint32_t heads = p.lse || p.scale_log2 != 0.0f ? p.HQ : p.H;
  dbg_rows(r, p.a, p.a_row, p.a_head, p, heads);
  dbg_rows(r, p.b, p.b_row, p.b_head, p, heads);
  if (p.lse) dbg_add(r, p.lse, 4ull * p.n_new * p.HQ);
  const uint64_t jobs = (uint64_t)p.n_units * p.H;
  if (p.tickets) dbg_add(r, p.tickets, 4ull * jobs);
  if (p.partials) dbg_add(r, p.partials, 4ull * jobs * p.splits * kStepRows * (p.D + 2u));
}
#endif

// ---------------------------------------------------------------- batch
struct C8Seq {
  uint32_t s;       // sequence
  uint32_t row;     // first row of its new tokens
  int32_t n_new;    // new tokens
  int32_t len;      // tokens held (>= 0)
  int32_t start;    // position of the first new token (may be negative)
  uint32_t unit;    // this unit's index within the sequence
};

// Units of a sequence with c new tokens number at most floor(c w / d) + x, so
// sequence s begins at base(s) = floor(cu[s] w / d) + x s, a bound that needs
// no scan over the sequences; the few units past a sequence's own are idle.
__device__ __forceinline__ uint32_t c8_base(uint32_t cu, uint32_t s, uint32_t w, uint32_t d, uint32_t x) {
  return (uint32_t)((uint64_t)cu * w / d) + x * s;
}

__device__ __forceinline__ int32_t ldg_i32(const int32_t* p) {
  return (int32_t)ldg_u32(reinterpret_cast<const uint32_t*>(p));
}

// Row, count and length of sequence q.s from its cu_new pair and lens entry.
__device__ __forceinline__ void c8_fill(const C8Params& p, C8Seq& q, int32_t c0, int32_t c1, int32_t len) {
  q.row = (uint32_t)c0;
  // rows past n_new are no memory of the caller's
  q.n_new = c0 < 0 || (uint32_t)c0 > p.n_new || c1 < c0 ? 0 : min(c1 - c0, (int32_t)(p.n_new - (uint32_t)c0));
  if (q.unit > 0x3fffffffu) q.n_new = 0;       // cu_new not ascending
  q.len = min(max(0, len), 0x7fff0000);        // positions + a tile stay in 32 bits
  q.start = q.len - q.n_new;
}

// The sequence of unit u: the last s with base(s) <= u, found by the whole warp
// 32 probes at a time; the last round's lanes hold what belongs to their sequence
// already, so up to 32 sequences take one trip to memory.  With per > 0, `per` units
// belong to each sequence.
__device__ __forceinline__ C8Seq c8_find(const C8Params& p, uint32_t u, uint32_t w, uint32_t d, uint32_t x,
                                         uint32_t per) {
  C8Seq q;
  if (per) {
    q.s = u / per;
    q.unit = u - q.s * per;
    const int32_t len = ldg_i32(p.lens + q.s);
    if (p.cu) c8_fill(p, q, ldg_i32(p.cu + q.s), ldg_i32(p.cu + q.s + 1u), len);
    else c8_fill(p, q, (int32_t)q.s, (int32_t)q.s + 1, len);
    return q;
  }
  const uint32_t lane = threadIdx.x & 31u;
  uint32_t lo = 0, n = p.n_seqs;  // the answer is in [lo, lo + n)
  while (n > 32u) {
    const uint32_t step = (n + 31u) / 32u;
    const uint32_t s = lo + lane * step;
    const bool in = lane * step < n;
    const bool le = in && c8_base((uint32_t)ldg_i32(p.cu + (in ? s : lo)), s, w, d, x) <= u;
    const uint32_t k = 31u - (uint32_t)__clz(__ballot_sync(0xffffffffu, le || lane == 0u));
    lo += k * step;
    n = min(step, n - k * step);
  }
  const uint32_t s = lo + min(lane, n - 1u);
  const int32_t c0 = ldg_i32(p.cu + s), c1 = ldg_i32(p.cu + s + 1u), len = ldg_i32(p.lens + s);
  const uint32_t base = c8_base((uint32_t)c0, s, w, d, x);
  const uint32_t k = 31u - (uint32_t)__clz(__ballot_sync(0xffffffffu, (lane < n && base <= u) || lane == 0u));
  q.s = lo + k;
  q.unit = u - __shfl_sync(0xffffffffu, base, k);
  c8_fill(p, q, __shfl_sync(0xffffffffu, c0, k), __shfl_sync(0xffffffffu, c1, k), __shfl_sync(0xffffffffu, len, k));
  return q;
}

__device__ __forceinline__ uint32_t c8_div_t(const C8Params& p, uint32_t n) {
  return (__umulhi(p.t_magic, n) + n) >> p.t_shift;
}

// Page id of page index i of sequence s, or -1 where there is none.
__device__ __forceinline__ int32_t c8_page(const C8Params& p, uint32_t s, uint32_t i) {
  if (i >= p.table_width) return -1;
  const int32_t id = ldg_i32(p.tables + (int64_t)s * p.table_stride + i);
  return (uint32_t)id < p.num_blocks ? id : -1;
}

__device__ __forceinline__ void c8_error(const C8Params& p, uint32_t s, uint32_t bit) {
  if (p.errors) {
    KVC_GUARD(p.errors + s, 4, return);
    atomicOr(p.errors + s, bit);
  }
}

__device__ __forceinline__ float ldg_f32(const float* p) {
  return __uint_as_float(ldg_u32(reinterpret_cast<const uint32_t*>(p)));
}

// ---------------------------------------------------------------- formats
// four floats -> four E4M3 bytes (first in the low byte): nearest even,
// saturating to +-448, NaN stays NaN
__device__ __forceinline__ uint32_t c8_enc4(float x0, float x1, float x2, float x3) {
  uint32_t d;
  asm("{ .reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3; mov.b32 %0, {lo, hi}; }"
      : "=r"(d)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return d;
}
// four E4M3 bytes -> two f16x2 words (exact)
__device__ __forceinline__ void c8_dec4(uint32_t w, uint32_t& h01, uint32_t& h23) {
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo;"
      " cvt.rn.f16x2.e4m3x2 %1, hi; }"
      : "=r"(h01), "=r"(h23)
      : "r"(w));
}
__device__ __forceinline__ float2 c8_h2f(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Let `kernel` have `bytes` of dynamic shared memory on the current device; the
// runtime is asked once per device (done: the kernel's own bits).
template <typename F>
inline bool allow_smem(F kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return true;
}

// FN<dtype, head_dim>(args) for the registered geometry.
#define KVC_C8_DISPATCH(FN, ...)                                                                   \
  switch (p.D) {                                                                                   \
    case 32: return p.dtype == KV_DT_FP16 ? FN<0, 32>(__VA_ARGS__) : FN<1, 32>(__VA_ARGS__);       \
    case 64: return p.dtype == KV_DT_FP16 ? FN<0, 64>(__VA_ARGS__) : FN<1, 64>(__VA_ARGS__);       \
    case 128: return p.dtype == KV_DT_FP16 ? FN<0, 128>(__VA_ARGS__) : FN<1, 128>(__VA_ARGS__);    \
    case 256: return p.dtype == KV_DT_FP16 ? FN<0, 256>(__VA_ARGS__) : FN<1, 256>(__VA_ARGS__);    \
  }                                                                                                \
  return KV_ERR_UNSUPPORTED_HEAD_DIM

}  // namespace kvc
