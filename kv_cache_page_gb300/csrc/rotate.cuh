// rotate.cuh -- the position rotation that the appending kernels apply on the way:
// what a lane holds of a vector, and how it turns it.
//
//   a' = a cos - b sin,  b' = b cos + a sin
//
// for the pairs (a, b) of the first R channels, angles by position from FP32 tables.
// Each product and sum is one FP32 rounding (nothing is contracted), so that a turned
// value does not depend on which kernel turned it.
#pragma once
#include "cache8_common.cuh"

namespace kvc {

// A vector of D values is D / 16 units of two 16-byte chunks, dealt to the lanes such that a pair never leaves
// its lane and neighbouring lanes hold neighbouring chunks: halves pair chunk 8 u with 8 u + R / 2, the rest of
// the vector and neighbours (whose pairs lie inside a chunk) pair it with the chunk half the way further.
struct RotUnit {
  uint32_t c0, c1;    // first channel of each chunk
  uint32_t t0, t1;    // place of their cosines in the table's row: four of each (halves: of both, eight in all)
  bool halves, n0, n1;
};

template <int D>
__device__ __forceinline__ RotUnit rot_unit(uint32_t R, bool neighbours, uint32_t u) {
  RotUnit r;
  r.halves = !neighbours && 16u * u < R;
  if (r.halves) {
    r.c0 = 8u * u;
    r.c1 = 8u * u + R / 2u;
  } else if (!neighbours && R) {
    r.c0 = R + 8u * u - R / 2u;  // R + 8 (u - R / 16)
    r.c1 = r.c0 + (D - R) / 2u;
  } else {
    r.c0 = 8u * u;
    r.c1 = 8u * u + D / 2u;
  }
  r.n0 = neighbours && r.c0 < R;
  r.n1 = neighbours && r.c1 < R;
  r.t0 = r.halves ? 8u * u : r.c0 / 2u;
  r.t1 = r.halves ? 8u * u + 4u : r.c1 / 2u;
  return r;
}

struct RotAngles {
  float4 c0, c1, s0, s1;
};

__device__ __forceinline__ float4 ldg_f4(const float* ptr) {
  KVC_GUARD(ptr, 16, return make_float4(0.f, 0.f, 0.f, 0.f));
  return __ldg(reinterpret_cast<const float4*>(ptr));
}

// Cosines and sines of position pos for the lane's unit; NaN past the table.
__device__ __forceinline__ RotAngles rot_angles(const AppendParams& p, const RotUnit& r, int32_t pos) {
  const float nan = __int_as_float(0x7fffffff);
  RotAngles a;
  a.c0 = a.c1 = a.s0 = a.s1 = make_float4(nan, nan, nan, nan);
  if ((uint32_t)pos < p.positions) {
    const int64_t at = (int64_t)pos * p.rot_stride;
    if (r.halves || r.n0) {
      a.c0 = ldg_f4(p.cos + at + r.t0);
      a.s0 = ldg_f4(p.sin + at + r.t0);
    }
    if (r.halves || r.n1) {
      a.c1 = ldg_f4(p.cos + at + r.t1);
      a.s1 = ldg_f4(p.sin + at + r.t1);
    }
  }
  return a;
}

// The pair (x, y) turned.
__device__ __forceinline__ void rot_pair(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)), b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
  y = b;
}

// The lane's 16 values (chunk c0 in x[0 .. 7], c1 in x[8 .. 15]) turned.
__device__ __forceinline__ void rot_turn(const RotUnit& r, const RotAngles& a, float (&x)[16]) {
  const float c[8] = {a.c0.x, a.c0.y, a.c0.z, a.c0.w, a.c1.x, a.c1.y, a.c1.z, a.c1.w};
  const float s[8] = {a.s0.x, a.s0.y, a.s0.z, a.s0.w, a.s1.x, a.s1.y, a.s1.z, a.s1.w};
  if (r.halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rot_pair(x[i], x[8 + i], c[i], s[i]);
  }
  if (r.n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rot_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
  }
  if (r.n1) {
#pragma unroll
    for (int i = 4; i < 8; ++i) rot_pair(x[2 * i], x[2 * i + 1], c[i], s[i]);
  }
}

template <int DT>
__device__ __forceinline__ void rot_unpack(const uint4& w0, const uint4& w1, float (&x)[16]) {
  float a[8], b[8];
  unpack8<DT>(w0, a);
  unpack8<DT>(w1, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = a[i], x[8 + i] = b[i];
}

// The lane's two chunks turned; what is not turned stays bit for bit, NaN among it.
template <int DT>
__device__ __forceinline__ void rot_row(const RotUnit& r, const RotAngles& a, uint4& w0, uint4& w1) {
  float x[16];
  rot_unpack<DT>(w0, w1, x);
  rot_turn(r, a, x);
  if (r.halves || r.n0)
    w0 = make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
  if (r.halves || r.n1)
    w1 = make_uint4(pack2<DT>(x[8], x[9]), pack2<DT>(x[10], x[11]), pack2<DT>(x[12], x[13]), pack2<DT>(x[14], x[15]));
}

// ---------------------------------------------------------------- rows of a batch
// How a warp's lanes are dealt to rows of `units` units: 2^log2 lanes to a row, 32 >> log2 rows at a time, a
// row's units in `slabs` slabs of `span` = iterations << log2.
struct RowMap {
  uint32_t log2, span, slabs, warps;
};

inline RowMap row_map(uint64_t rows, uint32_t units, uint32_t iterations) {
  RowMap m;
  m.log2 = 0;
  while (m.log2 < 5u && (1u << m.log2) < units) ++m.log2;
  m.span = iterations << m.log2;
  m.slabs = (units + m.span - 1u) / m.span;
  const uint64_t per = 32u >> m.log2, warps = (rows + per - 1u) / per * m.slabs;
  m.warps = warps > 0xfffffff0ull ? 0xffffffffu : (uint32_t)warps;  // 0xffffffff: too many
  return m;
}

struct RowPlace {
  bool in;      // the row belongs to a sequence
  uint32_t s;   // the sequence
  int32_t pos;  // position, negative where it has none
};

// Where row `row` of the lane is, row0 being the warp's first: the warp finds row0's sequence together, lanes
// whose row lies behind it look on from there by themselves.
__device__ __forceinline__ RowPlace row_place(const C8Params& p, uint32_t row0, uint32_t row) {
  RowPlace r;
  r.in = row < p.n_new;
  if (!p.cu) {
    r.s = r.in ? row : 0u;
    r.pos = min(max(0, ldg_i32(p.lens + r.s)), 0x7fff0000) - 1;
    return r;
  }
  C8Seq q = c8_find(p, row0, 1u, 1u, 0u, 0u);
  if (row != row0 && r.in && row >= (uint32_t)ldg_i32(p.cu + q.s + 1u)) {
    uint32_t lo = q.s, n = p.n_seqs - q.s;  // the last s with cu[s] <= row is in [lo, lo + n)
    while (n > 1u) {
      const uint32_t half = n / 2u;
      if ((uint32_t)ldg_i32(p.cu + lo + half) <= row) lo += half, n -= half;
      else n = half;
    }
    q.s = lo;
    const int32_t c0 = ldg_i32(p.cu + lo);
    q.unit = row - (uint32_t)c0;
    c8_fill(p, q, c0, ldg_i32(p.cu + lo + 1u), ldg_i32(p.lens + lo));
  } else {
    q.unit += row - row0;
  }
  r.in = r.in && q.unit < (uint32_t)q.n_new;
  r.s = q.s;
  r.pos = r.in ? q.start + (int32_t)q.unit : -1;
  return r;
}

// ---------------------------------------------------------------- queries
// Warp `warp` of the queries' part of an append: rows turned from q to q_out (which may be q: a lane loads, with
// ordinary loads, what it alone stores), I units of 32 bytes in flight a lane.  Rows without a position become 0.
template <int DT, int D, uint32_t I>
__device__ __forceinline__ void append_queries(const AppendParams& p, const RowMap& m, uint32_t warp) {
  constexpr uint32_t U = D / 16;
  if (warp >= m.warps) return;
  const uint32_t lane = threadIdx.x & 31u, per = 32u >> m.log2;
  const uint32_t group = warp / m.slabs, slab = warp - group * m.slabs;
  const uint32_t row0 = group * per, row = row0 + (lane >> m.log2);
  const uint32_t first = slab * m.span + (lane & ((1u << m.log2) - 1u)), units = p.HQ * U;
  const RotUnit r = rot_unit<D>(p.R, p.neighbours, first % U);  // the same for all iterations
  uint4 w[I][2];
#pragma unroll
  for (uint32_t i = 0; i < I; ++i) {
    const uint32_t u = first + (i << m.log2);
    const bool in = row < p.n_new && u < units;
    const uint16_t* src = p.q + (int64_t)row * p.q_row + (int64_t)(u / U) * p.q_head;
    w[i][0] = in ? ld_plain16(src + r.c0) : make_uint4(0, 0, 0, 0);
    w[i][1] = in ? ld_plain16(src + r.c1) : make_uint4(0, 0, 0, 0);
  }
  const RowPlace at = row_place(p, row0, row);
  if (!at.in) return;
  const RotAngles a = rot_angles(p, r, max(at.pos, 0));
#pragma unroll
  for (uint32_t i = 0; i < I; ++i) {
    const uint32_t u = first + (i << m.log2);
    if (u < units) {
      uint16_t* dst = p.q_out + (int64_t)row * p.q_out_row + (int64_t)(u / U) * p.q_out_head;
      rot_row<DT>(r, a, w[i][0], w[i][1]);
      if (at.pos < 0) w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
      st16(dst + r.c0, w[i][0]);
      st16(dst + r.c1, w[i][1]);
    }
  }
}

#ifdef KVC_BOUNDS_CHECK
inline void dbg_append(DbgRanges& r, const AppendParams& p) {
  if (p.R) {
    const uint64_t n = (uint64_t)p.rot_stride * (p.positions - 1u) + p.R / 2u;
    dbg_add(r, p.cos, 4ull * n);
    dbg_add(r, p.sin, 4ull * n);
  }
  dbg_rows(r, p.q, p.q_row, p.q_head, p, p.HQ);
  dbg_rows(r, p.q_out, p.q_out_row, p.q_out_head, p, p.HQ);
}
#endif

}  // namespace kvc
