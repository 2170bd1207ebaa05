// cache8_append.cu -- new tokens into the 8-bit pages, keys turned by their positions
// on the way, and the same tokens' queries.
//
// As in the plain write, a warp owns one (page, head), K or V or one after the other,
// so scale, rewritten codes and new codes take one pass and no atomics.  A turned key is
// FP32 and is quantised from there: its page's largest magnitude is that of the turned
// values, so the warp holds them (16 a lane and row, four rows at a time) until the scale is
// known.  Pages with more new tokens than that are read and turned twice, the second time
// from L2.
//
// Bound by memory for whole prompts: 3 bytes a value of K and V, 4 of queries.  Measured on a GB300,
// 4 x 8192 tokens with 8 KV heads and 32 query heads of 128 in BF16: 125 to 127 us, 5.9 TB/s (a plain copy 6.7).
#include "cache8_page.cuh"
#include "rotate.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kQueries = 8;  // iterations of a queries' warp: 256 bytes of loads in flight a lane, at 16 warps an SM

struct Append8 : AppendParams {
  RowMap qm;
  uint64_t q_share;  // of the blocks, times 2^32, rounded up: floor(b q_share / 2^32) of the first b blocks turn queries
};

#ifdef KVC_BOUNDS_CHECK
inline void dbg_ranges(DbgRanges& r, const Append8& p) {
  dbg_ranges(r, static_cast<const C8Params&>(p));  // (lse is NULL: a and b have num_kv_heads heads)
  dbg_append(r, p);
}
#endif

// Ask for the line that holds ptr (a hint).
__device__ __forceinline__ void prefetch_line(const void* ptr) {
  KVC_GUARD(ptr, 1, return);
  asm volatile("prefetch.global.L2 [%0];" ::"l"(ptr));
}

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) c8_append_kernel(const __grid_constant__ Append8 p) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, R = 4;  // lanes of a token's row, rows a warp holds at once, times R
  // blocks of pages and of queries alternate in proportion: the ones wait for instructions, the others for memory
  const uint32_t qb = (uint32_t)((blockIdx.x * p.q_share) >> 32);
  if ((uint32_t)(((blockIdx.x + 1ull) * p.q_share) >> 32) != qb)
    return append_queries<DT, D, kQueries>(p, p.qm, qb * kWarps + (threadIdx.x >> 5));
  const uint32_t lane = threadIdx.x & 31u;
  PageJob j;
  if (!page_find(p, (blockIdx.x - qb) * kWarps + (threadIdx.x >> 5), j) || j.t0 >= j.t1) return;
  j.id = c8_page(p, j.q.s, (uint32_t)j.page);  // (not looked at before the new values have been asked for)
  const int sub = lane / LPR, first = j.t0 + sub;
  const int32_t pos0 = j.page * (int32_t)p.T;
#pragma unroll 1
  for (uint32_t role = j.role; role < j.role + j.roles; ++role) {
    const bool turn = role == 0u;
    const RotUnit r = rot_unit<D>(turn ? p.R : 0u, turn && p.neighbours, lane % LPR);
    const int64_t rs = role ? p.b_row : p.a_row;
    const uint16_t* src = (role ? p.b : p.a) + (int64_t)j.head * (role ? p.b_head : p.a_head) + j.row0 * rs;
    float x[R][16];
    // rows t, t + RPI, ... of the page, turned; zeros past its new tokens
    auto rows_at = [&](int t) {
      uint4 w[R][2];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int at = t + i * RPI;
        const uint16_t* row = src + (int64_t)at * rs;
        w[i][0] = at < j.t1 ? ld_nc16(row + r.c0) : make_uint4(0, 0, 0, 0);
        w[i][1] = at < j.t1 ? ld_nc16(row + r.c1) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        rot_unpack<DT>(w[i][0], w[i][1], x[i]);
        if (turn && t + i * RPI < j.t1) rot_turn(r, rot_angles(p, r, pos0 + t + i * RPI), x[i]);
      }
    };
    rows_at(first);
    if (j.id < 0 || (role == j.role && pos0 + j.t1 > (int32_t)p.positions)) {
      if (j.head == 0u && j.role == 0u && lane == 0u && role == 0u)
        c8_error(p, j.q.s, (j.id < 0 ? KV_CACHE8_BAD_PAGE : 0u) |
                               ((uint32_t)(pos0 + j.t1) > p.positions ? KV_CACHE8_BAD_POSITION : 0u));
      if (j.id < 0) return;
    }
    uint8_t* page = (role ? p.v : p.k) + (int64_t)j.id * p.sb + (int64_t)j.head * p.sh;
    float* scale_at = (role ? p.v_scale : p.k_scale) + (int64_t)j.id * p.H + j.head;
    const float was = j.t0 > 0 ? ld_held_f32(scale_at) : 0.0f;
    // the codes held, in case the scale grows
    if (lane < (uint32_t)min(j.t0, 32)) prefetch_line(page + (int64_t)lane * p.st);
    // the largest magnitude; NaN are ignored, infinities are not
    float amax = 0.0f;
    for (int t = first; t - sub < j.t1; t += R * RPI) {
      if (t != first) rows_at(t);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float inf = __uint_as_float(0x7f800000u);
    if (!(amax < inf)) {  // infinities among the new values: the largest without them
      amax = 0.0f;
      for (int t = first; t - sub < j.t1; t += R * RPI) {
        rows_at(t);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[i][e]) < inf ? fabsf(x[i][e]) : 0.0f);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    float scale = page_scale(amax);
    if (j.t0 > 0) {
      if (scale > was) {  // the earlier tokens' codes under the larger scale
        const float f = was / scale;
        for (int t = lane / (2 * LPR); t < j.t0; t += RPI / 2) {
          uint2* at = reinterpret_cast<uint2*>(page + (int64_t)t * p.st + (lane % (2 * LPR)) * 8);
          KVC_GUARD(at, 8, continue);
          uint2 c = *at;
          uint32_t h0, h1, h2, h3;
          c8_dec4(c.x, h0, h1);
          c8_dec4(c.y, h2, h3);
          const float2 a = c8_h2f(h0), b = c8_h2f(h1), d = c8_h2f(h2), e = c8_h2f(h3);
          c.x = c8_enc4(a.x * f, a.y * f, b.x * f, b.y * f);
          c.y = c8_enc4(d.x * f, d.y * f, e.x * f, e.y * f);
          *at = c;
        }
      } else {
        scale = was;
      }
    }
    const float inv = 1.0f / scale;  // exact: a power of two
    const bool again = j.t1 - j.t0 > R * RPI;
    for (int t = first; t - sub < j.t1; t += R * RPI) {
      if (again) rows_at(t);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * RPI < j.t1) {
          uint8_t* dst = page + (int64_t)(t + i * RPI) * p.st;
          uint32_t c[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[e] = c8_enc4(x[i][4 * e] * inv, x[i][4 * e + 1] * inv, x[i][4 * e + 2] * inv, x[i][4 * e + 3] * inv);
          st8(dst + r.c0, make_uint2(c[0], c[1]));
          st8(dst + r.c1, make_uint2(c[2], c[3]));
        }
      }
    }
    if (lane == 0 && scale != was) st4(scale_at, __float_as_uint(scale));
    __syncwarp();
  }
}

template <int DT, int D>
int append_d(const AppendParams& p, void* stream) {
  Append8 a;
  static_cast<AppendParams&>(a) = p;
  // K and V in one warp where that leaves 32 warps an SM, as in the plain write
  a.both_roles = (uint64_t)p.H * p.n_units >= 32ull * kC8Sms ? 1u : 0u;
  const uint64_t warps = (a.both_roles ? 1ull : 2ull) * p.H * p.n_units;
  a.qm = row_map(p.q ? p.n_new : 0u, p.HQ * (D / 16), kQueries);
  const uint64_t pages = (warps + kWarps - 1u) / kWarps;
  const uint64_t queries = (a.qm.warps + (uint64_t)kWarps - 1u) / kWarps, grid = pages + queries;
  if (a.qm.warps == 0xffffffffu || grid > 0x7fffffffull || warps > 0xffffffffull) return KV_ERR_INVALID_ARG;
  a.q_share = ((queries << 32) + grid - 1u) / grid;
  return dbg_launch(
      stream,
      [&] {
        c8_append_kernel<DT, D><<<(unsigned)grid, kWarps * 32, 0, (cudaStream_t)stream>>>(a);
        return cudaGetLastError();
      },
      a);
}

}  // namespace

int launch_c8_append(const AppendParams& p, void* stream) { KVC_C8_DISPATCH(append_d, p, stream); }

}  // namespace kvc
