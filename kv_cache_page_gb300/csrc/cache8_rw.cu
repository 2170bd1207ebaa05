// cache8_rw.cu -- writing new tokens into the 8-bit pages, and reading tokens
// back in 16 bits.
//
// A warp owns one (page, head, K or V): no other warp touches that page's codes
// of that head or their scale, so the scale is found, the earlier codes are
// rewritten where it grows, and the new codes are stored without atomics and
// in one pass.  Consecutive warps take consecutive heads, whose rows lie side by
// side in [page, token, head, D] pages and in the 16-bit tensors.
#include "cache8_common.cuh"

namespace kvc {
namespace {

constexpr float kCodeMax = 448.0f;
constexpr int kExpMin = -60, kExpMax = 119;
constexpr int kWarps = 8;

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
  uint32_t role, head;
  int32_t page;       // index within the sequence
  int32_t t0, t1;     // tokens of the page that are new
  int32_t id;         // page id, -1: none
  int64_t row0;       // row of token 0 of the page (negative where it has none)
};

__device__ __forceinline__ bool page_job(const C8Params& p, uint32_t warp, PageJob& j) {
  const uint32_t heads2 = 2u * p.H;
  const uint32_t u = warp / heads2, r = warp - u * heads2;
  if (u >= p.n_units) return false;
  j.role = r >= p.H ? 1u : 0u;
  j.head = r - j.role * p.H;
  j.q = c8_find(p, u, 1u, p.T, 2u, p.cu ? 0u : 1u);
  const int32_t T = (int32_t)p.T;
  j.page = (int32_t)(c8_div_t(p, (uint32_t)max(j.q.start, 0)) + j.q.unit);
  const int64_t first = (int64_t)j.page * T;
  j.t0 = (int32_t)max((int64_t)max(j.q.start, 0) - first, (int64_t)0);
  j.t1 = (int32_t)min((int64_t)j.q.len - first, (int64_t)T);
  j.row0 = (int64_t)j.q.row + (first - j.q.start);
  j.id = -1;
  if (j.t0 < j.t1 && j.q.n_new > 0) {
    j.id = c8_page(p, j.q.s, (uint32_t)j.page);
    if (j.id < 0 && r == 0u && (threadIdx.x & 31u) == 0u) c8_error(p, j.q.s, KV_CACHE8_BAD_PAGE);
    return true;
  }
  return j.q.n_new > 0;
}

// The largest finite magnitude of packed 16-bit values, two running maxima per
// word; NaN operands are ignored, infinities are not (see finite_max).
template <int DT>
__device__ __forceinline__ uint32_t max2(uint32_t m, uint32_t w) {
  w &= 0x7fff7fffu;
  uint32_t d;
  if (DT == 0) asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  return d;
}
template <int DT>
__device__ __forceinline__ uint32_t drop_nonfinite2(uint32_t w) {
  const uint32_t e = DT == 0 ? 0x7c00u : 0x7f80u;
  w &= 0x7fff7fffu;
  if ((w & 0xffffu) >= e) w &= 0xffff0000u;
  if ((w >> 16) >= e) w &= 0xffffu;
  return w;
}

// R: 16-byte chunks of new values a lane holds; a page with more new tokens
// than 32 R chunks is read twice, the second time from L2.
template <int DT, int D, int R>
__global__ void __launch_bounds__(kWarps * 32) c8_write_kernel(const __grid_constant__ C8Params p) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a token's row, rows a warp loads at once
  const uint32_t lane = threadIdx.x & 31u;
  PageJob j;
  if (!page_job(p, blockIdx.x * kWarps + (threadIdx.x >> 5), j) || j.id < 0 || j.t0 >= j.t1) return;
  const int sub = lane / LPR, c8 = (lane % LPR) * 8;
  const uint16_t* src = (j.role ? p.b : p.a) + (int64_t)j.head * (j.role ? p.b_head : p.a_head) + c8;
  const int64_t rs = j.role ? p.b_row : p.a_row;
  uint8_t* dst = (j.role ? p.v : p.k) + (int64_t)j.id * p.sb + (int64_t)j.head * p.sh + c8;
  float* scale_at = (j.role ? p.v_scale : p.k_scale) + (int64_t)j.id * p.H + j.head;
  const float was = j.t0 > 0 ? ldg_f32(scale_at) : 0.0f;

  uint4 w[R];
  uint32_t m = 0;
  for (int t = j.t0; t < j.t1; t += R * RPI) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tt = t + r * RPI + sub;
      w[r] = tt < j.t1 ? ld_stream16(src + (j.row0 + tt) * rs) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m = max2<DT>(m, w[r].x);
      m = max2<DT>(m, w[r].y);
      m = max2<DT>(m, w[r].z);
      m = max2<DT>(m, w[r].w);
    }
  }
  float amax = fmaxf(lo_f32<DT>(m), hi_f32<DT>(m));
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!(amax < __uint_as_float(0x7f800000u))) {  // infinities among the new values: the largest without them
    m = 0;
    for (int t = j.t0 + sub; t < j.t1; t += RPI) {
      const uint4 x = ld_stream16(src + (j.row0 + t) * rs);
      m = max2<DT>(m, drop_nonfinite2<DT>(x.x));
      m = max2<DT>(m, drop_nonfinite2<DT>(x.y));
      m = max2<DT>(m, drop_nonfinite2<DT>(x.z));
      m = max2<DT>(m, drop_nonfinite2<DT>(x.w));
    }
    amax = fmaxf(lo_f32<DT>(m), hi_f32<DT>(m));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  float scale = page_scale(amax);
  if (j.t0 > 0) {
    if (scale > was) {  // the earlier tokens' codes under the larger scale
      const float f = was / scale;
      for (int t = sub; t < j.t0; t += RPI) {
        uint2* at = reinterpret_cast<uint2*>(dst + (int64_t)t * p.st);
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
  for (int t = j.t0; t < j.t1; t += R * RPI) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int tt = t + r * RPI + sub;
      if (tt >= j.t1) continue;
      if (j.t1 - j.t0 > R * RPI) w[r] = ld_nc16(src + (j.row0 + tt) * rs);
      float x[8];
      unpack8<DT>(w[r], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
      st8(dst + (int64_t)tt * p.st, make_uint2(c8_enc4(x[0], x[1], x[2], x[3]), c8_enc4(x[4], x[5], x[6], x[7])));
    }
  }
  if (lane == 0 && scale != was) st4(scale_at, __float_as_uint(scale));
}

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32) c8_read_kernel(const __grid_constant__ C8Params p) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, U = 8;
  const uint32_t lane = threadIdx.x & 31u;
  PageJob j;
  if (!page_job(p, blockIdx.x * kWarps + (threadIdx.x >> 5), j)) return;
  const int sub = lane / LPR, c8 = (lane % LPR) * 8;
  uint16_t* out = (j.role ? p.b : p.a) + (int64_t)j.head * (j.role ? p.b_head : p.a_head) + c8;
  const int64_t rs = j.role ? p.b_row : p.a_row;
  if (j.q.unit == 0u)  // rows before the sequence's first token
    for (int i = sub; i < min(-j.q.start, j.q.n_new); i += RPI)
      st16(out + ((int64_t)j.q.row + i) * rs, make_uint4(0, 0, 0, 0));
  if (j.t0 >= j.t1) return;
  const uint8_t* src = (j.role ? p.v : p.k) + (int64_t)j.id * p.sb + (int64_t)j.head * p.sh + c8;
  const float scale = j.id < 0 ? 0.0f : ldg_f32((j.role ? p.v_scale : p.k_scale) + (int64_t)j.id * p.H + j.head);
  // FP16: a code next to 448 under the scale of values next to 65504 stands for
  // 65536 (bf16 holds every code * scale exactly)
  const float top = DT == 0 ? 65504.0f : 3.38953139e38f;
  for (int t = j.t0; t < j.t1; t += U * RPI) {
    uint2 c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tt = t + u * RPI + sub;
      c[u] = tt < j.t1 && j.id >= 0 ? ld_nc8(src + (int64_t)tt * p.st) : make_uint2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tt = t + u * RPI + sub;
      if (tt >= j.t1) continue;
      uint32_t h[4];
      c8_dec4(c[u].x, h[0], h[1]);
      c8_dec4(c[u].y, h[2], h[3]);
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = c8_h2f(h[k]);
        x[2 * k] = f.x * scale;
        x[2 * k + 1] = f.y * scale;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = x[k] > top ? top : x[k];  // comparisons keep NaN
        x[k] = x[k] < -top ? -top : x[k];
      }
      st16(out + (j.row0 + tt) * rs, pack8<DT>(x));
    }
  }
}

template <typename F>
int launch_pages(F kernel, const C8Params& p, void* stream) {
  const uint64_t warps = 2ull * p.H * p.n_units;
  const uint64_t grid = (warps + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<(unsigned)grid, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
        return cudaGetLastError();
      },
      p);
}

template <int DT, int D>
int write_d(const C8Params& p, void* stream) {
  // a page of at most 4 KB of new values in 8 chunks a lane, larger ones in 16
  return p.T * D <= 2048u ? launch_pages(c8_write_kernel<DT, D, 8>, p, stream)
                          : launch_pages(c8_write_kernel<DT, D, 16>, p, stream);
}

}  // namespace

int launch_c8_write(const C8Params& p, void* stream) { KVC_C8_DISPATCH(write_d, p, stream); }

template <int DT, int D>
static int read_d(const C8Params& p, void* stream) {
  return launch_pages(c8_read_kernel<DT, D>, p, stream);
}
int launch_c8_read(const C8Params& p, void* stream) { KVC_C8_DISPATCH(read_d, p, stream); }

}  // namespace kvc
