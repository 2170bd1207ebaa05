// cache8_rw.cu -- writing new tokens into the 8-bit pages, and reading tokens
// back in 16 bits.
//
// A warp owns one (page, head), K or V or one after the other: no other warp touches
// that page's codes of that head or their scale, so the scale is found, the earlier
// codes are rewritten where it grows, and the new codes are stored without atomics
// and in one pass.  Consecutive warps take consecutive heads, whose rows lie side by
// side in [page, token, head, D] pages and in the 16-bit tensors.
//
// Bound by memory for whole prompts: 3 bytes a value.  What keeps a warp from it is
// the work around a page (finding its sequence, page and place: some 250
// instructions), so one warp takes K and V where there are warps enough to fill the
// GPU all the same; and conversions, which stay in FP16 where that is exact.
// Measured on a GB300, 4 x 8192 tokens of 8 heads of 128 in FP16: written and read
// back in 37 us (5.4 and 5.5 TB/s of 3 bytes a value; a plain copy 6.7).
#include "cache8_common.cuh"

namespace kvc {
namespace {


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
  uint32_t role, roles, head;  // first role and how many
  int32_t page;       // index within the sequence
  int32_t t0, t1;     // tokens of the page that are new
  int32_t id;         // page id, -1: none
  int64_t row0;       // row of token 0 of the page (negative where it has none)
};

__device__ __forceinline__ bool page_job(const C8Params& p, uint32_t warp, PageJob& j) {
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
  if (j.t0 < j.t1 && j.q.n_new > 0) {
    j.id = c8_page(p, j.q.s, (uint32_t)j.page);
    if (j.id < 0 && r == 0u && (threadIdx.x & 31u) == 0u) c8_error(p, j.q.s, KV_CACHE8_BAD_PAGE);
    return true;
  }
  return j.q.n_new > 0;
}

// The largest finite magnitude of packed 16-bit values, two running maxima per
// word; NaN operands are ignored, infinities are not (drop_nonfinite2 takes them out).
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

// 2^e as FP16 where it has one, e = -14 .. 15; 0 otherwise
__device__ __forceinline__ uint32_t half2_pow2(float s) {
  const int e = (int)(__float_as_uint(s) >> 23) - 127;
  if ((__float_as_uint(s) & 0x807fffffu) || e < -14 || e > 15) return 0u;
  return (uint32_t)(e + 15) * 0x04000400u;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// four FP16 -> four E4M3 bytes
__device__ __forceinline__ uint32_t enc_h4(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{ .reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f16x2 lo, %1; cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;"
      " mov.b32 %0, {lo, hi}; }"
      : "=r"(d)
      : "r"(a), "r"(b));
  return d;
}

// The scale that a page held: an ordinary load, because the same kernel stores there
// (this warp alone, what it makes of the value; so the load needs no other order).
__device__ __forceinline__ float ld_held_f32(const float* ptr) {
  KVC_GUARD(ptr, 4, return 0.0f);
  float v;
  asm("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(ptr));
  return v;
}

// R: 16-byte chunks of new values a lane holds; a page with more new tokens
// than 32 R chunks is read twice, the second time from L2.
template <int DT, int D, int R>
__global__ void __launch_bounds__(kWarps * 32, R == 8 ? 4 : 2) c8_write_kernel(const __grid_constant__ C8Params p) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a token's row, rows a warp loads at once
  const uint32_t lane = threadIdx.x & 31u;
  PageJob j;
  if (!page_job(p, blockIdx.x * kWarps + (threadIdx.x >> 5), j) || j.id < 0 || j.t0 >= j.t1) return;
  const int sub = lane / LPR, c8 = (lane % LPR) * 8;
  const int first = j.t0 + sub;
  for (uint32_t role = j.role; role < j.role + j.roles; ++role) {
    const int64_t rs = role ? p.b_row : p.a_row;
    // this lane's chunk of its first new token, and the steps to the next ones
    const uint16_t* src = (role ? p.b : p.a) + (int64_t)j.head * (role ? p.b_head : p.a_head) + c8 + (j.row0 + first) * rs;
    uint8_t* page = (role ? p.v : p.k) + (int64_t)j.id * p.sb + (int64_t)j.head * p.sh + c8;
    uint8_t* dst = page + (int64_t)first * p.st;
    const int64_t src_step = RPI * rs, dst_step = RPI * p.st;
    float* scale_at = (role ? p.v_scale : p.k_scale) + (int64_t)j.id * p.H + j.head;
    const float was = j.t0 > 0 ? ld_held_f32(scale_at) : 0.0f;

    uint4 w[R];
    uint32_t m = 0;
    {
      const uint16_t* at = src;
      for (int t = first; t - sub < j.t1; t += R * RPI) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          w[r] = t + r * RPI < j.t1 ? ld_stream16(at) : make_uint4(0, 0, 0, 0);
          at += src_step;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          m = max2<DT>(m, w[r].x);
          m = max2<DT>(m, w[r].y);
          m = max2<DT>(m, w[r].z);
          m = max2<DT>(m, w[r].w);
        }
      }
    }
    float amax = fmaxf(lo_f32<DT>(m), hi_f32<DT>(m));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!(amax < __uint_as_float(0x7f800000u))) {  // infinities among the new values: the largest without them
      m = 0;
      const uint16_t* at = src;
      for (int t = first; t < j.t1; t += RPI, at += src_step) {
        const uint4 x = ld_stream16(at);
        m = max2<DT>(m, drop_nonfinite2<DT>(x.x));
        m = max2<DT>(m, drop_nonfinite2<DT>(x.y));
        m = max2<DT>(m, drop_nonfinite2<DT>(x.z));
        m = max2<DT>(m, drop_nonfinite2<DT>(x.w));
      }
      __syncwarp();
      amax = fmaxf(lo_f32<DT>(m), hi_f32<DT>(m));
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    float scale = page_scale(amax);
    if (j.t0 > 0) {
      if (scale > was) {  // the earlier tokens' codes under the larger scale
        const float f = was / scale;
        for (int t = sub; t < j.t0; t += RPI) {
          uint2* at = reinterpret_cast<uint2*>(page + (int64_t)t * p.st);
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
    // FP16 values times a power of two that FP16 has are exact but below 2^-14, far under half of E4M3's
    // smallest step (2^-10)
    const uint32_t inv2 = DT == 0 ? half2_pow2(inv) : 0u;
    const bool again = j.t1 - j.t0 > R * RPI;
    const uint16_t* at = src;
    for (int t = first; t - sub < j.t1; t += R * RPI) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (t + r * RPI < j.t1) {
          if (again) w[r] = ld_nc16(at);
          uint2 y;
          if (DT == 0 && inv2) {
            y.x = enc_h4(hmul2(w[r].x, inv2), hmul2(w[r].y, inv2));
            y.y = enc_h4(hmul2(w[r].z, inv2), hmul2(w[r].w, inv2));
          } else {
            float x[8];
            unpack8<DT>(w[r], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            y = make_uint2(c8_enc4(x[0], x[1], x[2], x[3]), c8_enc4(x[4], x[5], x[6], x[7]));
          }
          st8(dst, y);
        }
        at += src_step;
        dst += dst_step;
      }
    }
    if (lane == 0 && scale != was) st4(scale_at, __float_as_uint(scale));
    __syncwarp();
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32) c8_read_kernel(const __grid_constant__ C8Params p) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, U = 8;
  const uint32_t lane = threadIdx.x & 31u;
  PageJob j;
  if (!page_job(p, blockIdx.x * kWarps + (threadIdx.x >> 5), j)) return;
  const int sub = lane / LPR, c8 = (lane % LPR) * 8;
  for (uint32_t role = j.role; role < j.role + j.roles; ++role) {
    uint16_t* out = (role ? p.b : p.a) + (int64_t)j.head * (role ? p.b_head : p.a_head) + c8;
    const int64_t rs = role ? p.b_row : p.a_row;
    if (j.q.unit == 0u)  // rows before the sequence's first token
      for (int i = sub; i < min(-j.q.start, j.q.n_new); i += RPI)
        st16(out + ((int64_t)j.q.row + i) * rs, make_uint4(0, 0, 0, 0));
    if (j.t0 >= j.t1) continue;
    const int first = j.t0 + sub;
    const uint8_t* src = (role ? p.v : p.k) + (int64_t)j.id * p.sb + (int64_t)j.head * p.sh + c8 + (int64_t)first * p.st;
    uint16_t* dst = out + (j.row0 + first) * rs;
    const int64_t src_step = RPI * p.st, dst_step = RPI * rs;
    const float scale = j.id < 0 ? 0.0f : ldg_f32((role ? p.v_scale : p.k_scale) + (int64_t)j.id * p.H + j.head);
    // FP16: a power of two that FP16 has multiplies with the one rounding of the result; from 2^8 on a product
    // may pass 65504 and saturates (a code next to 448 under the scale of values next to 65504 stands for
    // 65536).  bf16 holds every code * scale exactly.
    const uint32_t scale2 = DT == 0 && scale < 256.0f ? half2_pow2(scale) : 0u;
    for (int t = first; t - sub < j.t1; t += U * RPI) {
      uint2 c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        c[u] = t + u * RPI < j.t1 && j.id >= 0 ? ld_nc8(src) : make_uint2(0, 0);
        src += src_step;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * RPI < j.t1) {
          uint32_t h[4];
          c8_dec4(c[u].x, h[0], h[1]);
          c8_dec4(c[u].y, h[2], h[3]);
          uint4 y;
          if (DT == 0 && scale2) {
            y = make_uint4(hmul2(h[0], scale2), hmul2(h[1], scale2), hmul2(h[2], scale2), hmul2(h[3], scale2));
          } else {
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = c8_h2f(h[k]);
              x[2 * k] = f.x * scale;
              x[2 * k + 1] = f.y * scale;
            }
            if (DT == 0) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                x[k] = x[k] > 65504.0f ? 65504.0f : x[k];  // comparisons keep NaN
                x[k] = x[k] < -65504.0f ? -65504.0f : x[k];
              }
            }
            y = pack8<DT>(x);
          }
          st16(dst, y);
        }
        dst += dst_step;
      }
    }
  }
}

template <typename F>
int launch_pages(F kernel, const C8Params& p, void* stream) {
  C8Params c = p;
  // K and V in one warp where that leaves 32 warps an SM
  c.both_roles = (uint64_t)p.H * p.n_units >= 32ull * kC8Sms ? 1u : 0u;
  const uint64_t warps = (c.both_roles ? 1ull : 2ull) * p.H * p.n_units;
  const uint64_t grid = (warps + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<(unsigned)grid, kWarps * 32, 0, (cudaStream_t)stream>>>(c);
        return cudaGetLastError();
      },
      c);
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
