// cache8_step.cu -- attention of few query rows over the 8-bit cache: single
// tokens, drafted tokens, short chunks.
//
//   z_rj = scale s_k(j) (q_r . k_j),  out_r = sum_j 2^(z_rj - m_r) s_v(j) v_j / l_r
//
// Bound by reading the codes once (2 D bytes a token and KV head).  A CTA takes
// a row tile of one sequence and KV head (16 rows: the G query heads that share
// the KV head, times the new tokens) over one range of its keys; its warps walk
// the range 16 tokens at a time, each on its own, and join at the end.  Ranges
// of one row tile are joined by the CTA that finishes last, in range order, so
// the result does not depend on timing.
//
// Tiles go from global memory to the lane that needs them: the order in which
// dims and tokens are fed to the 16x8x16 matrix products is free as long as both
// operands agree, and is chosen such that a lane's K fragment is 16 contiguous
// codes of a token and its V fragment 16 contiguous codes of four tokens.  Each
// lane copies these asynchronously into shared memory slots of its own
// (cp.async), several tiles ahead: no lane reads another's slot, so the walk
// needs no barrier.  Codes become FP16 exactly; K's scale multiplies the scores,
// V's scale the weights.
#include "cache8_common.cuh"

namespace kvc {
namespace {

constexpr int kStepWarps = 4;
constexpr float kNegInf = -INFINITY;
// Weights are held as 2^(z - m) * 2^11 (in the factor that carries V's scale): FP16 then keeps 11 bits down to 2^-25
// of the row's largest weight, below that 2^-36 of it.  m may lag the true maximum
// by kLag (fewer rescalings of the sums): 2^(11 + kLag) = 2^15 < 65504.
constexpr float kLift = 2048.0f, kLag = 4.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copy N bytes to a shared slot, zeros when !ok.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t smem, const void* src, bool ok) {
#ifdef KVC_BOUNDS_CHECK
  if (ok && !dbg_ok(src, N)) ok = false;
#endif
  const uint32_t n = ok ? N : 0;
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem), "l"(src), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
struct StepShape {
  static constexpr int CH = D >= 64 ? 16 : 8;          // bytes of a K copy
  static constexpr int KC = D / 4 / CH;                // K copies of a lane and token
  static constexpr int VB = D / 8 >= 16 ? 16 : D / 8;  // bytes of a V copy
  static constexpr int VC = D / 8 / VB;                // V copies of a lane and token
  static constexpr int KS = D / 16;                    // k-steps of the score product
  static constexpr int NT = D / 8;                     // 8-wide column tiles of the output
  static constexpr int kTile = 32 * (2 * KC * CH + 4 * VC * VB);  // bytes of K and V of 16 tokens
};

// Shared memory of a warp's slots: [stage][K copies, V copies, scales][lane].
template <int D, bool PAGED16>
struct StepSmem {
  using S = StepShape<D>;
  static constexpr int kScales = PAGED16 ? 2 : 8;      // FP32 words of a lane: K and V scales
  static constexpr int kStage = S::kTile + 32 * 4 * kScales;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 4 : D == 64 ? 6 : 8;
  static constexpr int kQ = 16 * D * 2;
  static constexpr int kJoin = kStepWarps * 16 * (D + 4) * 4;  // the warps' sums, over the slots
  static constexpr int kSlots = kStepWarps * kStages * kStage;
  static constexpr int kBytes = kQ + 512 + (kSlots > kJoin ? kSlots : kJoin);
};

// loads of what other CTAs of this launch have stored (L2)
__device__ __forceinline__ float2 ld_join2(const float* ptr) {
  KVC_GUARD(ptr, 8, return make_float2(0.f, 0.f));
  return __ldcg(reinterpret_cast<const float2*>(ptr));
}
__device__ __forceinline__ float4 ld_join4(const float* ptr) {
  KVC_GUARD(ptr, 16, return make_float4(0.f, 0.f, 0.f, 0.f));
  return __ldcg(reinterpret_cast<const float4*>(ptr));
}

// One bit per byte of w that is an E4M3 NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// 4 tokens x 4 dims: word t holds token t's codes of dims 0..3; out word d the
// codes of tokens 0..3 at dim d.
__device__ __forceinline__ void transpose4(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t (&o)[4]) {
  const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w2, w3, 0x5140);  // (0,0')(1,1')
  const uint32_t c = __byte_perm(w0, w1, 0x7362), d = __byte_perm(w2, w3, 0x7362);
  o[0] = __byte_perm(a, b, 0x5410);
  o[1] = __byte_perm(a, b, 0x7632);
  o[2] = __byte_perm(c, d, 0x5410);
  o[3] = __byte_perm(c, d, 0x7632);
}

// PAGED16: pages are whole 16-token tiles, so a tile has one page and one pair
// of scales; otherwise each lane looks its tokens' pages up by itself.
template <int DT, int D, bool PAGED16>
__global__ void __launch_bounds__(kStepWarps * 32) c8_step_kernel(const __grid_constant__ C8Params p) {
  using S = StepShape<D>;
  using M = StepSmem<D, PAGED16>;
  constexpr int NS = M::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t g = lane >> 2, qd = lane & 3u;
  const uint32_t head = blockIdx.y;
  const uint32_t u = blockIdx.x / p.splits, split = blockIdx.x - u * p.splits;

  const uint32_t tiles1 = (p.G + kStepRows - 1) / kStepRows;
  const C8Seq q = c8_find(p, u, p.G, kStepRows, 1u, tiles1);
  const uint32_t rows = (uint32_t)q.n_new * p.G, r0 = q.unit * kStepRows;
  if (r0 >= rows || rows < p.min_rows || rows > p.max_rows) return;
  const uint32_t n_rows = min(kStepRows, rows - r0);

  // the keys that some row of the tile sees
  const int32_t first_pos = q.start + (int32_t)(r0 / p.G), last_pos = q.start + (int32_t)((r0 + n_rows - 1u) / p.G);
  int32_t hi = p.causal ? min(q.len, last_pos + 1) : q.len;
  int32_t lo = p.window ? max(0, first_pos - (int32_t)min(p.window, 0x7fffffffu) + 1) : 0;
  hi = max(hi, 0);
  if (first_pos < 0) lo = 0;
  lo &= ~15;  // tiles start at multiples of 16
  const uint32_t keys = hi > lo ? (uint32_t)(hi - lo) : 0u;
  // ranges: p.chunk keys each, longer where p.splits of them would not reach
  uint32_t chunk = p.chunk;
  if ((uint64_t)chunk * p.splits < keys) chunk = ((keys + p.splits - 1) / p.splits + 15u) & ~15u;
  const uint32_t n_split = keys ? (keys + chunk - 1) / chunk : 1u;
  if (split >= n_split) return;
  const int32_t c_lo = lo + (int32_t)(split * chunk);
  const int32_t c_hi = (int32_t)min((int64_t)hi, (int64_t)c_lo + chunk);

  // Q as FP16 fragments, rows scaled by a power of two into FP16's range (bf16;
  // exact but for values 2^-39 of the row's largest): lane (g, qd) of k-step
  // 4 c + i holds dims 64 c + 16 qd + 4 i .. + 3 (D = 32: 8 qd + 4 i) of rows g, g + 8.
  uint32_t* s_q = reinterpret_cast<uint32_t*>(smem);
  float* s_row = reinterpret_cast<float*>(smem + M::kQ);  // per row: scale * log2(e) / row scaling
  {
    // 8 threads to a row; each converts D / 8 dims
    const uint32_t r = tid >> 3, part = tid & 7u;
    constexpr int PER = D / 8;
    const bool in = r < n_rows;
    const uint32_t rr = r0 + (in ? r : 0u);
    const uint32_t tok = rr / p.G, hd = head * p.G + rr - tok * p.G;
    const uint16_t* src = p.a + ((int64_t)q.row + tok) * p.a_row + (int64_t)hd * p.a_head + part * PER;
    uint32_t w[PER / 2];
    if (PER >= 8) {
#pragma unroll
      for (int k = 0; k < PER / 8; ++k) {
        const uint4 x = in ? ld_nc16(src + 8 * k) : make_uint4(0, 0, 0, 0);
        w[(4 * k) % (PER / 2)] = x.x;
        w[(4 * k + 1) % (PER / 2)] = x.y;
        w[(4 * k + 2) % (PER / 2)] = x.z;
        w[(4 * k + 3) % (PER / 2)] = x.w;
      }
    } else {
      const uint2 x = in ? ld_nc8(src) : make_uint2(0, 0);
      w[0] = x.x;
      w[1] = x.y;
    }
    int ex = 0;
    if (DT == 1) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < PER / 2; ++k) {
        m = max(m, (w[k] & 0x7fffu) < 0x7f80u ? (w[k] & 0x7fffu) : 0u);
        m = max(m, ((w[k] >> 16) & 0x7fffu) < 0x7f80u ? ((w[k] >> 16) & 0x7fffu) : 0u);
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      // the largest magnitude, in [2^k, 2^(k+1)), goes to [2^14, 2^15)
      const int k = (int)(m >> 7) - 127;
      ex = m ? min(max(14 - k, -120), 120) : 0;
    }
    const float f = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
    for (int k = 0; k < PER / 2; ++k)
      if (DT == 1) w[k] = pack2<0>(lo_f32<1>(w[k]) * f, hi_f32<1>(w[k]) * f);
    // word k of this thread: dims part * PER + 2k, + 1
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) {
      const uint32_t dim = part * PER + 2 * k;
      uint32_t ks, l4, pair;
      if (D >= 64) {
        ks = (dim >> 6) * 4 + ((dim >> 2) & 3u);
        l4 = (dim >> 4) & 3u;
      } else {
        ks = (dim >> 2) & 1u;
        l4 = (dim >> 3) & 3u;
      }
      pair = (dim >> 1) & 1u;
      // fragment registers: a0 (row g, k lo), a1 (row g + 8, k lo), a2 (row g, k hi), a3 (row g + 8, k hi)
      s_q[(ks * 32 + (r & 7u) * 4 + l4) * 4 + pair * 2 + (r >> 3)] = w[k];
    }
    // two factors so that neither under- nor overflows alone
    if (part == 0) s_row[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
  }
  __syncthreads();

  // visible keys of this lane's rows g and g + 8
  int32_t vis_hi[2], vis_lo[2];
  float rf[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t r = g + 8 * h;
    const int32_t pos = q.start + (int32_t)((r0 + r) / p.G);
    vis_hi[h] = p.causal ? min(q.len, pos + 1) : q.len;
    vis_lo[h] = p.window ? (int32_t)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
    if (r >= n_rows || pos < 0) vis_hi[h] = 0;
    rf[h] = s_row[r];
  }
  // tiles between these need no mask
  const int32_t full_hi = first_pos < 0 ? 0 : p.causal ? min(q.len, first_pos + 1) : q.len;
  const int32_t full_lo = p.window ? (int32_t)max((int64_t)0, (int64_t)last_pos - p.window + 1) : 0;

  float o[S::NT][4];
#pragma unroll
  for (int n = 0; n < S::NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
  float vref = 1.17549435e-38f, vinv = 0.0f;  // V scales are held relative to the largest so far

  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(smem + M::kQ + 512) + warp * (NS * M::kStage);
  const int32_t n_tiles = (c_hi - c_lo + 15) / 16;
  const uint8_t* kbase = p.k + (int64_t)head * p.sh;
  const uint8_t* vbase = p.v + (int64_t)head * p.sh;
  bool bad = false;

  // page of tile t's tokens (PAGED16), one tile ahead of its use
  auto page_of = [&](int32_t t) -> int32_t {
    const int32_t tok = c_lo + 16 * t;
    return tok < c_hi ? c8_page(p, q.s, c8_div_t(p, (uint32_t)tok)) : -2;
  };
  auto issue = [&](int32_t t, int stage, int32_t id) {
    const uint32_t at = slots + stage * M::kStage;
    const int32_t tok0 = c_lo + 16 * t;
    if (PAGED16) {
      const uint32_t in_page = (uint32_t)tok0 - c8_div_t(p, (uint32_t)tok0) * p.T;
      const bool page_ok = id >= 0;
      if (id == -1) bad = true;
      const int64_t off = page_ok ? (int64_t)id * p.sb + (int64_t)in_page * p.st : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t tt = g + 8 * h;
        const bool ok = page_ok && tok0 + (int32_t)tt < c_hi;
        const uint8_t* src = kbase + (ok ? off + (int64_t)tt * p.st : 0);
#pragma unroll
        for (int c = 0; c < S::KC; ++c)
          cp_async<S::CH>(at + ((h * S::KC + c) * 32 + lane) * S::CH, src + c * 4 * S::CH + qd * S::CH, ok);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t tt = 2 * qd + (i & 1) + 8 * (i >> 1);
        const bool ok = page_ok && tok0 + (int32_t)tt < c_hi;
        const uint8_t* src = vbase + (ok ? off + (int64_t)tt * p.st : 0);
#pragma unroll
        for (int c = 0; c < S::VC; ++c)
          cp_async<S::VB>(at + 2 * S::KC * 32 * S::CH + ((i * S::VC + c) * 32 + lane) * S::VB,
                          src + c * 8 * S::VB + g * S::VB, ok);
      }
      const int64_t si = page_ok ? (int64_t)id * p.H + head : 0;
      cp_async<4>(at + S::kTile + lane * 4, p.k_scale + si, page_ok);
      cp_async<4>(at + S::kTile + 128 + lane * 4, p.v_scale + si, page_ok);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t tok = tok0 + (int32_t)(g + 8 * h);
        bool ok = tok < c_hi;
        const uint32_t pi = c8_div_t(p, (uint32_t)tok);
        const int32_t pid = ok ? c8_page(p, q.s, pi) : -1;
        if (ok && pid < 0) bad = true;
        ok = ok && pid >= 0;
        const uint8_t* src = kbase + (ok ? (int64_t)pid * p.sb + (int64_t)((uint32_t)tok - pi * p.T) * p.st : 0);
#pragma unroll
        for (int c = 0; c < S::KC; ++c)
          cp_async<S::CH>(at + ((h * S::KC + c) * 32 + lane) * S::CH, src + c * 4 * S::CH + qd * S::CH, ok);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t tok = tok0 + (int32_t)(2 * qd + (i & 1) + 8 * (i >> 1));
        bool ok = tok < c_hi;
        const uint32_t pi = c8_div_t(p, (uint32_t)tok);
        const int32_t pid = ok ? c8_page(p, q.s, pi) : -1;
        ok = ok && pid >= 0;
        const uint8_t* src = vbase + (ok ? (int64_t)pid * p.sb + (int64_t)((uint32_t)tok - pi * p.T) * p.st : 0);
#pragma unroll
        for (int c = 0; c < S::VC; ++c)
          cp_async<S::VB>(at + 2 * S::KC * 32 * S::CH + ((i * S::VC + c) * 32 + lane) * S::VB,
                          src + c * 8 * S::VB + g * S::VB, ok);
        // a scale of 0 marks a token without a page
        const int64_t si = ok ? (int64_t)pid * p.H + head : 0;
        cp_async<4>(at + S::kTile + (i * 32 + lane) * 4, p.k_scale + si, ok);
        cp_async<4>(at + S::kTile + ((4 + i) * 32 + lane) * 4, p.v_scale + si, ok);
      }
    }
  };

  int32_t next_id = PAGED16 ? page_of((int32_t)warp) : 0;
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    const int32_t t = (int32_t)warp + s * kStepWarps;
    const int32_t id = next_id;
    if (t < n_tiles) {
      if (PAGED16) next_id = page_of(t + kStepWarps);
      issue(t, s, id);
    }
    cp_commit();
  }
  int stage = 0;
  for (int32_t t = (int32_t)warp; t < n_tiles; t += kStepWarps) {
    {
      const int32_t tn = t + (NS - 1) * kStepWarps;
      const int sn = stage == 0 ? NS - 1 : stage - 1;
      if (tn < n_tiles) {
        const int32_t id = next_id;
        if (PAGED16) next_id = page_of(tn + kStepWarps);
        issue(tn, sn, id);
      }
      cp_commit();
      cp_wait<NS - 1>();
    }
    const uint8_t* sp = smem + M::kQ + 512 + warp * (NS * M::kStage) + stage * M::kStage;
    stage = stage == NS - 1 ? 0 : stage + 1;
    const int32_t tok0 = c_lo + 16 * t;

    // scores of 16 tokens: s[h][.] for tokens 8 h + 2 qd, + 1
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < S::KC; ++c) {
      uint32_t kw[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* at = sp + ((h * S::KC + c) * 32 + lane) * S::CH;
        if (S::CH == 16) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          kw[h][0] = x.x; kw[h][1] = x.y; kw[h][2] = x.z; kw[h][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          kw[h][0] = x.x; kw[h][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < S::CH / 4; ++i) {
        const uint4 a = *reinterpret_cast<const uint4*>(s_q + ((c * (S::CH / 4) + i) * 32 + lane) * 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b0, b1;
          c8_dec4(kw[h][i], b0, b1);
          mma16816(s[h], a.x, a.y, a.z, a.w, b0, b1);
        }
      }
    }
    float ks[4], vs[4];
    if (PAGED16) {
      ks[0] = ks[1] = ks[2] = ks[3] = *reinterpret_cast<const float*>(sp + S::kTile + lane * 4);
      vs[0] = vs[1] = vs[2] = vs[3] = *reinterpret_cast<const float*>(sp + S::kTile + 128 + lane * 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ks[i] = *reinterpret_cast<const float*>(sp + S::kTile + (i * 32 + lane) * 4);
        vs[i] = *reinterpret_cast<const float*>(sp + S::kTile + ((4 + i) * 32 + lane) * 4);
      }
    }
    // tokens without a page have the scale 0 of a skipped copy
    const bool no_page = PAGED16 ? ks[0] == 0.0f : __any_sync(0xffffffffu, ks[0] == 0.0f || ks[1] == 0.0f || ks[2] == 0.0f || ks[3] == 0.0f);
    const bool masked = no_page || tok0 + 16 > full_hi || tok0 < full_lo;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[h][e] = (s[h][e] * ks[2 * h + (e & 1)]) * rf[e >> 1];
    if (masked) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t tok = tok0 + (int32_t)(8 * h + 2 * qd + (e & 1));
          const int r = e >> 1;
          if (tok >= vis_hi[r] || tok < vis_lo[r] || ks[2 * h + (e & 1)] == 0.0f) s[h][e] = kNegInf;
        }
    }
    // running maxima; the sums are rescaled only where a maximum grew by more than kLag
    bool grow = false;
    float mt[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      mt[r] = x;
      grow |= x > m[r] + kLag;  // -inf + kLag = -inf: any finite score of a fresh row
    }
    float vt = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
    if (!PAGED16) {
      vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 1));
      vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 2));
    }
    if (__any_sync(0xffffffffu, grow || vt > vref)) {
      const float vn = fmaxf(vt, vref);
      const float fv = vref / vn;
      vref = vn;
      vinv = kLift / vn;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mn = mt[r] > m[r] + kLag ? mt[r] : m[r];
        const float f = m[r] == kNegInf ? 0.0f : ex2(m[r] - mn);
        m[r] = mn;
        l[r] *= f;
        const float fo = f * fv;
#pragma unroll
        for (int n = 0; n < S::NT; ++n) {
          o[n][2 * r] *= fo;
          o[n][2 * r + 1] *= fo;
        }
      }
    }
    float vr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) vr[i] = PAGED16 && i ? vr[0] : vs[i] * vinv;
    uint32_t pa[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[r] == kNegInf ? 0.0f : m[r];
        const float p0 = ex2(s[h][2 * r] - base), p1 = ex2(s[h][2 * r + 1] - base);
        l[r] += p0 + p1;
        // a weight of 0 stays 0 whatever the scale (a masked token of a page that holds infinities)
        const float w0 = p0 == 0.0f ? 0.0f : p0 * vr[2 * h], w1 = p1 == 0.0f ? 0.0f : p1 * vr[2 * h + 1];
        pa[2 * h + r] = pack2<0>(w0, w1);
      }
    // V: the lane's four tokens, transposed to pairs of tokens per dim
    uint32_t any_nan = 0;
#pragma unroll
    for (int c = 0; c < S::VC; ++c) {
      uint32_t vw[4][S::VB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* at = sp + 2 * S::KC * 32 * S::CH + ((i * S::VC + c) * 32 + lane) * S::VB;
        if (S::VB == 16) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          vw[i][0] = x.x;
          vw[i][1 % (S::VB / 4)] = x.y;
          vw[i][2 % (S::VB / 4)] = x.z;
          vw[i][3 % (S::VB / 4)] = x.w;
        } else if (S::VB == 8) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          vw[i][0] = x.x;
          vw[i][1 % (S::VB / 4)] = x.y;
        } else {
          vw[i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      if (masked) {
        // a NaN that some row does not see must not reach it through 0 * NaN:
        // NaN codes become 0 here and are put back below where they are seen
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < S::VB / 4; ++k) {
            const uint32_t nb = nan_bytes(vw[i][k]);
            any_nan |= nb;
            vw[i][k] &= ~((nb >> 7) * 0xffu);
          }
      }
#pragma unroll
      for (int k = 0; k < S::VB / 4; ++k) {
        uint32_t tr[4];
        transpose4(vw[0][k], vw[1][k], vw[2][k], vw[3][k], tr);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t b0, b1;
          c8_dec4(tr[d], b0, b1);
          mma16816(o[c * S::VB + 4 * k + d], pa[0], pa[1], pa[2], pa[3], b0, b1);
        }
      }
    }
    if (masked && __any_sync(0xffffffffu, any_nan != 0u)) {
      // rows x dims where a visible token's value is NaN: count them with the same product
      uint32_t seen[4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          seen[2 * h + r] = (s[h][2 * r] == kNegInf ? 0u : 0x3c00u) | (s[h][2 * r + 1] == kNegInf ? 0u : 0x3c000000u);
#pragma unroll
      for (int c = 0; c < S::VC; ++c)
#pragma unroll
        for (int k = 0; k < S::VB / 4; ++k) {
          uint32_t w[4], tr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint32_t*>(
                       sp + 2 * S::KC * 32 * S::CH + ((i * S::VC + c) * 32 + lane) * S::VB + 4 * k);
          transpose4(nan_bytes(w[0]), nan_bytes(w[1]), nan_bytes(w[2]), nan_bytes(w[3]), tr);
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            // 0x80 bytes -> 1.0 halves
            const uint32_t b0 = (tr[d] & 0x80u ? 0x3c00u : 0u) | (tr[d] & 0x8000u ? 0x3c000000u : 0u);
            const uint32_t b1 = (tr[d] & 0x800000u ? 0x3c00u : 0u) | (tr[d] & 0x80000000u ? 0x3c000000u : 0u);
            float cnt[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(cnt, seen[0], seen[1], seen[2], seen[3], b0, b1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cnt[e] > 0.0f) o[c * S::VB + 4 * k + d][e] = __int_as_float(0x7fffffff);
          }
        }
    }
  }
  cp_wait<0>();
  if (PAGED16 ? (bad && lane == 0u) : bad) c8_error(p, q.s, KV_CACHE8_BAD_PAGE);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }

  // ---- join the warps: every row to the largest maximum among them
  __syncthreads();
  float* s_m = reinterpret_cast<float*>(smem + M::kQ);  // [row][warp] maxima, then the tile's
  float* s_o = reinterpret_cast<float*>(smem + M::kQ + 512);  // [warp][16][D + 4]
  float* s_l = reinterpret_cast<float*>(smem);          // [row][warp]
  constexpr int OS = D + 4;
  if (qd == 0) {
    s_m[g * kStepWarps + warp] = m[0];
    s_m[(g + 8) * kStepWarps + warp] = m[1];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t row = g + 8 * r;
    float mx = kNegInf;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) mx = fmaxf(mx, s_m[row * kStepWarps + w]);
    const float f = m[r] == kNegInf ? 0.0f : ex2(m[r] - mx);
    const float fo = m[r] == kNegInf ? 0.0f : f * (vref * (1.0f / kLift));
    if (qd == 0) s_l[row * kStepWarps + warp] = l[r] * f;
    // column 2 qd + e of tile n is dim (2 qd + e) * VB + (n mod VB) of its 8 VB dims
    float* dst = s_o + (warp * 16 + row) * OS;
#pragma unroll
    for (int c = 0; c < S::VC; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < S::VB; k += 4) {
          const int n = c * S::VB + k;
          *reinterpret_cast<float4*>(dst + c * 8 * S::VB + (2 * qd + e) * S::VB + k) =
              make_float4(o[n][2 * r + e] * fo, o[n + 1][2 * r + e] * fo, o[n + 2][2 * r + e] * fo,
                          o[n + 3][2 * r + e] * fo);
        }
  }
  __syncthreads();
  // 8 threads to a row, D / 8 dims each (4 at a time, 32 apart)
  const uint32_t row = tid >> 3, part = tid & 7u;
  float mx = kNegInf, ls = 0.0f;
#pragma unroll
  for (int w = 0; w < kStepWarps; ++w) {
    mx = fmaxf(mx, s_m[row * kStepWarps + w]);
    ls += s_l[row * kStepWarps + w];
  }
  float acc[D / 8];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(s_o + (w * 16 + row) * OS + c * 32 + part * 4);
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
    acc[4 * c] = x.x; acc[4 * c + 1] = x.y; acc[4 * c + 2] = x.z; acc[4 * c + 3] = x.w;
  }
  const uint32_t job = u * p.H + head;
  if (n_split > 1u) {
    // ---- leave the range's sums; the last CTA of the job joins the ranges
    float* base = p.partials + (uint64_t)job * p.splits * (kStepRows * (D + 2));
    float* mine = base + (uint64_t)split * (kStepRows * (D + 2));
    if (row < n_rows) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        st16(mine + row * D + c * 32 + part * 4,
             make_uint4(__float_as_uint(acc[4 * c]), __float_as_uint(acc[4 * c + 1]), __float_as_uint(acc[4 * c + 2]),
                        __float_as_uint(acc[4 * c + 3])));
      if (part == 0) st8(mine + kStepRows * D + 2 * row, make_uint2(__float_as_uint(mx), __float_as_uint(ls)));
    }
    __syncthreads();
    uint32_t* s_last = reinterpret_cast<uint32_t*>(smem + M::kQ);
    if (tid == 0) {
      uint32_t last = 0;
      KVC_GUARD(p.tickets + job, 4, last = 2);
      if (last == 0) {
        __threadfence();
        last = atomicAdd(p.tickets + job, 1u) == n_split - 1u ? 1u : 0u;
        if (last) p.tickets[job] = 0;  // as the next call finds it
        __threadfence();
      }
      *s_last = last;
    }
    __syncthreads();
    if (*s_last != 1u) return;
    // maxima first, then the sums, in range order
    mx = kNegInf;
    if (row < n_rows)
      for (uint32_t k = 0; k < n_split; ++k)
        mx = fmaxf(mx, ld_join2(base + (uint64_t)k * (kStepRows * (D + 2)) + kStepRows * D + 2 * row).x);
    ls = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) acc[k] = 0.0f;
    if (row < n_rows)
      for (uint32_t k = 0; k < n_split; ++k) {
        const float* part_k = base + (uint64_t)k * (kStepRows * (D + 2));
        const float2 ml = ld_join2(part_k + kStepRows * D + 2 * row);
        const float f = ml.x == kNegInf ? 0.0f : ex2(ml.x - mx);
        ls += ml.y * f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const float4 y = ld_join4(part_k + row * D + c * 32 + part * 4);
          acc[4 * c] += y.x * f;
          acc[4 * c + 1] += y.y * f;
          acc[4 * c + 2] += y.z * f;
          acc[4 * c + 3] += y.w * f;
        }
      }
  }
  if (row >= n_rows) return;
  const uint32_t rr = r0 + row, tok = rr / p.G, hd = head * p.G + rr - tok * p.G;
  const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
  uint16_t* out = p.b + ((int64_t)q.row + tok) * p.b_row + (int64_t)hd * p.b_head;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    st8(out + c * 32 + part * 4,
        ls == 0.0f ? make_uint2(0, 0)
                   : make_uint2(pack2<DT>(acc[4 * c] * inv, acc[4 * c + 1] * inv),
                                pack2<DT>(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv)));
  if (p.lse && part == 0)
    st4(p.lse + ((int64_t)q.row + tok) * p.HQ + hd,
        __float_as_uint(ls == 0.0f ? kNegInf : (mx + log2f(ls)) * 0.693147180559945309f));
}

template <int DT, int D, bool PAGED16>
int step_launch(const C8Params& p, void* stream) {
  constexpr int bytes = StepSmem<D, PAGED16>::kBytes;
  const auto kernel = c8_step_kernel<DT, D, PAGED16>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return KV_ERR_CUDA;
  const uint64_t gx = (uint64_t)p.n_units * p.splits;
  if (gx > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<dim3((unsigned)gx, p.H), kStepWarps * 32, bytes, (cudaStream_t)stream>>>(p);
        return cudaGetLastError();
      },
      p);
}

template <int DT, int D>
int step_d(const C8Params& p, void* stream) {
  return p.T % 16 == 0 ? step_launch<DT, D, true>(p, stream) : step_launch<DT, D, false>(p, stream);
}

}  // namespace

int launch_c8_step(const C8Params& p, void* stream) { KVC_C8_DISPATCH(step_d, p, stream); }

}  // namespace kvc
