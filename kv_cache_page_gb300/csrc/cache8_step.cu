// cache8_step.cu -- attention of few query rows over the 8-bit cache: single
// tokens, drafted tokens, short chunks.
//
//   z_rj = scale s_k(j) (q_r . k_j),  out_r = sum_j 2^(z_rj - m_r) s_v(j) v_j / l_r
//
// Bound by reading the codes once (2 D bytes a token and KV head).  A CTA takes
// a row tile of one sequence and KV head (16 rows: the G query heads that share
// the KV head, times the new tokens) over one range of its keys; its warps walk
// the range 32 tokens at a time (16 for D = 256), each on its own, and join at the
// end.  Ranges of one row tile are joined by the CTA that finishes last, in range
// order, so the result does not depend on timing.
//
// A warp copies its tiles asynchronously into shared memory slots of its own
// (cp.async), a stage or more ahead; no barrier is needed in the walk.  The order
// in which dims are fed to the 16x8x16 score product is free as long as both
// operands agree, and is chosen such that a lane's K fragment is 16 contiguous
// codes of a token, read from slots that the lane itself copied.  V's fragments
// need runs of tokens at one dim: 16 x 16 byte tiles transposed by ldmatrix, rows
// swizzled over the banks.  The tokens of a 16-token tile are dealt to the score
// product's columns such that its result is the second product's operand as it
// stands (see tok_of).  Codes become FP16 exactly; K's scale multiplies the scores,
// V's scale the weights.
//
// What the walk costs besides bytes is instructions, at 12 warps an SM: per 16
// tokens and D = 128, 64 conversions and 32 products (16 with at most 8 query rows)
// are the floor.  Measured on a GB300, 8 heads of 128: 64 sequences of 100 to 8192 tokens
// 66 us (4.4 TB/s of codes), one of 131072 with 4 heads 36 us (3.8).
#include <type_traits>

#include "cache8_common.cuh"

namespace kvc {
namespace {

constexpr float kNegInf = -INFINITY;
// Weights are held as 2^(z - m) * 2^11 (in the factor that carries V's scale):
// FP16 then keeps 11 bits down to 2^-25 of the row's largest weight, below that
// 2^-36 of it.  m may lag the true maximum by kLag (fewer rescalings of the sums):
// 2^(11 + kLag) = 2^15 < 65504.
constexpr float kLift = 2048.0f, kLag = 4.0f;
// Sums of weights times V that warps and ranges join are held 2^-24 times as large: with V next to 2^128 they
// would leave FP32's range before they are normalised (2^20 keys, each weight up to 2^kLag, still fit).
constexpr float kJoin = 16777216.0f;

// A barrier of the CTA that counts threads, whether or not their warp is
// converged (__syncthreads() asks for converged warps, and the branches here on
// one thread's bookkeeping and on loaded values do not promise that).
__device__ __forceinline__ void cta_sync() { asm volatile("barrier.sync 0;" ::: "memory"); }

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

// Copy N bytes to a shared slot; zeros when !ok.
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
template <int N>
__device__ __forceinline__ void cp_async(uint32_t smem, const void* src) {
  KVC_GUARD(src, N, return);
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two 16 x 16 byte tiles, transposed: lanes 0-15 give the rows' addresses of the
// first, lanes 16-31 of the second; r0, r1 (second: r2, r3) hold rows 4 (lane & 3)
// .. + 3 of column lane >> 2 and of column (lane >> 2) + 8.
__device__ __forceinline__ void ldsm_t16x2(uint32_t (&r)[4], uint32_t smem) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem));
}

template <int D>
struct StepShape {
  static constexpr int TS = D == 256 ? 16 : 32;        // tokens of a warp's step
  static constexpr int HT = TS / 16;                   // 16-token tiles of a step
  static constexpr int CH = D >= 64 ? 16 : 8;          // bytes of a K copy
  static constexpr int KC = D / 4 / CH;                // K copies of a lane and token
  static constexpr int VR = 512 / D;                   // token rows that a warp's 16-byte V copies cover
  static constexpr int kK = TS * D;                    // bytes of a stage's K and of its V
  // and FP32 scales of K and V per token; V tiles start at multiples of a row (addressed by xor)
  static constexpr int kStage = 2 * kK + (TS == 16 ? 256 : 8 * TS);
  static_assert(kStage % 256 == 0, "");
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 2 : D == 64 ? 3 : 4;
  static constexpr int kQ = 16 * D * 2;
  static constexpr int kSmall = 2048;                  // rows' factors, maxima, sums
};
template <int D, int W>
constexpr int step_smem() {
  using S = StepShape<D>;
  constexpr int slots = W * S::kStages * S::kStage, join = W * 16 * (D + 4) * 4;
  constexpr int ranges = (int)kMaxSplits * 16 * 8;
  return S::kQ + S::kSmall + (slots > join ? (slots > ranges ? slots : ranges) : (join > ranges ? join : ranges));
}

// Column c of score tile h (8 wide) of a 16-token tile is token
// 4 (c >> 1) + (c & 1) + 2 h: the lane that holds columns 2 q, 2 q + 1 of both score
// tiles then holds tokens 4 q .. 4 q + 3, as ldmatrix deals V's rows.
__device__ __forceinline__ uint32_t tok_of(uint32_t c, uint32_t h) { return 4u * (c >> 1) + (c & 1u) + 2u * h; }

// Byte offset of 16-byte chunk c of token row t in a V tile: 8 consecutive rows
// of one chunk lie in 8 different bank groups.
template <int D>
__device__ __forceinline__ uint32_t v_at(uint32_t t, uint32_t c) {
  constexpr uint32_t R = D / 16;  // chunks of a row
  if (R >= 8) return t * D + ((c ^ (t & 7u)) << 4);
  if (R == 4) return t * D + ((c ^ ((t >> 1) & 3u)) << 4);
  return t * D + ((c ^ ((t >> 2) & 1u)) << 4);
}

// loads of what other CTAs of this launch have stored (L2)
__device__ __forceinline__ float2 ld_join2(const float* ptr) {
  KVC_GUARD(ptr, 8, return make_float2(0.f, 0.f));
  return __ldcg(reinterpret_cast<const float2*>(ptr));
}
__device__ __forceinline__ float4 ld_join4(const float* ptr) {
  KVC_GUARD(ptr, 16, return make_float4(0.f, 0.f, 0.f, 0.f));
  return __ldcg(reinterpret_cast<const float4*>(ptr));
}

// The high bit of each byte of w that is an E4M3 NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Transpose of an 8 x 8 tile of FP16, two values of a row to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// PAGED16: pages are whole 16-token tiles, so a tile lies in one page; otherwise
// every token's page is looked up by itself.
// N8: row tiles of at most 8 rows (one token and up to 8 query heads a KV head, the
// usual step).  The products then have the tokens (scores) and the dims (output) as
// their 16 rows and the 8 query rows as their columns: half the products, half the
// exponentials and half the accumulators of 16 query rows.  The fragments of K and V
// are the same; the weights pass through a transposition in registers.
template <int DT, int D, bool PAGED16, int W, bool N8>
__global__ void __launch_bounds__(W * 32, W == 4 ? (D == 256 ? 2 : 3) : 1)
    c8_step_kernel(const __grid_constant__ C8Params p) {
  using S = StepShape<D>;
  constexpr int NS = S::kStages, TS = S::TS, HT = S::HT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t g = lane >> 2, qd = lane & 3u;
  // heads next to each other: their rows of a page lie side by side, and are read at about the same time
  const uint32_t us = blockIdx.x / p.H, head = blockIdx.x - us * p.H;
  const uint32_t u = us / p.splits, split = us - u * p.splits;

  const C8Seq q = c8_find(p, u, p.G, kStepRows, 1u, p.per_seq);
  const uint32_t rows = (uint32_t)q.n_new * p.G, r0 = q.unit * kStepRows;
  if (r0 >= rows || rows < p.min_rows || rows > p.max_rows) return;
  const uint32_t n_rows = min(kStepRows, rows - r0);

  // the keys that some row of the tile sees
  const int32_t first_pos = q.start + (int32_t)(r0 / p.G), last_pos = q.start + (int32_t)((r0 + n_rows - 1u) / p.G);
  const int32_t hi = max(p.causal ? min(q.len, last_pos + 1) : q.len, 0);
  int32_t lo = p.window && first_pos >= 0 ? max(0, first_pos - (int32_t)min(p.window, 0x7fffffffu) + 1) : 0;
  if (PAGED16) lo &= ~15;  // a page's tiles start at multiples of 16; else the page of a token before may be freed
  const uint32_t keys = hi > lo ? (uint32_t)(hi - lo) : 0u;
  // ranges: p.chunk keys each, longer where p.splits of them would not reach
  uint32_t chunk = p.chunk;
  if ((uint64_t)chunk * p.splits < keys) chunk = ((keys + p.splits - 1) / p.splits + 31u) & ~31u;
  const uint32_t n_split = keys ? (keys + chunk - 1) / chunk : 1u;
  if (split >= n_split) return;
  const int32_t c_lo = lo + (int32_t)(split * chunk);
  const int32_t c_hi = (int32_t)min((int64_t)hi, (int64_t)c_lo + chunk);
  const int32_t n_steps = (c_hi - c_lo + TS - 1) / TS;

  uint8_t* my_slots = smem + S::kQ + S::kSmall + warp * (NS * S::kStage);
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(my_slots);
  bool bad = false;

  // this lane's copies: K tokens tok_of(g, h) at dims of its quad; V chunk lane % (D / 16) of rows
  // v_row + VR i, whose place in the V tile repeats every NV rows but for i VR D bytes.
  const uint32_t v_row = lane / (D / 16), v_chunk = lane % (D / 16);
  const uint8_t* k_src = p.k + (int64_t)head * p.sh + qd * S::CH + (PAGED16 ? (int64_t)tok_of(g, 0) * p.st : 0);
  const uint8_t* v_src = p.v + (int64_t)head * p.sh + v_chunk * 16 + (PAGED16 ? (int64_t)v_row * p.st : 0);
  const uint32_t k_dst = lane * S::CH;
  constexpr int NV = D == 256 ? 4 : 2;
  uint32_t v_dst[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v_dst[i] = S::kK + v_at<D>(v_row + S::VR * i, v_chunk) - S::VR * D * i;
  const int32_t* table = p.tables + (int64_t)q.s * p.table_stride;

  // raw table entry of this lane's token of step t, one step ahead of its use
  auto entry_of = [&](int32_t t) -> int32_t {
    const int32_t tok = c_lo + TS * t + (int32_t)(lane % TS);
    if (tok >= c_hi) return -2;
    const uint32_t i = c8_div_t(p, (uint32_t)tok);
    return i < p.table_width ? ldg_i32(table + i) : -1;
  };
  // Start the copies of step t.  Tokens without a page, and those past the range
  // (entry -2), are not copied: their slots hold what they held, their scales 0.
  auto issue = [&](int32_t t, int stage, int32_t entry) {
    const uint32_t at = slots + stage * S::kStage;
    const int32_t tok = c_lo + TS * t + (int32_t)(lane % TS);
    const bool ok = (uint32_t)entry < p.num_blocks;
    bad |= !ok && entry != -2;
    const uint32_t in_page = (uint32_t)tok - c8_div_t(p, (uint32_t)tok) * p.T;
    const int64_t off = ok ? (int64_t)entry * p.sb + (int64_t)in_page * p.st : -1;
    const uint32_t si = ok ? (uint32_t)entry : 0u;
    // (steps of 16 tokens: lanes 16 .. 31 copy the same words once more)
    cp_async<4>(at + 2 * S::kK + (lane % TS) * 4, p.k_scale + head + (uint64_t)si * p.H, ok);
    cp_async<4>(at + 2 * S::kK + 4 * TS + (lane % TS) * 4, p.v_scale + head + (uint64_t)si * p.H, ok);
#pragma unroll
    for (int t16 = 0; t16 < HT; ++t16) {
      if (PAGED16) {
        // a tile's tokens all lie in its first token's page (those past the length hold anything)
        const int64_t base = __shfl_sync(0xffffffffu, off, 16 * t16);
        if (base >= 0) {
          const uint8_t* ks = k_src + base;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < S::KC; ++c)
              cp_async<S::CH>(at + k_dst + ((t16 * 2 + h) * S::KC + c) * 32 * S::CH, ks + c * 4 * S::CH);
            ks += p.st2;
          }
          const uint8_t* vs = v_src + base;
#pragma unroll
          for (int i = 0; i < 16 / S::VR; ++i) {
            cp_async<16>(at + v_dst[i % NV] + (16 * t16 + i * S::VR) * D, vs);
            vs += p.stv;
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t b = __shfl_sync(0xffffffffu, off, 16 * t16 + tok_of(g, h));
          if (b >= 0) {
#pragma unroll
            for (int c = 0; c < S::KC; ++c)
              cp_async<S::CH>(at + k_dst + ((t16 * 2 + h) * S::KC + c) * 32 * S::CH, k_src + b + c * 4 * S::CH);
          }
        }
#pragma unroll
        for (int i = 0; i < 16 / S::VR; ++i) {
          const int64_t b = __shfl_sync(0xffffffffu, off, 16 * t16 + v_row + i * S::VR);
          if (b >= 0) cp_async<16>(at + v_dst[i % NV] + (16 * t16 + i * S::VR) * D, v_src + b);
        }
      }
    }
  };

  int32_t entry = entry_of((int32_t)warp);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    const int32_t t = (int32_t)warp + s * W;
    if (t < n_steps) {
      const int32_t e = entry;
      entry = entry_of(t + W);
      issue(t, s, e);
    }
    cp_commit();
  }

  // Q as FP16 fragments, rows scaled by a power of two into FP16's range (bf16; exact
  // down to 2^-31 of the row's largest, below that to 2^-39 of it): lane (g, qd) of k-step
  // 4 c + i holds dims 64 c + 16 qd + 4 i .. + 3 (D = 32: 8 qd + 4 i) of rows g, g + 8.
  uint32_t* s_q = reinterpret_cast<uint32_t*>(smem);
  float* s_row = reinterpret_cast<float*>(smem + S::kQ);  // per row: scale * log2(e) / row scaling
  if (W == 4 || tid < 128u) {
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
      uint32_t ks, l4;
      if (D >= 64) {
        ks = (dim >> 6) * 4 + ((dim >> 2) & 3u);
        l4 = (dim >> 4) & 3u;
      } else {
        ks = (dim >> 2) & 1u;
        l4 = (dim >> 3) & 3u;
      }
      // fragment registers: a0 (row g, k lo), a1 (row g + 8, k lo), a2 (row g, k hi), a3 (row g + 8, k hi)
      // (N8: b0 (k lo), b1 (k hi) of column g)
      if (!N8) s_q[(ks * 32 + (r & 7u) * 4 + l4) * 4 + ((dim >> 1) & 1u) * 2 + (r >> 3)] = w[k];
      else if (r < 8u) s_q[(ks * 32 + r * 4 + l4) * 2 + ((dim >> 1) & 1u)] = w[k];
    }
    if (part == 0) s_row[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - ex) << 23);
  }
  cta_sync();

  // this lane's rows of a score tile
  const uint32_t row_of[2] = {N8 ? 2 * qd : g, N8 ? 2 * qd + 1 : g + 8};
  const float rf[2] = {s_row[row_of[0]], s_row[row_of[1]]};
  // steps between these need no mask
  const int32_t full_hi = min(c_hi, first_pos < 0 ? 0 : p.causal ? min(q.len, first_pos + 1) : q.len);
  const int32_t full_lo = p.window ? (int32_t)max((int64_t)0, (int64_t)last_pos - p.window + 1) : 0;

  constexpr int NT = N8 ? D / 16 : D / 8;  // output tiles: 16 dims x 8 rows, or 16 rows x 8 dims
  constexpr int SH = N8 ? HT : 2 * HT;     // score tiles: 16 tokens x 8 rows, or 16 rows x 8 tokens
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
  // V scales are held relative to the largest that the row has seen
  float vref[2] = {1.17549435e-38f, 1.17549435e-38f}, vinv[2] = {0.0f, 0.0f};

  int stage = 0;
  for (int32_t t = (int32_t)warp; t < n_steps; t += W) {
    {
      const int32_t tn = t + (NS - 1) * W;
      const int sn = stage == 0 ? NS - 1 : stage - 1;
      __syncwarp();  // every lane is done with the stage that is refilled
      if (tn < n_steps) {
        const int32_t e = entry;
        entry = entry_of(tn + W);
        issue(tn, sn, e);
      }
      cp_commit();
      cp_wait<NS - 1>();
      __syncwarp();  // V and the scales were copied by other lanes
    }
    const uint8_t* sp = my_slots + stage * S::kStage;
    // V row lane & 15, chunk lane >> 4; chunk 2 c + (lane >> 4) of a row lies at this ^ (c << 5)
    const uint32_t sv = slots + stage * S::kStage + S::kK + v_at<D>(lane & 15u, lane >> 4);
    stage = stage == NS - 1 ? 0 : stage + 1;
    const int32_t tok0 = c_lo + TS * t;

    // scores: s[2 t16 + h][.] of columns 2 qd, + 1 of rows g, g + 8 (N8: s[t16][.] of tokens g, g + 8 as rows,
    // query rows 2 qd, + 1)
    float s[SH][4];
#pragma unroll
    for (int h = 0; h < SH; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.0f;
#pragma unroll
    for (int c = 0; c < S::KC; ++c) {
      uint32_t kw[2 * HT][4];
#pragma unroll
      for (int h = 0; h < 2 * HT; ++h) {
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
        if constexpr (N8) {
          const uint2 b = *reinterpret_cast<const uint2*>(s_q + ((c * (S::CH / 4) + i) * 32 + lane) * 2);
#pragma unroll
          for (int t16 = 0; t16 < HT; ++t16) {
            uint32_t a0, a1, a2, a3;
            c8_dec4(kw[2 * t16][i], a0, a2);
            c8_dec4(kw[2 * t16 + 1][i], a1, a3);
            mma16816(s[t16], a0, a1, a2, a3, b.x, b.y);
          }
        } else {
          const uint4 a = *reinterpret_cast<const uint4*>(s_q + ((c * (S::CH / 4) + i) * 32 + lane) * 4);
#pragma unroll
          for (int h = 0; h < 2 * HT; ++h) {
            uint32_t b0, b1;
            c8_dec4(kw[h][i], b0, b1);
            mma16816(s[h], a.x, a.y, a.z, a.w, b0, b1);
          }
        }
      }
    }
    // scales of tokens 16 t16 + 4 qd .. + 3; column (h, e) of a tile is token 2 h + e of these
    // (N8: of tokens tok_of(g, 0), tok_of(g, 1), in .x and .y)
    float vt[2] = {0.0f, 0.0f};
    bool hole = false;  // a token has the scale 0 of one that was not copied
    float4 vs[HT];
#pragma unroll
    for (int t16 = 0; t16 < HT; ++t16) {
      const float* kp = reinterpret_cast<const float*>(sp + 2 * S::kK) + 16 * t16;
      const float* vp = kp + TS;
      float4 k4;
      if (PAGED16) {
        k4 = make_float4(*kp, *kp, *kp, *kp);
        vs[t16] = make_float4(*vp, *vp, *vp, *vp);
        hole |= k4.x == 0.0f;
        vt[0] = fmaxf(vt[0], vs[t16].x);
      } else if (N8) {
        k4 = make_float4(kp[tok_of(g, 0)], kp[tok_of(g, 1)], 1.0f, 1.0f);
        vs[t16] = make_float4(vp[tok_of(g, 0)], vp[tok_of(g, 1)], 0.0f, 0.0f);
        hole |= k4.x == 0.0f || k4.y == 0.0f;
        vt[0] = fmaxf(vt[0], fmaxf(vs[t16].x, vs[t16].y));
      } else {
        k4 = *reinterpret_cast<const float4*>(kp + 4 * qd);
        vs[t16] = *reinterpret_cast<const float4*>(vp + 4 * qd);
        hole |= k4.x == 0.0f || k4.y == 0.0f || k4.z == 0.0f || k4.w == 0.0f;
        vt[0] = fmaxf(vt[0], fmaxf(fmaxf(vs[t16].x, vs[t16].y), fmaxf(vs[t16].z, vs[t16].w)));
      }
      if (N8) {
        s[t16][0] *= k4.x * rf[0]; s[t16][1] *= k4.x * rf[1];
        s[t16][2] *= k4.y * rf[0]; s[t16][3] *= k4.y * rf[1];
      } else {
        s[(2 * t16) % SH][0] *= k4.x * rf[0]; s[(2 * t16) % SH][1] *= k4.y * rf[0];
        s[(2 * t16) % SH][2] *= k4.x * rf[1]; s[(2 * t16) % SH][3] *= k4.y * rf[1];
        s[(2 * t16 + 1) % SH][0] *= k4.z * rf[0]; s[(2 * t16 + 1) % SH][1] *= k4.w * rf[0];
        s[(2 * t16 + 1) % SH][2] *= k4.z * rf[1]; s[(2 * t16 + 1) % SH][3] *= k4.w * rf[1];
      }
    }
    if (!PAGED16) hole = __any_sync(0xffffffffu, hole);
    vt[1] = vt[0];
    const bool masked = hole || tok0 + TS > full_hi || tok0 < full_lo;
    if (masked) {
      // visible keys of this lane's rows
      int32_t vis_hi[2], vis_lo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t r = row_of[h];
        const int32_t pos = q.start + (int32_t)((r0 + r) / p.G);
        vis_hi[h] = p.causal ? min(c_hi, pos + 1) : c_hi;  // c_hi: at most the length
        vis_lo[h] = p.window ? (int32_t)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
        if (r >= n_rows || pos < 0) vis_hi[h] = 0;
      }
#pragma unroll
      for (int h = 0; h < SH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t i = N8 ? 16 * h + tok_of(g, e >> 1) : 16 * (h >> 1) + 4 * qd + 2 * (h & 1) + (e & 1);
          const int32_t tok = tok0 + (int32_t)i;
          const int r = N8 ? e & 1 : e >> 1;
          if (tok >= vis_hi[r] || tok < vis_lo[r] ||
              (hole && *reinterpret_cast<const float*>(sp + 2 * S::kK + i * 4) == 0.0f))
            s[h][e] = kNegInf;
        }
      // the scale of a page that the row does not see must not push its weights out of FP16's range
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        vt[r] = 0.0f;
#pragma unroll
        for (int t16 = 0; t16 < HT; ++t16) {
          const float v4[4] = {vs[t16].x, vs[t16].y, vs[t16].z, vs[t16].w};
#pragma unroll
          for (int i = 0; i < (PAGED16 ? 1 : N8 ? 2 : 4); ++i) {
            const int32_t a = tok0 + 16 * t16 + (PAGED16 ? 0 : N8 ? (int32_t)tok_of(g, i) : (int32_t)(4 * qd) + i);
            if (a < vis_hi[r] && a + (PAGED16 ? 16 : 1) > vis_lo[r]) vt[r] = fmaxf(vt[r], v4[i]);
          }
        }
      }
    }
    // running maxima; the sums are rescaled only where a maximum grew by more than kLag
    bool grow = false;
    float mt[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = kNegInf;
#pragma unroll
      for (int h = 0; h < SH; ++h) x = fmaxf(x, N8 ? fmaxf(s[h][r], s[h][2 + r]) : fmaxf(s[h][2 * r], s[h][2 * r + 1]));
#pragma unroll
      for (int d = N8 ? 4 : 1; d < (N8 ? 32 : 4); d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
      mt[r] = x;
      grow |= x > m[r] + kLag;  // -inf + kLag = -inf: any finite score of a fresh row
    }
    if (!PAGED16) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int d = N8 ? 4 : 1; d < (N8 ? 32 : 4); d *= 2) vt[r] = fmaxf(vt[r], __shfl_xor_sync(0xffffffffu, vt[r], d));
      }
    }
    if (__any_sync(0xffffffffu, grow || vt[0] > vref[0] || vt[1] > vref[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float vn = fmaxf(vt[r], vref[r]);
        const float mn = mt[r] > m[r] + kLag ? mt[r] : m[r];
        const float f = m[r] == kNegInf ? 0.0f : ex2(m[r] - mn);
        const float fo = f * (vref[r] / vn);
        m[r] = mn;
        l[r] *= f;
        vref[r] = vn;
        vinv[r] = vt[r] > 0.0f || vinv[r] != 0.0f ? kLift / vn : 0.0f;  // 0 until the row has seen a scale
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][N8 ? r : 2 * r] *= fo;
          o[n][N8 ? 2 + r : 2 * r + 1] *= fo;
        }
      }
    }
    const float b0 = m[0] == kNegInf ? 0.0f : m[0], b1 = m[1] == kNegInf ? 0.0f : m[1];
    uint32_t pa[HT][4];
#pragma unroll
    for (int t16 = 0; t16 < HT; ++t16) {
      const float v4[4] = {vs[t16].x, PAGED16 ? vs[t16].x : vs[t16].y, PAGED16 ? vs[t16].x : vs[t16].z,
                           PAGED16 ? vs[t16].x : vs[t16].w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (N8) {  // tokens tok_of(g, h), rows 2 qd, + 1: transposed to row g, tokens 4 qd + 2 h, + 1
          const float z0 = s[t16][2 * h], z1 = s[t16][2 * h + 1];
          const float p0 = ex2(z0 - b0), p1 = ex2(z1 - b1);
          l[0] += p0;
          l[1] += p1;
          float x0 = p0 * ((h ? v4[1] : v4[0]) * vinv[0]), x1 = p1 * ((h ? v4[1] : v4[0]) * vinv[1]);
          if (masked) {
            x0 = z0 == kNegInf ? 0.0f : x0;
            x1 = z1 == kNegInf ? 0.0f : x1;
          }
          pa[t16][h] = transpose8(pack2<0>(x0, x1));
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float z0 = s[(2 * t16 + h) % SH][2 * r], z1 = s[(2 * t16 + h) % SH][2 * r + 1];
            const float p0 = ex2(z0 - (r ? b1 : b0)), p1 = ex2(z1 - (r ? b1 : b0));
            l[r] += p0 + p1;
            float x0 = p0 * (v4[2 * h] * vinv[r]), x1 = p1 * (v4[2 * h + 1] * vinv[r]);
            if (masked) {  // 0 whatever the scale of the page that holds a token the row does not see
              x0 = z0 == kNegInf ? 0.0f : x0;
              x1 = z1 == kNegInf ? 0.0f : x1;
            }
            pa[t16][2 * h + r] = pack2<0>(x0, x1);
          }
        }
      }
    }
    // V: words of four tokens (4 qd .. + 3) at dims 8 n + g
    uint32_t any_nan = 0;
#pragma unroll
    for (int t16 = 0; t16 < HT; ++t16)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t vw[4];
        ldsm_t16x2(vw, (sv ^ (c << 5)) + 16 * t16 * D);
        if (masked) {
          // a NaN that some row does not see must not reach it through 0 * NaN:
          // NaN codes become 0 here and are put back below where they are seen
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t nb = nan_bytes(vw[k]);
            any_nan |= nb;
            vw[k] &= ~((nb >> 7) * 0xffu);
          }
        }
        if constexpr (N8) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // dims 16 (2 c + k) + g, + 8
            uint32_t a0, a1, a2, a3;
            c8_dec4(vw[2 * k], a0, a2);
            c8_dec4(vw[2 * k + 1], a1, a3);
            mma16816(o[2 * c + k], a0, a1, a2, a3, pa[t16][0], pa[t16][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v0, v1;
            c8_dec4(vw[k], v0, v1);
            mma16816(o[(4 * c + k) % NT], pa[t16][0], pa[t16][1], pa[t16][2], pa[t16][3], v0, v1);
          }
        }
      }
    if (masked && __any_sync(0xffffffffu, any_nan != 0u)) {
      // rows x dims where a visible token's value is NaN: count them with the same product
#pragma unroll 1
      for (int t16 = 0; t16 < HT; ++t16) {
        uint32_t seen[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (N8) {
            const float z0 = t16 ? s[HT - 1][2 * h] : s[0][2 * h], z1 = t16 ? s[HT - 1][2 * h + 1] : s[0][2 * h + 1];
            seen[h] = transpose8((z0 == kNegInf ? 0u : 0x3c00u) | (z1 == kNegInf ? 0u : 0x3c000000u));
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float z0 = t16 ? s[(2 * (HT - 1) + h) % SH][2 * r] : s[h][2 * r];
              const float z1 = t16 ? s[(2 * (HT - 1) + h) % SH][2 * r + 1] : s[h][2 * r + 1];
              seen[2 * h + r] = (z0 == kNegInf ? 0u : 0x3c00u) | (z1 == kNegInf ? 0u : 0x3c000000u);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t vw[4], v[4][2];
          ldsm_t16x2(vw, (sv ^ (c << 5)) + 16 * t16 * D);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t nb = nan_bytes(vw[k]);  // 0x80 bytes -> 1.0 halves
            v[k][0] = (nb & 0x80u ? 0x3c00u : 0u) | (nb & 0x8000u ? 0x3c000000u : 0u);
            v[k][1] = (nb & 0x800000u ? 0x3c00u : 0u) | (nb & 0x80000000u ? 0x3c000000u : 0u);
          }
#pragma unroll
          for (int k = 0; k < (N8 ? 2 : 4); ++k) {
            float cnt[4] = {0.f, 0.f, 0.f, 0.f};
            if (N8) mma16816(cnt, v[(2 * k) & 3][0], v[(2 * k + 1) & 3][0], v[(2 * k) & 3][1], v[(2 * k + 1) & 3][1], seen[0], seen[1]);
            else mma16816(cnt, seen[0], seen[1], seen[2], seen[3], v[k][0], v[k][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cnt[e] > 0.0f) o[((N8 ? 2 : 4) * c + k) % NT][e] = __int_as_float(0x7fffffff);
          }
        }
      }
    }
  }
  cp_wait<0>();
  if (bad) c8_error(p, q.s, KV_CACHE8_BAD_PAGE);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int d = N8 ? 4 : 1; d < (N8 ? 32 : 4); d *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
  }

  // ---- join the warps: every row to the largest maximum among them
  float* s_m = s_row + 16;               // [row][warp] maxima
  float* s_l = s_m + 16 * W;             // [row][warp] sums, at the row's maximum
  float2* s_fin = reinterpret_cast<float2*>(smem);  // row: maximum and kJoin / sum, over Q once no warp needs that
  float* s_o = reinterpret_cast<float*>(smem + S::kQ + S::kSmall);  // [warp][16][D + 4], over the slots
  static_assert((16 + 32 * W) * 4 + 128 <= S::kSmall, "");
  constexpr int OS = D + 4;
  const bool holder = N8 ? g == 0u : qd == 0u;  // one lane for each row
  if (holder) {
    s_m[row_of[0] * W + warp] = m[0];
    s_m[row_of[1] * W + warp] = m[1];
  }
  cta_sync();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t row = row_of[r];
    float mx = kNegInf;
#pragma unroll
    for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[row * W + w]);
    const float f = m[r] == kNegInf ? 0.0f : ex2(m[r] - mx);
    const float fo = m[r] == kNegInf ? 0.0f : f * (vref[r] * (1.0f / (kLift * kJoin)));
    if (holder) s_l[row * W + warp] = l[r] * f;
    float* dst = s_o + (warp * 16 + row) * OS;
    if (N8) {  // tile n: dims 16 n + g, + 8 of the lane's rows
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        dst[16 * n + g] = o[n][r] * fo;
        dst[16 * n + 8 + g] = o[n][2 + r] * fo;
      }
    } else {  // column 2 qd + e of tile n is dim 8 n + 2 qd + e
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<float2*>(dst + 8 * n + 2 * qd) = make_float2(o[n][(2 * r) & 3] * fo, o[n][(2 * r + 1) & 3] * fo);
    }
  }
  cta_sync();
  const uint32_t job = u * p.H + head;
  float* base = p.partials + (uint64_t)job * p.splits * (kStepRows * (D + 2));
  float* mine = base + (uint64_t)split * (kStepRows * (D + 2));
  // a row's maximum and sum: the factor of its outputs, and lse
  auto finish_row = [&](uint32_t row, float mx, float ls) {
    s_fin[row] = make_float2(mx, ls == 0.0f ? 0.0f : kJoin / ls);
    if (p.lse && row < n_rows) {
      const uint32_t rr = r0 + row, tok = rr / p.G, hd = head * p.G + rr - tok * p.G;
      st4(p.lse + ((int64_t)q.row + tok) * p.HQ + hd,
          __float_as_uint(ls == 0.0f ? kNegInf : (mx + log2f(ls)) * 0.693147180559945309f));
    }
  };
  auto finish_out = [&](uint32_t r, uint32_t d4, float4 x) {
    const float inv = s_fin[r].y;
    const uint32_t rr = r0 + r, tok = rr / p.G, hd = head * p.G + rr - tok * p.G;
    st8(p.b + ((int64_t)q.row + tok) * p.b_row + (int64_t)hd * p.b_head + d4 * 4,
        inv == 0.0f ? make_uint2(0, 0)
                    : make_uint2(pack2<DT>(x.x * inv, x.y * inv), pack2<DT>(x.z * inv, x.w * inv)));
  };
  if (tid < n_rows) {
    float mx = kNegInf, ls = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      mx = fmaxf(mx, s_m[tid * W + w]);
      ls += s_l[tid * W + w];
    }
    if (n_split > 1u) st8(mine + kStepRows * D + 2 * tid, make_uint2(__float_as_uint(mx), __float_as_uint(ls)));
    else finish_row(tid, mx, ls);
  }
  if (n_split == 1u) cta_sync();
  for (uint32_t c4 = tid; c4 < n_rows * (D / 4); c4 += W * 32) {
    const uint32_t r = c4 / (D / 4), d4 = c4 % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(s_o + (w * 16 + r) * OS + d4 * 4);
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
    if (n_split > 1u)
      st16(mine + r * D + d4 * 4, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                                             __float_as_uint(x.w)));
    else finish_out(r, d4, x);
  }
  if (n_split == 1u) return;

  // ---- the last CTA of the row tile joins the ranges
  cta_sync();
  uint32_t* s_last = reinterpret_cast<uint32_t*>(s_m);
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
  cta_sync();
  if (*s_last != 1u) return;
  // maxima and sums of all ranges at once, then a range's factor in place of its maximum
  float2* s_ml = reinterpret_cast<float2*>(smem + S::kQ + S::kSmall);  // [range][16 rows], over the slots
  for (uint32_t k0 = tid; k0 < n_split * kStepRows; k0 += W * 32 * 4) {
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = k0 + i * W * 32;
      if (k < n_split * kStepRows && k % kStepRows < n_rows)
        y[i] = ld_join2(base + (uint64_t)(k / kStepRows) * (kStepRows * (D + 2)) + kStepRows * D + 2 * (k % kStepRows));
      else y[i] = make_float2(kNegInf, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i * W * 32 < n_split * kStepRows) s_ml[k0 + i * W * 32] = y[i];
  }
  cta_sync();
  if (W == 4 || tid < 128u) {
    const uint32_t row = tid >> 3, part = tid & 7u;
    float mx = kNegInf, ls = 0.0f;
    for (uint32_t k = part; k < n_split; k += 8) mx = fmaxf(mx, s_ml[k * kStepRows + row].x);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    for (uint32_t k = part; k < n_split; k += 8) {
      const float2 ml = s_ml[k * kStepRows + row];
      const float f = ml.x == kNegInf ? 0.0f : ex2(ml.x - mx);
      ls += ml.y * f;
      s_ml[k * kStepRows + row].x = f;
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    if (part == 0) finish_row(row, mx, ls);
  }
  cta_sync();
  // four dims a thread, all ranges in order, 16 loads in flight: of one place, or of 2 or 4 where there are few ranges
  auto join = [&](auto per_place) {
    constexpr uint32_t P = decltype(per_place)::value, C = 16 / P;
    for (uint32_t c0 = tid; c0 < n_rows * (D / 4); c0 += W * 32 * C) {
      float4 x[C];
#pragma unroll
      for (uint32_t i = 0; i < C; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t k0 = 0; k0 < n_split; k0 += P) {
        float4 y[C][P];
#pragma unroll
        for (uint32_t i = 0; i < C; ++i) {
          const uint32_t c4 = c0 + i * W * 32;
#pragma unroll
          for (uint32_t k = 0; k < P; ++k)
            if (k0 + k < n_split && c4 < n_rows * (D / 4))
              y[i][k] = ld_join4(base + (uint64_t)(k0 + k) * (kStepRows * (D + 2)) + c4 * 4);
        }
#pragma unroll
        for (uint32_t i = 0; i < C; ++i) {
          const uint32_t c4 = c0 + i * W * 32;
#pragma unroll
          for (uint32_t k = 0; k < P; ++k)
            if (k0 + k < n_split && c4 < n_rows * (D / 4)) {
              const float f = s_ml[(k0 + k) * kStepRows + c4 / (D / 4)].x;
              x[i].x += y[i][k].x * f;
              x[i].y += y[i][k].y * f;
              x[i].z += y[i][k].z * f;
              x[i].w += y[i][k].w * f;
            }
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < C; ++i) {
        const uint32_t c4 = c0 + i * W * 32;
        if (c4 < n_rows * (D / 4)) finish_out(c4 / (D / 4), c4 % (D / 4), x[i]);
      }
    }
  };
  if (n_split <= 4u) join(std::integral_constant<uint32_t, 4>{});
  else if (n_split <= 8u) join(std::integral_constant<uint32_t, 8>{});
  else join(std::integral_constant<uint32_t, 16>{});
}

template <int DT, int D, bool PAGED16, int W, bool N8>
int step_launch(const C8Params& p, void* stream) {
  constexpr int bytes = step_smem<D, W>();
  const auto kernel = c8_step_kernel<DT, D, PAGED16, W, N8>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, bytes, done)) return KV_ERR_CUDA;
  const uint64_t gx = (uint64_t)p.n_units * p.splits * p.H;
  if (gx > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<(unsigned)gx, W * 32, bytes, (cudaStream_t)stream>>>(p);
        return cudaGetLastError();
      },
      p);
}

template <int DT, int D, bool PAGED16>
int step_p(const C8Params& p, void* stream) {
  constexpr int BIG = D == 256 ? 8 : 12;
  if (p.step_warps > 4)
    return p.rows8 ? step_launch<DT, D, PAGED16, BIG, true>(p, stream) : step_launch<DT, D, PAGED16, BIG, false>(p, stream);
  return p.rows8 ? step_launch<DT, D, PAGED16, 4, true>(p, stream) : step_launch<DT, D, PAGED16, 4, false>(p, stream);
}

template <int DT, int D>
int step_d(const C8Params& p, void* stream) {
  return p.T % 16 == 0 ? step_p<DT, D, true>(p, stream) : step_p<DT, D, false>(p, stream);
}

}  // namespace

int launch_c8_step(const C8Params& p, void* stream) { KVC_C8_DISPATCH(step_d, p, stream); }

}  // namespace kvc
