// cache16_step.cu -- attention of few query rows over the 16-bit pages: single tokens,
// drafted tokens, short chunks.
//
//   z_rj = scale (q_r . k_j),  out_r = sum_j 2^(z_rj - m_r) v_j / l_r
//
// Bound by reading K and V once (4 D bytes a token and KV head).  A row tile is the G query
// heads of a KV head times the new tokens, 8 or 16 rows at a time; a job is a row tile of a
// sequence and a KV head, its keys in steps of 16 or 32 tokens.  The lengths are on the
// device, so the split is made there: every CTA adds up the steps of all sequences, takes
// an equal share of the row of all jobs' steps (the last of one job, some whole ones, the
// first of another; of few jobs an even part of one), and finds where that begins.  No CTA is
// idle while another has two shares, whatever the lengths, and the host need not know them.
//
// In a CTA the warps take a job's steps in turn, each on its own: asynchronous copies into
// slots of its own, steps ahead, without barriers; they join at the job's end.  A job that
// lies in several shares leaves a partial result in each, and the CTA that finishes last
// joins them in the order of the keys, so the result does not depend on timing.
//
// Both products have the tokens (scores) and the dims (outputs) as their 16 rows and 8 query
// rows as their columns: K's tile is the operand as it lies, V's as ldmatrix transposes it,
// and the weights pass through a transposition in registers.  A weight is split into 16-bit
// terms, two of FP16 or three of BF16, with a product for each, so that it keeps what FP32
// arithmetic gave it (two BF16 terms were 0 to 3 % faster with 8 query rows, 3 to 7 with 16).
//
// Measured on a GB300, 8 heads of 128: 64 sequences of 100 to 8192 tokens 99 to 103 us (5.7 TB/s; a
// plain copy 6.7), one of 131072 with 4 heads 57 us (4.7; the walk 36 to 41 us of it, 4 to start, 8 to join).
#include <algorithm>

#include "cache8_common.cuh"

namespace kvc {

#ifdef KVC_BOUNDS_CHECK
inline void dbg_ranges(DbgRanges& r, const C16Params& p) {
  const uint64_t last = (uint64_t)p.sb * (p.num_blocks - 1u) + (uint64_t)p.st * (p.T - 1u) +
                        (uint64_t)p.sh * (p.H - 1u) + 2u * p.D;
  dbg_add(r, p.k, dbg_slot_bytes(last));
  dbg_add(r, p.v, dbg_slot_bytes(last));
  dbg_add(r, p.tables, 4ull * ((uint64_t)p.table_stride * (p.n_seqs - 1u) + p.table_width));
  dbg_add(r, p.lens, 4ull * p.n_seqs);
  if (p.cu) dbg_add(r, p.cu, 4ull * (p.n_seqs + 1u));
  if (p.errors) dbg_add(r, p.errors, 4ull * p.n_seqs);
  dbg_rows(r, p.a, p.a_row, p.a_head, p, p.HQ);
  dbg_rows(r, p.b, p.b_row, p.b_head, p, p.HQ);
  if (p.lse) dbg_add(r, p.lse, 4ull * p.n_new * p.HQ);
  dbg_add(r, p.tickets, 4ull * 3u * kC16Ctas);
  dbg_add(r, p.partials, 4ull * kC16Ctas * 2u * kStepRows * (p.D + 2u));
}
#endif

namespace {

constexpr float kNegInf = -INFINITY;
// m may lag the true maximum by kLag (fewer rescalings of the sums).
constexpr float kLag = 4.0f;
// A weight 2^(z - m) enters V's product times this.  FP16: the largest are 2^11 .. 2^15, so that 2^-25, half of the smallest
// FP16, is 2^-36 of the largest.  BF16: 2^-24 .. 2^-20, so that sums over 2^20 keys of V next to 2^128 stay in FP32's range.
// (A factor is exact; added to the exponent it would cost the score bits: 24 holds 2^-19 of it.)
template <int DT>
constexpr float kHold = DT == 0 ? 0x1p11f : 0x1p-24f;
// It enters as this many 16-bit terms, each the nearest to what the earlier ones leave: 24 bits in three BF16 terms, 22 in two of
// FP16, as fine as ex2.approx (2^-22).  One BF16 term would be as coarse as the output's rounding; two (2^-18) showed in outputs
// whose values nearly cancel.
template <int DT>
constexpr int kTerms = DT == 0 ? 2 : 3;

// A barrier of the CTA that counts threads, whether or not their warp is converged.
__device__ __forceinline__ void cta_sync() { asm volatile("barrier.sync 0;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == 0)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t smem) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t smem) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem)
               : "memory");
}
// Transpose of an 8 x 8 tile of 16-bit values, two values of a row to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Copy 16 bytes to a shared slot; zeros when !ok.
__device__ __forceinline__ void cp16z(uint32_t smem, const void* src, bool ok) {
#ifdef KVC_BOUNDS_CHECK
  if (ok && !dbg_ok(src, 16)) ok = false;
#endif
  const uint32_t n = ok ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp16(uint32_t smem, const void* src) {
  KVC_GUARD(src, 16, return);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}

// loads of what other CTAs of this launch have stored (L2)
__device__ __forceinline__ float4 ld_join4(const float* ptr) {
  KVC_GUARD(ptr, 16, return make_float4(0.f, 0.f, 0.f, 0.f));
  return __ldcg(reinterpret_cast<const float4*>(ptr));
}
__device__ __forceinline__ float2 ld_join2(const float* ptr) {
  KVC_GUARD(ptr, 8, return make_float2(0.f, 0.f));
  return __ldcg(reinterpret_cast<const float2*>(ptr));
}

// Warps of a CTA, two of which share an SM: the start of a job and the joins of one hide behind
// the other.  CTAs of 8 warps, one an SM: 64 uneven sequences 103 us against 101, 48 with one KV head 27 against 25.
constexpr int kWarps = 4, kThreads16 = 32 * kWarps;
// What a job costs its CTA besides its steps (its first copies, the joins), in steps; equal shares count it (even parts do not).
// Shares that did not count it left CTAs with many short jobs three times as long as the others.  200 sequences of 10 to
// 6000 tokens, 4 KV heads, with 4, 8, 12, 16, 20 and 24: head_dim 32 49, 41, 39, 41, 42, 44 us; 64 57, 47, 48, 50, 52, 55;
// 128 89, 79, 79, 79, 80, 81; 256 154, 146, 148, 149, 151, 152.  So one number does for all; with 64 sequences of 100 to 8192
// tokens or 256 of 200 to 1500 it makes 4 % at most from 8 to 16.
constexpr uint32_t kStart = 12;
constexpr uint32_t kLeast = kStart + 4;  // of a share
// Partials that are joined at once; more are joined in groups.  One sequence of 131072 with 2 heads, 152 partials, at once and
// in groups: head_dim 32 27 and 19 us, 64 33 and 25, 128 51 and 37, 256 96 and 63; with 4 heads, 76 partials: 31 and 28, 38 and
// 35, 62 and 57, 116 and 102.  6, 12 or 24 makes no difference for any head_dim.
constexpr uint32_t kFlat = 12;

template <int D>
struct Shape16 {
  static constexpr int TS = D >= 128 ? 16 : 32;    // tokens of a step
  static constexpr int HT = TS / 16;
  static constexpr int C = D / 8;                  // 16-byte chunks of a row
  static constexpr int RPI = 32 / C;               // rows that a warp's copy instruction covers
  // Rows lie an odd number of chunks apart: 8 rows' chunks of one column are in 8 different bank groups.
  static constexpr int kPitch = D * 2 + 16;
  static constexpr int kSlot = TS * kPitch;        // K's rows of a step, or V's
  // Steps that copies are ahead; a warp's slots hold these, K and V one after the other, and the K or V in use.
  static constexpr int kAhead = D == 256 ? 1 : D == 32 ? 3 : 2;
  static constexpr int NS = 2 * kAhead + 1;
  static constexpr int kQ = 16 * kPitch;
  static constexpr int kSmall = 1024;
  static constexpr int kOut = D + 4;               // floats of a row in the join of the warps
  static constexpr int kSmem = kQ + kSmall + kWarps * NS * kSlot;
};
// n / G for n < 2^31
__device__ __forceinline__ uint32_t div_g(const C16Params& p, uint32_t n) {
  return (__umulhi(p.g_magic, n) + n) >> p.g_shift;
}

// A sequence of the batch, and how many steps its jobs have.
struct Seq16 {
  C8Seq q;
  int32_t lo, hi;   // keys that some row sees; lo at a 16-token tile where pages are whole tiles
  bool past;        // tokens lie past the table's row
  uint32_t steps;   // of a job
  uint32_t len;     // of a job in the row of all jobs: its parts, or its steps and kStart
  uint32_t jobs;
};
// a / b.  Small ones (as they mostly are) by an FP32 quotient, which is off by one at most, and its remainder: the long
// divisions, several in a row at each start of a CTA, took it most of a microsecond.
__device__ __forceinline__ uint64_t div64(uint64_t a, uint64_t b) {
  if (((a | b) >> 22) == 0) {
    const int32_t x = (int32_t)a, y = (int32_t)b;
    int32_t q = (int32_t)__fdividef((float)x, (float)y);
    const int32_t r = x - q * y;
    if (r < 0) --q;
    if (r >= y) ++q;
    return (uint64_t)q;
  }
  return a / b;
}

// most: the most steps of a part where jobs are split evenly, 0 where shares go over the jobs.
template <int D, bool PAGED16, int TR>
__device__ __forceinline__ Seq16 seq16(const C16Params& p, uint32_t s, uint32_t most) {
  Seq16 x;
  x.q.s = s;
  x.q.unit = 0;
  const int32_t len = ldg_i32(p.lens + s);
  if (p.cu) c8_fill(p, x.q, ldg_i32(p.cu + s), ldg_i32(p.cu + s + 1u), len);
  else c8_fill(p, x.q, (int32_t)s, (int32_t)s + 1, len);
  const uint64_t reach = (uint64_t)p.table_width * p.T;
  x.past = (uint64_t)x.q.len > reach;
  x.hi = x.past ? (int32_t)reach : x.q.len;
  x.lo = p.window && x.q.start >= 0 ? max(0, x.q.start - (int32_t)min(p.window, 0x7fffffffu) + 1) : 0;
  if (PAGED16) x.lo &= ~15;
  constexpr int TS = Shape16<D>::TS;
  x.steps = x.hi > x.lo ? ((uint32_t)(x.hi - x.lo) + TS - 1u) / TS : 1u;  // (rows that see nothing are a step)
  x.jobs = ((uint32_t)x.q.n_new * p.G + TR - 1u) / TR * p.H;
  x.len = most ? (uint32_t)div64(x.steps + most - 1u, most) : x.steps + kStart;
  return x;
}

// PAGED16: pages are whole 16-token tiles, so a tile lies in one page; otherwise every token's page is
// looked up by itself.  NT: 8-row column blocks of a row tile.
template <int DT, int D, bool PAGED16, int NT>
__global__ void __launch_bounds__(kThreads16) c16_step_kernel(const __grid_constant__ C16Params p) {
  using S = Shape16<D>;
  constexpr int NS = S::NS, kAhead = S::kAhead, TS = S::TS, HT = S::HT, TR = 8 * NT, KS = D / 16;
  constexpr uint32_t kFull = TS == 32 ? 0xffffffffu : 0xffffu;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  constexpr uint32_t threads = kThreads16, W = kWarps;
  const uint32_t g = lane >> 2, qd = lane & 3u;
  const uint32_t sm_q = (uint32_t)__cvta_generic_to_shared(smem);
  float* s_m = reinterpret_cast<float*>(smem + S::kQ);             // [row][warp] maxima
  float* s_l = s_m + 16 * kWarps;                                       // [row][warp] sums, at the row's maximum
  float2* s_fin = reinterpret_cast<float2*>(s_l + 16 * kWarps);         // row: maximum, 1 / sum
  unsigned long long* s_tot = reinterpret_cast<unsigned long long*>(s_fin + 16);  // warps' steps, then where to begin
  uint32_t* s_last = reinterpret_cast<uint32_t*>(s_tot + 2 * kWarps);
  static_assert(16 * kWarps * 8 + 16 * 8 + 2 * kWarps * 8 + 4 <= S::kSmall, "");
  uint8_t* slots = smem + S::kQ + S::kSmall;
  float* s_o = reinterpret_cast<float*>(slots);                    // [warp][TR][kOut], over the slots
  float2* s_ml = reinterpret_cast<float2*>(slots);                 // [partial][TR], over the slots
  static_assert((int)kC16Ctas * 16 * 8 <= kWarps * S::NS * S::kSlot && 16 * S::kOut * 4 <= S::NS * S::kSlot, "");
  const uint32_t my_slots = sm_q + S::kQ + S::kSmall + warp * (NS * S::kSlot);

  // ---- this CTA's share
  // All jobs one after the other.  Few jobs: each is split into even parts of `most` steps at most, a part to a CTA.  Else
  // equal shares of the row go over the jobs' ends, each job counted as its steps and kStart.
  uint64_t at, end, share;
  uint32_t s, most = 0;
  uint64_t base;  // where sequence s begins
  {
    const uint32_t per = (p.n_seqs + threads - 1u) / threads, i0 = min(tid * per, p.n_seqs), i1 = min(i0 + per, p.n_seqs);
    if (p.even) {
      unsigned long long steps = 0, jobs = 0;
      for (uint32_t i = i0; i < i1; ++i) {
        const Seq16 y = seq16<D, PAGED16, TR>(p, i, 0u);
        steps += (unsigned long long)y.steps * y.jobs;
        jobs += y.jobs;
      }
#pragma unroll
      for (int d = 16; d; d /= 2) {
        steps += __shfl_xor_sync(0xffffffffu, steps, d);
        jobs += __shfl_xor_sync(0xffffffffu, jobs, d);
      }
      if (lane == 0u) s_tot[warp] = steps, s_tot[kWarps + warp] = jobs;
      cta_sync();
      steps = jobs = 0;
#pragma unroll
      for (uint32_t w = 0; w < W; ++w) steps += s_tot[w], jobs += s_tot[kWarps + w];
      cta_sync();
      // the parts of all jobs number steps / most, and one more at most for each job
      if (2u * jobs <= gridDim.x)
        most = max((uint32_t)div64(steps + gridDim.x - jobs - 1u, gridDim.x - jobs), kLeast - kStart);
    }
    unsigned long long mine = 0;
    for (uint32_t i = i0; i < i1; ++i) {
      const Seq16 y = seq16<D, PAGED16, TR>(p, i, most);
      mine += (unsigned long long)y.len * y.jobs;
    }
    unsigned long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= (uint32_t)d) inc += y;
    }
    if (lane == 31u) s_tot[warp] = inc;
    cta_sync();
    unsigned long long before = 0, total = 0;
#pragma unroll
    for (uint32_t w = 0; w < W; ++w) {
      before += w < warp ? s_tot[w] : 0ull;
      total += s_tot[w];
    }
    share = most ? 1ull : max((unsigned long long)div64(total + gridDim.x - 1u, gridDim.x), (unsigned long long)kLeast);
    at = (uint64_t)blockIdx.x * share;
    if (at >= total) return;
    end = min(at + share, (uint64_t)total);
    unsigned long long pre = before + inc - mine;
    if (pre <= at && at < pre + mine) {
      uint32_t i = i0;
      for (;; ++i) {
        const Seq16 y = seq16<D, PAGED16, TR>(p, i, most);
        const unsigned long long n = (unsigned long long)y.len * y.jobs;
        if (at < pre + n) break;
        pre += n;
      }
      s_tot[kWarps] = pre;
      s_tot[kWarps + 1] = i;
    }
    cta_sync();
    base = s_tot[kWarps];
    s = (uint32_t)s_tot[kWarps + 1];
  }

  // this lane's place in the copies and the fragments of a tile
  const uint32_t c_row = lane / S::C, c_chunk = lane % S::C;
  const uint32_t c_dst = my_slots + c_row * S::kPitch + c_chunk * 16;
  const uint32_t k_at = my_slots + (lane & 15u) * S::kPitch + ((lane >> 4) << 4);
  const uint32_t v_at = my_slots + ((lane & 7u) + ((lane >> 4) << 3)) * S::kPitch + (((lane >> 3) & 1u) << 4);

  Seq16 x = seq16<D, PAGED16, TR>(p, s, most);
  const uint64_t begin = at;
  const uint64_t job = div64(at - base, x.len);
  uint64_t job0 = base + job * x.len;  // where the job begins
  uint32_t tile = job < p.H ? 0u : (uint32_t)div64(job, p.H), head = (uint32_t)(job - (uint64_t)tile * p.H);
  for (bool first = true; at < end; first = false) {
    if (!first) {  // the next job: at is where it begins
      job0 = at;
      if (++head == p.H) head = 0, ++tile;
      while (at >= base + (uint64_t)x.len * x.jobs) {  // the next sequence (one without new tokens has no jobs)
        base += (uint64_t)x.len * x.jobs;
        x = seq16<D, PAGED16, TR>(p, ++s, most);
        head = tile = 0;
      }
    }
    const uint32_t from = (uint32_t)(at - job0), to = (uint32_t)min((uint64_t)x.len, end - job0);
    at = job0 + to;
    // the steps of this part, the CTA of the job's first part, and how many there are
    uint32_t step0, n_steps, cta0 = blockIdx.x, n_parts = 1u;
    if (most) {
      const uint32_t size = x.len == 1u ? x.steps : (uint32_t)div64(x.steps + x.len - 1u, x.len);
      step0 = from * size;
      if (step0 >= x.steps) break;  // (even parts may be one fewer)
      n_steps = min(size, x.steps - step0);
      cta0 = blockIdx.x - from;
      n_parts = x.len == 1u ? 1u : (uint32_t)div64(x.steps + size - 1u, size);
    } else {
      // the steps of [from, to), kStart of which are none; a job's parts are with the CTA whose share has its first step and
      // those up to its last
      step0 = max(from, kStart) - kStart;
      n_steps = max(to, kStart) - kStart - step0;
      if (n_steps == 0u) continue;  // the CTA after this one begins the job
      if (job0 + kStart < begin) cta0 = (uint32_t)div64(job0 + kStart, share);
      if (cta0 != blockIdx.x || job0 + x.len > end) n_parts = (uint32_t)div64(job0 + x.len - 1u, share) - cta0 + 1u;
    }

    const uint32_t r0 = tile * TR, n_rows = min((uint32_t)TR, (uint32_t)x.q.n_new * p.G - r0);
    const int32_t first_pos = x.q.start + (int32_t)div_g(p, r0), last_pos = x.q.start + (int32_t)div_g(p, r0 + n_rows - 1u);
    // keys that some row of the tile sees, and the steps that hold them
    const int32_t t_hi = last_pos < 0 ? 0 : p.causal ? min(x.hi, last_pos + 1) : x.hi;
    const int32_t t_lo = p.window && first_pos >= 0 ? max(0, first_pos - (int32_t)min(p.window, 0x7fffffffu) + 1) : 0;
    const int32_t x_lo = max((int32_t)step0, t_lo > x.lo ? (t_lo - x.lo) / TS : 0);
    const int32_t x_hi = min((int32_t)(step0 + n_steps), t_hi > x.lo ? (t_hi - x.lo + TS - 1) / TS : 0);
    const bool several = first_pos != last_pos;  // rows of several positions: they do not all see the same keys
    const int32_t* table = p.tables + (int64_t)x.q.s * p.table_stride;
    bool bad = x.past && tid == 0u;

    // raw table entry of this lane's token of step t; -2 past the keys
    auto entry_of = [&](int32_t t) -> int32_t {
      const int32_t tok = x.lo + TS * t + (int32_t)(lane % TS);
      return t < x_hi && tok < t_hi ? ldg_i32(table + c8_div_t(p, (uint32_t)tok)) : -2;
    };
    const uint8_t* k_src = p.k + (int64_t)head * p.sh + c_chunk * 16 + (PAGED16 ? (int64_t)c_row * p.st : 0);
    const uint8_t* v_src = p.v + (int64_t)head * p.sh + c_chunk * 16 + (PAGED16 ? (int64_t)c_row * p.st : 0);
    // Where the lane's token of step t lies; returns the tokens that are there, a bit each.
    auto place = [&](int32_t t, int32_t entry, int64_t& off) -> uint32_t {
      const int32_t tok = x.lo + TS * t + (int32_t)(lane % TS);
      const bool in = tok >= t_lo && tok < t_hi, page = (uint32_t)entry < p.num_blocks;
      bad |= in && !page;
      const uint32_t in_page = (uint32_t)tok - c8_div_t(p, (uint32_t)tok) * p.T;
      off = (int64_t)entry * p.sb + (int64_t)in_page * p.st;
      return __ballot_sync(0xffffffffu, in && page) & kFull;
    };
    // Start the copies of a step's K or V.  Tokens that no row sees, and those without a page, become zeros.
    auto issue = [&](const uint8_t* src, int slot, uint32_t there, int64_t off) {
      const uint32_t dst = c_dst + slot * S::kSlot;
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const uint32_t bits = HT == 1 ? there : (there >> (16 * h)) & 0xffffu;
        const int64_t tile_off = __shfl_sync(0xffffffffu, off, 16 * h);
        if (PAGED16 && bits == 0xffffu) {
          const uint8_t* at = src + tile_off;
#pragma unroll
          for (int i = 0; i < 16 / S::RPI; ++i) {
            cp16(dst + (16 * h + i * S::RPI) * S::kPitch, at);
            at += S::RPI * p.st;
          }
        } else {
#pragma unroll 4
          for (int i = 0; i < 16 / S::RPI; ++i) {
            const uint32_t row = c_row + S::RPI * i;
            const bool ok = (bits >> row) & 1u;
            const int64_t o = PAGED16 ? tile_off + (int64_t)(S::RPI * i) * p.st : __shfl_sync(0xffffffffu, off, 16 * h + row);
            cp16z(dst + (16 * h + i * S::RPI) * S::kPitch, ok ? src + o : p.k, ok);
          }
        }
      }
    };

    cta_sync();  // the job before is done with shared memory
    uint32_t there[kAhead + 1];  // of the steps in flight, the oldest first
    int32_t entry;
    {
      int32_t e[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) e[i] = entry_of(x_lo + (int32_t)(warp + i * W));
      entry = entry_of(x_lo + (int32_t)(warp + kAhead * W));
      for (uint32_t i = tid; i < TR * (D / 8); i += threads) {
        const uint32_t r = i / (D / 8), c = i % (D / 8), rr = r0 + min(r, n_rows - 1u), tok = div_g(p, rr);
        const uint16_t* src = p.a + ((int64_t)x.q.row + tok) * p.a_row + (int64_t)(head * p.G + rr - tok * p.G) * p.a_head + c * 8;
        cp16z(sm_q + r * S::kPitch + c * 16, src, r < n_rows);
      }
      cp_commit();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int32_t t = x_lo + (int32_t)(warp + i * W);
        there[i] = 0u;
        if (t < x_hi) {
          int64_t off;
          there[i] = place(t, e[i], off);
          issue(k_src, 2 * i, there[i], off);
          cp_commit();
          issue(v_src, 2 * i + 1, there[i], off);
        } else {
          cp_commit();
        }
        cp_commit();
      }
    }
    cp_wait<2 * kAhead>();  // the queries
    cta_sync();
    // the queries' fragments: in registers, or (where the sums leave no room) read again at each step
    constexpr bool kHeld = D < 256;
    const uint32_t q_at = sm_q + (lane & 7u) * S::kPitch + ((lane >> 3) << 4);
    uint32_t qf[kHeld ? NT : 1][kHeld ? KS / 2 : 1][4];
    if constexpr (kHeld) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) ldsm4(qf[n][k], q_at + n * 8 * S::kPitch + k * 64);
    }
    // steps between these need no mask by rows
    const int32_t full_hi = !several ? 0x7fffffff : first_pos < 0 ? 0 : p.causal ? first_pos + 1 : 0x7fffffff;
    const int32_t full_lo = several && p.window ? (int32_t)max((int64_t)0, (int64_t)last_pos - p.window + 1) : 0;

    float o[KS][NT][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    float m[NT][2], l[NT][2];  // of rows 8 n + 2 qd, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kNegInf, l[n][0] = l[n][1] = 0.0f;

    int slot = 0;  // of K; V's is the next one
    for (int32_t t = x_lo + (int32_t)warp; t < x_hi; t += (int32_t)W) {
      const int32_t tn = t + (int32_t)(kAhead * W);
      int64_t off = 0;
      __syncwarp();  // every lane is done with the slot that is refilled
      there[kAhead] = 0u;
      if (tn < x_hi) {
        there[kAhead] = place(tn, entry, off);
        entry = entry_of(tn + (int32_t)W);
        issue(k_src, slot == 0 ? NS - 1 : slot - 1, there[kAhead], off);
      }
      cp_commit();
      cp_wait<2 * kAhead>();
      __syncwarp();  // the other lanes' copies
      const uint32_t bits = there[0], more = there[kAhead];
      const uint32_t sk = k_at + slot * S::kSlot, sv = v_at + (slot == NS - 1 ? 0 : slot + 1) * S::kSlot;
      const int k_slot = slot;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) there[i] = there[i + 1];
      slot = slot >= NS - 2 ? slot + 2 - NS : slot + 2;
      const int32_t tok0 = x.lo + TS * t;

      // scores of tokens 16 h + g, + 8 and rows 8 n + 2 qd, + 1
      constexpr int Z = HT * NT == 1 ? 2 : 1;  // chains of products that do not wait for each other
      float z[HT][NT][4];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float y[Z][NT][4];
#pragma unroll
        for (int c = 0; c < Z; ++c)
#pragma unroll
          for (int n = 0; n < NT; ++n) y[c][n][0] = y[c][n][1] = y[c][n][2] = y[c][n][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          uint32_t a[4], b[4], w[NT][4];
          ldsm4(a, sk + h * 16 * S::kPitch + k * 64);
          ldsm4(b, sk + h * 16 * S::kPitch + k * 64 + 32);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (kHeld) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[n][i] = qf[n][k][i];
            } else {
              ldsm4(w[n], q_at + n * 8 * S::kPitch + k * 64);
            }
            mma16816<DT>(y[0][n], a, w[n][0], w[n][1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<DT>(y[Z - 1][n], b, w[n][2], w[n][3]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[h][n][e] = (Z == 2 ? y[0][n][e] + y[Z - 1][n][e] : y[0][n][e]) * p.scale_log2;
      }
      __syncwarp();  // K's slot is read
      if (tn < x_hi) issue(v_src, k_slot, more, off);
      cp_commit();
      const bool by_row = tok0 + TS > full_hi || tok0 < full_lo;
      // which of the step's tokens row 8 n + 2 qd + r sees, a bit each
      auto sees = [&](int n, int r) -> uint32_t {
        if (!by_row) return bits;
        const int32_t pos = x.q.start + (int32_t)div_g(p, r0 + 8u * n + 2u * qd + r);
        // the first token that it sees no more, and the first that it sees, from the step's first on
        const int32_t hi = pos < 0 ? 0 : p.causal ? min(max(pos + 1 - tok0, 0), TS) : TS;
        const int32_t lo = p.window ? (int32_t)min(max((int64_t)pos - p.window + 1 - tok0, (int64_t)0), (int64_t)TS) : 0;
        return bits & (uint32_t)((1ull << hi) - 1ull) & ~(uint32_t)((1ull << lo) - 1ull);
      };
      if (by_row || bits != kFull) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t seen = sees(n, r) >> g;
#pragma unroll
            for (int h = 0; h < HT; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!((seen >> (16 * h + 8 * e)) & 1u)) z[h][n][2 * e + r] = kNegInf;
          }
      }
      // running maxima; the sums are rescaled only where a maximum grew by more than kLag
      bool grow = false;
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) grow |= z[h][n][e] > m[n][e & 1] + kLag;  // -inf + kLag = -inf: any finite score
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = kNegInf;
#pragma unroll
            for (int h = 0; h < HT; ++h) mx = fmaxf(mx, fmaxf(z[h][n][r], z[h][n][2 + r]));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(mx, m[n][r]);
            const float f = m[n][r] == kNegInf ? 0.0f : ex2(m[n][r] - mn);
            m[n][r] = mn;
            l[n][r] *= f;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[i][n][r] *= f;
              o[i][n][2 + r] *= f;
            }
          }
      }
      // weights, split in terms and transposed: row g, tokens 2 qd, + 1 (+ 8 e)
      uint32_t w[kTerms<DT>][HT][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float b0 = m[n][0] == kNegInf ? 0.0f : m[n][0], b1 = m[n][1] == kNegInf ? 0.0f : m[n][1];
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float p0 = ex2(z[h][n][2 * e] - b0), p1 = ex2(z[h][n][2 * e + 1] - b1);
            l[n][0] += p0;
            l[n][1] += p1;
            p0 *= kHold<DT>, p1 *= kHold<DT>;
#pragma unroll
            for (int i = 0; i < kTerms<DT>; ++i) {
              const uint32_t x = pack2<DT>(p0, p1);
              w[i][h][n][e] = transpose8(x);
              p0 -= lo_f32<DT>(x), p1 -= hi_f32<DT>(x);
            }
          }
      }
      cp_wait<2 * kAhead>();
      __syncwarp();  // the other lanes' copies of V
      // V: dims 16 i + g, + 8 of tokens 2 qd, + 1, + 8, + 9
      constexpr uint32_t E = DT == 0 ? 0x7c00u : 0x7f80u, one = DT == 0 ? 0x3c00u : 0x3f80u;
      bool odd = false;
      if (by_row) {
        // an infinity or a NaN that some row does not see must not reach it through 0 times it
#pragma unroll 1
        for (int i = 0; i < HT * KS; ++i) {
          uint32_t a[4];
          ldsm4_t(a, sv + (i / KS) * 16 * S::kPitch + (i % KS) * 32);
#pragma unroll
          for (int k = 0; k < 4; ++k) odd |= (a[k] & E) == E || (a[k] & (E << 16)) == (E << 16);
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      if (!odd) {
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldsm4_t(a, sv + h * 16 * S::kPitch + i * 32);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int t = 0; t < kTerms<DT>; ++t) mma16816<DT>(o[i][n], a, w[t][h][n][0], w[t][h][n][1]);
          }
      } else {
        // Such values become 0, and NaN is put where they are seen: rows x dims with one, counted by the same product.  (Seen by
        // the mask: a score of -inf weighs 0, and 0 times such a value is no number.)
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          uint32_t seen[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t s0 = sees(n, 0) >> (g + 16u * h), s1 = sees(n, 1) >> (g + 16u * h);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              seen[n][e] = transpose8((((s0 >> (8 * e)) & 1u) ? one : 0u) | (((s1 >> (8 * e)) & 1u) ? one << 16 : 0u));
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t a[4], b[4];
            ldsm4_t(a, sv + h * 16 * S::kPitch + i * 32);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool lo = (a[k] & E) == E, hi = (a[k] & (E << 16)) == (E << 16);
              b[k] = (lo ? one : 0u) | (hi ? one << 16 : 0u);
              a[k] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int t = 0; t < kTerms<DT>; ++t) mma16816<DT>(o[i][n], a, w[t][h][n][0], w[t][h][n][1]);
              float cnt[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<DT>(cnt, b, seen[n][0], seen[n][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (cnt[e] > 0.0f) o[i][n][e] = __int_as_float(0x7fffffff);
            }
          }
        }
      }
    }
    cp_wait<0>();
    if (bad) c8_error(p, x.q.s, KV_CACHE8_BAD_PAGE);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], d);

    // ---- join the warps: every row to the largest maximum among them
    if (g == 0u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s_m[(8 * n + 2 * qd) * W + warp] = m[n][0];
        s_m[(8 * n + 2 * qd + 1) * W + warp] = m[n][1];
      }
    }
    cta_sync();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t row = 8u * n + 2u * qd + r;
        float mx = kNegInf;
        for (uint32_t w = 0; w < W; ++w) mx = fmaxf(mx, s_m[row * W + w]);
        const float f = m[n][r] == kNegInf ? 0.0f : ex2(m[n][r] - mx);
        if (g == 0u) s_l[row * W + warp] = l[n][r] * f;
        float* dst = s_o + (warp * TR + row) * S::kOut;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          dst[16 * i + g] = o[i][n][r] * f;
          dst[16 * i + 8 + g] = o[i][n][2 + r] * f;
        }
      }
    cta_sync();

    const uint64_t part_floats = TR * (D + 2);
    // partials of a job that several CTAs hold: the first CTA's is its second one (the job begins in its share),
    // every other's its first
    auto part_of = [&](uint32_t k) { return p.partials + (2ull * (cta0 + k) + (k == 0u ? 1u : 0u)) * part_floats; };
    float* mine = part_of(blockIdx.x - cta0);
    // a row's maximum and sum: the factor of its outputs, and lse
    auto finish_row = [&](uint32_t row, float mx, float ls) {
      s_fin[row] = make_float2(mx, ls == 0.0f ? 0.0f : (1.0f / kHold<DT>) / ls);
      if (p.lse && row < n_rows) {
        const uint32_t rr = r0 + row, tok = div_g(p, rr), hd = head * p.G + rr - tok * p.G;
        st4(p.lse + ((int64_t)x.q.row + tok) * p.HQ + hd,
            __float_as_uint(ls == 0.0f ? kNegInf : (mx + log2f(ls)) * 0.693147180559945309f));
      }
    };
    auto finish_out = [&](uint32_t r, uint32_t d4, float4 y) {
      const float inv = s_fin[r].y;
      const uint32_t rr = r0 + r, tok = div_g(p, rr), hd = head * p.G + rr - tok * p.G;
      st8(p.b + ((int64_t)x.q.row + tok) * p.b_row + (int64_t)hd * p.b_head + d4 * 4,
          inv == 0.0f ? make_uint2(0, 0)
                      : make_uint2(pack2<DT>(y.x * inv, y.y * inv), pack2<DT>(y.z * inv, y.w * inv)));
    };
    if (tid < n_rows) {
      float mx = kNegInf, ls = 0.0f;
      for (uint32_t w = 0; w < W; ++w) {
        mx = fmaxf(mx, s_m[tid * W + w]);
        ls += s_l[tid * W + w];
      }
      if (n_parts > 1u) st8(mine + TR * D + 2 * tid, make_uint2(__float_as_uint(mx), __float_as_uint(ls)));
      else finish_row(tid, mx, ls);
    }
    if (n_parts == 1u) cta_sync();
    for (uint32_t c4 = tid; c4 < n_rows * (D / 4); c4 += threads) {
      const uint32_t r = c4 / (D / 4), d4 = c4 % (D / 4);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t w = 0; w < W; ++w) {
        const float4 a = *reinterpret_cast<const float4*>(s_o + (w * TR + r) * S::kOut + d4 * 4);
        y.x += a.x; y.y += a.y; y.z += a.z; y.w += a.w;
      }
      if (n_parts > 1u)
        st16(mine + c4 * 4, make_uint4(__float_as_uint(y.x), __float_as_uint(y.y), __float_as_uint(y.z), __float_as_uint(y.w)));
      else finish_out(r, d4, y);
    }
    if (n_parts == 1u) continue;

    // ---- the CTA that finishes last joins the job's partial results
    // Whether this CTA is the last of n at a ticket.
    auto last_of = [&](uint32_t* ticket, uint32_t n) -> bool {
      cta_sync();
      if (tid == 0) {
        uint32_t last = 0;
        KVC_GUARD(ticket, 4, last = 2);
        if (last == 0) {
          // releases what this CTA stored (the barrier above put it before), acquires what the others did
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(last) : "l"(ticket) : "memory");
          last = last == n - 1u ? 1u : 0u;
          if (last) *ticket = 0;  // as the next call finds it
        }
        *s_last = last;
      }
      cta_sync();
      return *s_last == 1u;
    };
    // Join partials first, first + stride, ... (n of them) in this order: a row's outputs and lse, or (!whole) a partial
    // in place of the first.
    auto join = [&](uint32_t first, uint32_t stride, uint32_t n, bool whole) {
      // four dims a thread at each of its places; kU partials' loads at each place are in flight
      constexpr uint32_t kP = TR * D / 4 > threads ? TR * D / 4 / threads : 1, kU = (NT == 2 || D == 256 ? 8 : 16) / kP;
      float4 a[kP][kU], y[kP];
      auto load = [&](uint32_t k0) {
#pragma unroll
        for (uint32_t i = 0; i < kP; ++i)
#pragma unroll
          for (uint32_t k = 0; k < kU; ++k) {
            const uint32_t c4 = tid + i * threads;
            if (k0 + k < n && c4 < n_rows * (D / 4)) a[i][k] = ld_join4(part_of(first + (k0 + k) * stride) + c4 * 4);
          }
      };
      load(0);  // on their way while the factors are found
      for (uint32_t k = tid; k < n * TR; k += threads)
        s_ml[k] = k % TR < n_rows ? ld_join2(part_of(first + k / TR * stride) + TR * D + 2 * (k % TR)) : make_float2(kNegInf, 0.0f);
      cta_sync();
      for (uint32_t i = tid; i < 8u * TR; i += threads) {  // 8 threads a row
        const uint32_t row = i >> 3, part = i & 7u;
        float mx = kNegInf, ls = 0.0f;
        for (uint32_t k = part; k < n; k += 8) mx = fmaxf(mx, s_ml[k * TR + row].x);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        for (uint32_t k = part; k < n; k += 8) {
          const float2 ml = s_ml[k * TR + row];
          const float f = ml.x == kNegInf ? 0.0f : ex2(ml.x - mx);
          ls += ml.y * f;
          s_ml[k * TR + row].x = f;
        }
#pragma unroll
        for (int d = 1; d < 8; d *= 2) ls += __shfl_xor_sync(0xffffffffu, ls, d);
        if (part == 0) {
          if (whole) finish_row(row, mx, ls);
          else if (row < n_rows) st8(part_of(first) + TR * D + 2 * row, make_uint2(__float_as_uint(mx), __float_as_uint(ls)));
        }
      }
      cta_sync();
#pragma unroll
      for (uint32_t i = 0; i < kP; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t k0 = 0; k0 < n; k0 += kU) {
        if (k0) load(k0);
#pragma unroll
        for (uint32_t i = 0; i < kP; ++i)
#pragma unroll
          for (uint32_t k = 0; k < kU; ++k) {
            const uint32_t c4 = tid + i * threads;
            if (k0 + k < n && c4 < n_rows * (D / 4)) {
              const float f = s_ml[(k0 + k) * TR + c4 / (D / 4)].x;
              y[i].x += a[i][k].x * f;
              y[i].y += a[i][k].y * f;
              y[i].z += a[i][k].z * f;
              y[i].w += a[i][k].w * f;
            }
          }
      }
#pragma unroll
      for (uint32_t i = 0; i < kP; ++i) {
        const uint32_t c4 = tid + i * threads;
        if (c4 < n_rows * (D / 4)) {
          if (whole) finish_out(c4 / (D / 4), c4 % (D / 4), y[i]);
          else st16(part_of(first) + c4 * 4, make_uint4(__float_as_uint(y[i].x), __float_as_uint(y[i].y), __float_as_uint(y[i].z),
                                                        __float_as_uint(y[i].w)));
        }
      }
    };
    // Many partials are joined in groups of about their number's square root, each by its last CTA, then the groups.
    // (A group's tickets go by its first CTA: one job at most begins in a CTA's share, and one at most goes on into it.)
    uint32_t first_part = 0, stride = 1, n = n_parts, *ticket = p.tickets + cta0;
    const uint32_t group = n_parts <= kFlat ? n_parts : (uint32_t)sqrtf((float)n_parts) + 1u;
    if (group < n_parts) {
      first_part = (blockIdx.x - cta0) / group * group;
      n = min(group, n_parts - first_part);
      ticket += first_part + (first_part ? kC16Ctas : 0u);
    }
    bool whole = group == n_parts;
#pragma unroll 1
    while (last_of(ticket, n)) {
      join(first_part, stride, n, whole);
      if (whole) break;
      first_part = 0, stride = group, n = (n_parts + group - 1u) / group, whole = true;
      ticket = p.tickets + 2u * kC16Ctas + cta0;
    }
  }
}

template <int DT, int D, bool PAGED16, int NT>
int step_launch(const C16Params& p, uint32_t ctas, void* stream) {
  const auto kernel = c16_step_kernel<DT, D, PAGED16, NT>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, Shape16<D>::kSmem, done)) return KV_ERR_CUDA;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<ctas, kThreads16, Shape16<D>::kSmem, (cudaStream_t)stream>>>(p);
        return cudaGetLastError();
      },
      p);
}

template <int DT, int D>
int step_d(const C16Params& p, uint32_t ctas, void* stream) {
  if (p.T % 16 == 0)
    return p.tile_rows == 8u ? step_launch<DT, D, true, 1>(p, ctas, stream) : step_launch<DT, D, true, 2>(p, ctas, stream);
  return p.tile_rows == 8u ? step_launch<DT, D, false, 1>(p, ctas, stream) : step_launch<DT, D, false, 2>(p, ctas, stream);
}

}  // namespace

// Two CTAs an SM, fewer where the batch cannot have as many shares: host fields only, the device finds
// how many steps there are.
int launch_c16_attend(const C16Params& params, uint64_t jobs, uint64_t keys, void* stream) {
  C16Params p = params;
  const uint64_t most = kC16Ctas, steps = keys / (p.D >= 128u ? 16u : 32u) + 2u;
  // Up to half as many jobs as CTAs: even parts, one to a CTA, cost some CTAs at worst and no CTA two jobs (48 sequences with one KV
  // head, 96 jobs: 24.3 us with shares).
  p.even = 2u * jobs <= most ? 1u : 0u;
  const uint32_t ctas = (uint32_t)std::min<uint64_t>(
      most, p.even ? jobs * ((steps + kLeast - kStart - 1u) / (kLeast - kStart) + 1u) : (jobs * (steps + kStart) + kLeast - 1u) / kLeast);
  KVC_C8_DISPATCH(step_d, p, ctas, stream);
}

}  // namespace kvc
