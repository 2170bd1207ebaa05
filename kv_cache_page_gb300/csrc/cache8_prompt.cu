// cache8_prompt.cu -- attention of many query rows over the 8-bit cache: whole
// prompts and chunks of them.
//
//   S = Q K^T,  P = 2^(scale s_k S - m),  O = sum over key tiles of (s_v P) V
//
// Bound by the matrix products (4 D operations per query-key pair) and, next to
// them, by the exponentials.  A CTA takes 256 rows (two tiles of 128: the G query
// heads that share a KV head, times 256 / G new tokens) of one sequence and KV
// head, and walks the keys 128 at a time:
//   warps 8-11, 12-14  read the codes of V and of K, make FP16 of them (exactly) and
//               lay them out for the tensor cores, two tiles deep;
//   warp 15     issues the products: scores of both row tiles into TMEM, weights
//               (from TMEM) times V into accumulators in TMEM;
//   warps 0-3, 4-7  the softmax of row tile 0 and 1, a thread to a row: scores from
//               TMEM, weights back over them as FP16, the running maximum and sum.
// While one row tile's softmax runs, the tensor cores work on the other's products.
// The accumulators are rescaled only where a row's maximum grew by more than kLag.
//
// K and V share one layout, rows of 64 dims (128 bytes, 128-byte swizzle) per
// token: as the score product's B operand dims are its inner index (K-major), as the
// output product's B operand tokens are (MN-major), so V needs no transposition.
//
// Measured on a GB300, 2 prompts of 8192 tokens, 32 query heads of 128: 1.17 ms, 0.94 PFLOP/s
// (a plain matrix product: 1.94).  Of some 4850 clocks a key tile the softmax of a row
// tile takes 2800, its two products and the waits for them the rest; both row tiles
// overlap.  256 rows a CTA because K and V are converted once for both tiles; 128 keys
// because scores and outputs of two row tiles then fill the 512 columns of TMEM.
//
// Every wait has a limit; past it the CTA gives up, reports KV_CACHE8_STALLED and
// releases what it holds.
#include "cache8_common.cuh"

namespace kvc {
namespace {

constexpr float kNegInf = -INFINITY;
// Weights are held as 2^(z - m) * 2^11, m at most kLag below the true maximum (as
// the step kernel holds them).
constexpr float kLift = 11.0f, kLag = 4.0f;  // kLift: the logarithm
// The logarithm of V's scale in a weight's exponent, relative to the row's reference, is held at this at least:
// such weights, at most 2^(kLag + kFarV), are 0 in FP16 either way, and the sum gets them back whole (of a page of
// zeros, scale 2^-60, next to one of 2^100 they would leave FP32's range).
constexpr float kFarV = -40.0f;
constexpr int kKeys = 128;           // keys of a tile
constexpr int kSoftWarps = 8, kVWarps = 4, kKWarps = 3, kMmaWarp = kSoftWarps + kKWarps + kVWarps;
constexpr int kPromptThreads = (kMmaWarp + 1) * 32;
constexpr long long kWaitClocks = 4000000000ll;
constexpr uint32_t kWaitHint = 100000;  // ns that one try may sleep (polling would take issue slots from the softmax)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// at least kFarV; NaN stays NaN
__device__ __forceinline__ float far_v(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(kFarV));
  return y;
}

// The split of the registers between the roles (see the kernel).  The
// bounds-checked build leaves it out: its checks are calls, which the compiler
// cannot fit into a fixed split.
#ifdef KVC_BOUNDS_CHECK
__device__ __forceinline__ void regs_inc() {}
__device__ __forceinline__ void regs_dec() {}
#else
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 176;"); }
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); }
#endif

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival for the warp, after what all its lanes did (32 arrivals on one
// barrier are carried out one after the other).
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31u) == 0u) mbar_arrive(bar);
  __syncwarp();
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred q; mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 q, [%1], %2, %3; selp.u32 %0, 1, 0, q; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kWaitHint)
      : "memory");
  return ok != 0u;
}
// Wait for the phase of this parity; false when some two seconds have passed or
// another thread gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* stop) {
  if (mbar_try(bar, parity)) return true;
  const long long begin = clock64();
  for (;;) {
#pragma unroll 1
    for (int n = 0; n < 8; ++n)
      if (mbar_try(bar, parity)) return true;
    if (*stop) return false;
    if (clock64() - begin > kWaitClocks) {
      *stop = 1u;
      return false;
    }
  }
}

// ---------------------------------------------------------------- tensor cores
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The barrier gets an arrival when this thread's products so far are done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Shared memory operand: start, byte strides, 128-byte swizzle.
__host__ __device__ constexpr uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(ok));
  return ok != 0u;
}
// kind::f16, FP16 operands, FP32 accumulator, M = 128; bt: B is MN-major.
__host__ __device__ constexpr uint32_t tc_idesc(uint32_t n, uint32_t bt) {
  return (1u << 4) | (bt << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred q; setp.ne.u32 q, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred q; setp.ne.u32 q, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 columns of the warp's 32 TMEM lanes: a thread gets its lane's.
__device__ __forceinline__ void tm_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tm_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int D>
struct PromptShape {
  static constexpr int DG = D >= 64 ? D / 64 : 1;        // 64-dim groups (D = 32: half of one)
  static constexpr uint32_t kQTile = DG * 128 * 128;     // bytes
  static constexpr uint32_t kTile = DG * kKeys * 128;    // of K or V
  static constexpr uint32_t kQ = 0, kK = 2 * kQTile, kV = kK + 2 * kTile;
  // records of 4 tiles, FP32: K's scales [128], V's [128], log2 of V's [128] (whole pages: 8 of each), V's
  // largest, whether K has a 0
  static constexpr uint32_t kScale = kV + 2 * kTile;
  static constexpr uint32_t kScaleStage = (3 * kKeys + 4) * 4;
  static constexpr uint32_t kNan = kScale + 4 * kScaleStage;         // [record][token][D / 32] bits of V's NaN codes
  static constexpr uint32_t kRowNan = kNan + 4 * kKeys * (D / 32) * 4; // [row][D / 32]: dims whose output is NaN
  static constexpr uint32_t kBar = kRowNan + 256 * (D / 32) * 4;
  static constexpr uint32_t kBytes = kBar + 256;
  static constexpr uint32_t kS = 0, kO = 256;            // TMEM columns: scores 2 x 128, then outputs 2 x D
};

// ---------------------------------------------------------------- a row's scores
// A thread's row of a 128-key tile: bare products in TMEM at s_at (read twice, 32 at
// a time, the next on their way: holding all 128 left the compiler too few registers
// to overlap anything); K's and V's scales, of whole pages per 16 tokens, else per
// token; rf the row's factor; z = x k rf.  MASK: only
// columns [lo_c, hi_c) are seen, and of these none without a page: of whole pages
// their factor is -1 (a page's own may be 0, where scale and row are tiny), else their
// K scale is 0.
template <bool PAGED16, bool MASK>
__device__ __forceinline__ float row_max(uint32_t s_at, const float* ks, const float (&f8)[8], float rf, int32_t lo_c,
                                         int32_t hi_c) {
  float mt = kNegInf;
  uint32_t x[2][32];
  tm_ld32(s_at, x[0]);
#pragma unroll
  for (int c = 0; c < kKeys / 32; ++c) {
    tm_wait_ld();
    if (c + 1 < kKeys / 32) tm_ld32(s_at + 32 * (c + 1), x[(c + 1) & 1]);
    if (PAGED16) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float f = f8[2 * c + g];
        const int32_t hg = MASK && f < 0.0f ? -1 : hi_c;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int col = 32 * c + 16 * g + i;
          y[i] = __uint_as_float(x[c & 1][16 * g + i]);
          if (MASK && !(col < hg && col >= lo_c)) y[i] = kNegInf;
        }
#pragma unroll
        for (int i = 0; i < 5; ++i) y[i] = max3(y[3 * i], y[3 * i + 1], y[3 * i + 2]);
        y[0] = fmaxf(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[15]));
        mt = fmaxf(mt, __fmul_rn(y[0], MASK ? fabsf(f) : f));  // (-inf * 0 is NaN, which the maximum leaves out)
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 k = *reinterpret_cast<const float4*>(ks + 32 * c + i);
        const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 32 * c + i + e;
          float z = __fmul_rn(__uint_as_float(x[c & 1][i + e]), __fmul_rn(kk[e], rf));
          if (MASK && !(col < hi_c && col >= lo_c && kk[e] != 0.0f)) z = kNegInf;
          mt = fmaxf(mt, z);
        }
      }
    }
  }
  return mt;
}
// The weights times V's scale (relative to the row's reference, 2^-lref), as FP16
// over the scores; the sum of the bare weights.  The scale goes into the exponent,
// w = 2^(z - base + lv + lref) with lv its logarithm, and out of the sum again by
// its inverse, once for the tokens that share it.
// EXACT: z rounded as row_max rounded it before base is taken off.
template <bool PAGED16, bool MASK, bool EXACT>
__device__ __forceinline__ float row_weights(uint32_t s_at, const float* ks, const float* lv, const float (&f8)[8],
                                             const float (&l8)[8], float rf, float lref, float base, int32_t lo_c,
                                             int32_t hi_c) {
  constexpr int G = PAGED16 ? 16 : 4;  // columns handled together; of whole pages they share their scales
  float total = 0.0f;
  uint32_t x[2][32], w[2][16];
  tm_ld32(s_at, x[0]);
#pragma unroll
  for (int c = 0; c < kKeys / 32; ++c) {
    tm_wait_ld();
    if (c + 1 < kKeys / 32) tm_ld32(s_at + 32 * (c + 1), x[(c + 1) & 1]);
    if (c > 0) tm_st16(s_at + 16 * (c - 1), w[(c - 1) & 1]);  // (a chunk late: this one's work fills its tail)
#pragma unroll
    for (int i = 0; i < 32; i += G) {
      const int col = 32 * c + i;
      float kk[4], ll[4];
      if (PAGED16) {
        kk[0] = kk[1] = kk[2] = kk[3] = f8[col / 16];
        ll[0] = ll[1] = ll[2] = ll[3] = far_v(l8[col / 16] + lref);
        // a page that the row sees nothing of: its scale must not matter
        if (MASK && (col >= hi_c || col + 16 <= lo_c)) ll[0] = ll[1] = ll[2] = ll[3] = 0.0f;
      } else {
        const float4 k = *reinterpret_cast<const float4*>(ks + col), l = *reinterpret_cast<const float4*>(lv + col);
        kk[0] = k.x; kk[1] = k.y; kk[2] = k.z; kk[3] = k.w;
        ll[0] = far_v(l.x + lref); ll[1] = far_v(l.y + lref);
        ll[2] = far_v(l.z + lref); ll[3] = far_v(l.w + lref);
      }
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < G; e += 2) {
        const float k0 = kk[e & 3], k1 = kk[(e + 1) & 3];
        const float2 xx = make_float2(__uint_as_float(x[c & 1][i + e]), __uint_as_float(x[c & 1][i + e + 1]));
        const float2 f = PAGED16 ? make_float2(k0, k1) : make_float2(__fmul_rn(k0, rf), __fmul_rn(k1, rf));
        float2 z;
        if (EXACT)
          z = make_float2(__fadd_rn(__fadd_rn(__fmul_rn(xx.x, f.x), -base), ll[e & 3]),
                          __fadd_rn(__fadd_rn(__fmul_rn(xx.y, f.y), -base), ll[(e + 1) & 3]));
        else
          z = fma2(xx, f, make_float2(ll[e & 3] - base, ll[(e + 1) & 3] - base));
        if (MASK) {
          z.x = col + e < hi_c && col + e >= lo_c && (PAGED16 ? !(k0 < 0.0f) : k0 != 0.0f) ? z.x : kNegInf;
          z.y = col + e + 1 < hi_c && col + e + 1 >= lo_c && (PAGED16 ? !(k1 < 0.0f) : k1 != 0.0f) ? z.y : kNegInf;
        }
        const float2 y = make_float2(ex2(z.x), ex2(z.y));
        if (PAGED16) {
          sum = add2(sum, y);
        } else {
          if (!MASK || z.x != kNegInf) total += y.x * ex2(-ll[e & 3]);
          if (!MASK || z.y != kNegInf) total += y.y * ex2(-ll[(e + 1) & 3]);
        }
        w[c & 1][(i + e) / 2] = pack2<0>(y.x, y.y);
      }
      if (PAGED16) total += (sum.x + sum.y) * ex2(-ll[0]);
    }
  }
  tm_st16(s_at + 16 * (kKeys / 32 - 1), w[(kKeys / 32 - 1) & 1]);
  return total;
}

// ---------------------------------------------------------------- codes to FP16 tiles
// W warps bring K (IS_K) or V of tile after tile into its two stages.  A 16-byte
// chunk of codes, CPR of a 64-dim group a token, a thread to each, makes two 16-byte
// chunks of FP16 (8 lanes in turn, 4 chunks of two tokens, write to 8 different bank
// groups).  A chunk of the next tile is asked for as soon as one of this tile is
// written, its page known a tile earlier.
template <int D, bool PAGED16, bool IS_K, int W>
__device__ __forceinline__ void load_tiles(const C8Params& p, const C8Seq& q, uint8_t* smem, uint32_t head, int32_t lo,
                                           int32_t hi, int32_t n_steps, uint32_t full, uint32_t empty,
                                           uint32_t scales, volatile uint32_t* stop, uint32_t* nan_seen) {
  using S = PromptShape<D>;
  constexpr int CPR = D >= 64 ? 4 : 2;
  constexpr int RPI = W * 32 / CPR;                        // token rows at once
  constexpr int NR = (kKeys + RPI - 1) / RPI, N = NR * S::DG;  // chunks of a thread and tile: rows, then groups
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t lt = threadIdx.x - (kSoftWarps + (IS_K ? kVWarps : 0)) * 32u;
  const uint32_t row = lt / CPR, c = lt % CPR;
  const uint8_t* src = (IS_K ? p.k : p.v) + (int64_t)head * p.sh + c * 16;
  const uint32_t dst0 = row * 128 + (((2 * c) ^ (row & 7u)) << 4), dst1 = row * 128 + (((2 * c + 1) ^ (row & 7u)) << 4);
  bool bad = false;
  // Byte offset in the cache of a token's row (PAGED16: of a run of 16 tokens), -1:
  // none.  PAGED16: lane g & 7 holds the offset and page of run g of a tile; tokens
  // past the last one in its run hold anything.
  auto place = [&](int32_t tok, int32_t& id) -> int64_t {
    id = -1;
    if (tok >= hi) return -1;
    const uint32_t i = c8_div_t(p, (uint32_t)tok);
    id = c8_page(p, q.s, i);
    if (id < 0) {
      bad = true;
      return -1;
    }
    return (int64_t)id * p.sb + (int64_t)((uint32_t)tok - i * p.T) * p.st;
  };
  uint4 x[N];  // (of tokens without a page: what an earlier tile had; their scales are 0)
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = make_uint4(0, 0, 0, 0);
  const int64_t row_off[2] = {(int64_t)(row & 15u) * p.st, (int64_t)((row + RPI) & 15u) * p.st};
  // the scales of both, brought with V: a V stage stays until the softmax is done with its tile, a K stage does not
  float ksc[(kKeys + W * 32 - 1) / (W * 32)], vsc[(kKeys + W * 32 - 1) / (W * 32)];
  int32_t id = -1;
  int64_t run = -1;
  int32_t entry = -2;  // raw table entry of this lane's run of the tile asked for, -2: past the last token
  auto ask = [&](int32_t j) {
    const int32_t tok = lo + j * kKeys + 16 * (int32_t)(lane & 7u);
    entry = -2;
    if (PAGED16 && tok < hi) {
      const uint32_t i = c8_div_t(p, (uint32_t)tok);
      entry = i < p.table_width ? ldg_i32(p.tables + (int64_t)q.s * p.table_stride + i) : -1;
    }
  };
  // Where the rows of tile j lie, and its scales (asked for; in registers a tile later).
  const uint8_t* from[NR];
  auto locate = [&](int32_t j) {
    const int32_t tok0 = lo + j * kKeys;
    if (PAGED16) {
      const int32_t tok = tok0 + 16 * (int32_t)(lane & 7u);
      const bool ok = (uint32_t)entry < p.num_blocks;
      bad |= !ok && entry != -2;
      id = ok ? entry : -1;
      run = ok ? (int64_t)entry * p.sb + (int64_t)((uint32_t)tok - c8_div_t(p, (uint32_t)tok) * p.T) * p.st : -1;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t r = i * RPI + row;  // token row of the tile
      int64_t off = -1;
      if (PAGED16) {
        off = __shfl_sync(0xffffffffu, run, (r >> 4) & 7u);
      } else if (kKeys % RPI == 0 || r < kKeys) {
        int32_t ignore;
        off = place(tok0 + (int32_t)r, ignore);
      }
      from[i] = off >= 0 && (kKeys % RPI == 0 || r < kKeys) ? src + off + (PAGED16 ? row_off[i & 1] : 0) : nullptr;
    }
    if (!IS_K && PAGED16) {  // lane g & 7: run g
      ksc[0] = id >= 0 ? ldg_f32(p.k_scale + (int64_t)id * p.H + head) : 0.0f;
      vsc[0] = id >= 0 ? ldg_f32(p.v_scale + (int64_t)id * p.H + head) : 0.0f;
    }
#pragma unroll
    for (int i = 0; !IS_K && !PAGED16 && i * W * 32 < kKeys; ++i) {
      const uint32_t r = i * W * 32 + lt;
      int32_t at = -1;
      if (r < kKeys) place(tok0 + (int32_t)r, at);
      ksc[i] = at >= 0 ? ldg_f32(p.k_scale + (int64_t)at * p.H + head) : 0.0f;
      vsc[i] = at >= 0 ? ldg_f32(p.v_scale + (int64_t)at * p.H + head) : 0.0f;
    }
  };
  auto fetch = [&](int i) {  // chunk i of the tile located last
    if (from[i / S::DG]) x[i] = ld_nc16(from[i / S::DG] + 64 * (i % S::DG));
  };
  auto nan_of = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
  ask(0);
  locate(0);
  ask(1);
#pragma unroll
  for (int i = 0; i < N; ++i) fetch(i);
  for (int32_t j = 0; j < n_steps; ++j) {
    const uint32_t st = j & 1, ph = (j >> 1) & 1;
    if (!IS_K) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) any |= nan_of(x[i].x) | nan_of(x[i].y) | nan_of(x[i].z) | nan_of(x[i].w);
      any = __any_sync(0xffffffffu, any != 0u) ? 1u : 0u;
      if (any) {  // NaN codes become 0; where they were is kept, a bit each, for the rows that see them
#pragma unroll
        for (int i = 0; i < N; ++i) {
          uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
          uint32_t bits = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t nb = nan_of(w[k]);
            w[k] &= ~((nb >> 7) * 0xffu);
            bits |= (((nb >> 7) * 0x01020408u) >> 24) << (4 * k);  // one bit per byte, in order
          }
          const uint32_t r = (i / S::DG) * RPI + row;
          if (r < kKeys)
            reinterpret_cast<uint16_t*>(smem + S::kNan)[((j & 3) * kKeys + r) * (D / 16) + (i % S::DG) * 4 + c] =
                (uint16_t)bits;
        }
      }
      if (lane == 0) reinterpret_cast<uint8_t*>(nan_seen)[4 * (j & 3) + (lt >> 5)] = (uint8_t)any;
    }
    float* sc = reinterpret_cast<float*>(smem + S::kScale + (j & 3) * S::kScaleStage);
    if (!IS_K && PAGED16 && lt < 32u) {
      float top = vsc[0];
#pragma unroll
      for (int d = 1; d < 8; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const bool hole = __any_sync(0xffffffffu, ksc[0] == 0.0f);
      if (lane < 8u) {
        sc[lane] = ksc[0];
        sc[kKeys + lane] = vsc[0];
        sc[2 * kKeys + lane] = vsc[0] > 0.0f ? lg2(vsc[0]) : vsc[0];
      }
      if (lane == 0u) {
        sc[3 * kKeys] = top;
        sc[3 * kKeys + 1] = hole ? 1.0f : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; !IS_K && !PAGED16 && i * W * 32 < kKeys; ++i)
      if (kKeys % (W * 32) == 0 || i * W * 32 + lt < kKeys) {
        sc[i * W * 32 + lt] = ksc[i];
        sc[kKeys + i * W * 32 + lt] = vsc[i];
        sc[2 * kKeys + i * W * 32 + lt] = vsc[i] > 0.0f ? lg2(vsc[i]) : vsc[i];
      }
    // The softmax wants these and the NaN flags before V itself: they do not wait for V's stage.  (Record j mod 4
    // is free: the softmax is past tile j - 3, whose product this loop has waited for.)
    if (!IS_K) mbar_arrive_warp(scales + 8 * (j & 3));
    if (!__all_sync(0xffffffffu, mbar_wait(empty + 8 * st, ph ^ 1u, stop))) break;
    uint8_t* tile = smem + (IS_K ? S::kK : S::kV) + st * S::kTile;
    locate(j + 1);
    ask(j + 2);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint4 h0, h1;
      c8_dec4(x[i].x, h0.x, h0.y);
      c8_dec4(x[i].y, h0.z, h0.w);
      c8_dec4(x[i].z, h1.x, h1.y);
      c8_dec4(x[i].w, h1.z, h1.w);
      uint8_t* at = tile + (i % S::DG) * (kKeys * 128) + (i / S::DG) * (RPI * 128);
      if (kKeys % RPI == 0 || (i / S::DG) * RPI + row < kKeys) {
        *reinterpret_cast<uint4*>(at + dst0) = h0;
        *reinterpret_cast<uint4*>(at + dst1) = h1;
      }
      fetch(i);  // the next tile's, while the others are converted
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive_warp(full + 8 * st);
  }
  if (bad) c8_error(p, q.s, KV_CACHE8_BAD_PAGE);
}

template <int DT, int D, bool PAGED16>
__global__ void __launch_bounds__(kPromptThreads, 1) c8_prompt_kernel(const __grid_constant__ C8Params p) {
  using S = PromptShape<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;

  // late row tiles first: under a causal mask they have the most keys
  const uint32_t us = blockIdx.x / p.H, head = blockIdx.x - us * p.H;
  const C8Seq q = c8_find(p, p.n_units - 1u - us, p.G, kPromptRows, 1u, 0u);
  const uint32_t rows = (uint32_t)q.n_new * p.G, r0 = q.unit * kPromptRows;
  if (q.unit > rows / kPromptRows || r0 >= rows || rows < p.min_rows || rows > p.max_rows) return;
  const uint32_t n_rows = min(kPromptRows, rows - r0);
  const uint32_t n_tiles = n_rows > 128u ? 2u : 1u;

  // the keys that some row sees
  const int32_t first_pos = q.start + (int32_t)(r0 / p.G), last_pos = q.start + (int32_t)((r0 + n_rows - 1u) / p.G);
  const int32_t hi = max(p.causal ? min(q.len, last_pos + 1) : q.len, 0);
  int32_t lo = p.window && first_pos >= 0 ? max(0, first_pos - (int32_t)min(p.window, 0x7fffffffu) + 1) : 0;
  if (PAGED16) lo &= ~15;  // runs of 16 tokens; else the page of a token before may be freed
  const int32_t n_steps = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;

  // barriers
  const uint32_t bar = sbase + S::kBar;
  const uint32_t k_full = bar, k_empty = bar + 16, v_full = bar + 32, v_empty = bar + 48;  // [2]
  const uint32_t s_full = bar + 64, p_full = bar + 80, pv_done = bar + 96;                  // [2]
  const uint32_t q_full = bar + 144, c_full = bar + 152;                                   // c_full: [4]
  volatile uint32_t* stop = reinterpret_cast<volatile uint32_t*>(smem + S::kBar + 112);
  uint32_t* nan_seen = reinterpret_cast<uint32_t*>(smem + S::kBar + 192);   // [record]: a byte a loading warp, V has NaN codes
  uint32_t* any_row_nan = reinterpret_cast<uint32_t*>(smem + S::kBar + 124);
  uint32_t* tm_at = reinterpret_cast<uint32_t*>(smem + S::kBar + 128);
  if (tid == 0) {
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, kKWarps);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, kVWarps);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(c_full + 8 * i, kVWarps);
      mbar_init(c_full + 8 * i + 16, kVWarps);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(pv_done + 8 * i, 1);
      nan_seen[i] = nan_seen[i + 2] = 0;
    }
    mbar_init(q_full, kSoftWarps);
    *stop = 0;
    *any_row_nan = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(tm_at))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tm_at;

  // ---- Q to shared memory, each softmax warp its own 32 rows; bf16 rows are scaled by
  // a power of two into FP16's range (exact down to 2^-31 of the row's largest, below that
  // to 2^-39 of it)
  const uint32_t r = tid;  // row of the CTA, for threads of the softmax
  const bool in = tid < 256u && r < n_rows;
  const uint32_t rr = r0 + (in ? r : 0u), tok_r = rr / p.G, hd = head * p.G + rr - tok_r * p.G;
  float rf = p.scale_log2;
  if (tid < 256u) {
    constexpr uint32_t LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows at once
    const int64_t off = in ? ((int64_t)q.row + tok_r) * p.a_row + (int64_t)hd * p.a_head : -1;
    const uint32_t c = lane % LPR;
#pragma unroll
    for (uint32_t h = 0; h < LPR; h += LPR / 2) {  // half of the rows' loads in flight at a time
      uint4 x[LPR / 2];
#pragma unroll
      for (uint32_t i = 0; i < LPR / 2; ++i) {
        const int64_t o = __shfl_sync(0xffffffffu, off, (h + i) * RPI + lane / LPR);
        x[i] = o >= 0 ? ld_nc16(p.a + o + 8 * c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (uint32_t i = 0; i < LPR / 2; ++i) {
        const uint32_t row = (h + i) * RPI + lane / LPR;
        if (DT == 1) {
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, m = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            m = max(m, (w[k] & 0x7fffu) < 0x7f80u ? (w[k] & 0x7fffu) : 0u);
            m = max(m, ((w[k] >> 16) & 0x7fffu) < 0x7f80u ? ((w[k] >> 16) & 0x7fffu) : 0u);
          }
#pragma unroll
          for (uint32_t d = LPR / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
          // the largest magnitude, in [2^k, 2^(k+1)), goes to [2^14, 2^15)
          const int ex = m ? min(max(14 - ((int)(m >> 7) - 127), -120), 120) : 0;
          const float f = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack2<0>(lo_f32<1>(w[k]) * f, hi_f32<1>(w[k]) * f);
          x[i] = make_uint4(w[0], w[1], w[2], w[3]);
          // the row's thread undoes the scaling in its factor
          const int e_row = __shfl_sync(0xffffffffu, ex, (lane % RPI) * LPR);
          if (lane / RPI == h + i) rf = p.scale_log2 * __uint_as_float((uint32_t)(127 - e_row) << 23);
        }
        *reinterpret_cast<uint4*>(smem + S::kQ + (warp >> 2) * S::kQTile + (c >> 3) * (128 * 128) +
                                  ((warp & 3u) * 32u + row) * 128 + (((c & 7u) ^ (row & 7u)) << 4)) = x[i];
      }
    }
    uint32_t* rn = reinterpret_cast<uint32_t*>(smem + S::kRowNan) + r * (D / 32);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) rn[k] = 0;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive_warp(q_full);
  }

  // Registers: 512 threads start with 128 each; the softmax takes 176 (two chunks of 32 scores
  // and their weights under way), the others keep 80: 256 x 176 + 256 x 80 = 512 x 128.
  // A warpgroup makes its split at one place: warps 12 .. 15, of two roles, are one.
  // (Two prompts of 8192 tokens, D = 128: 1174 us this way, 1194 with one place for warps
  // 8 .. 15, 1218 with K's loaders before the products.)
  static_assert(kPromptThreads == 512 && kSoftWarps == 8, "");
  if (warp < kSoftWarps) {
    // ================================================================ softmax
    regs_inc();
    const uint32_t t = warp >> 2;
    float m = kNegInf, l = 0.0f, vref = 1.17549435e-38f, lref = 0.0f;  // lref: 11 - log2(vref), once the row has seen a scale
    bool fine = true;
    if (t < n_tiles) {
      const uint32_t tl = tm + ((warp & 3u) << 21);  // the warp's 32 lanes (lane << 16)
      const uint32_t s_at = tl + S::kS + t * 128, o_at = tl + S::kO + t * D;
      const int32_t pos = q.start + (int32_t)tok_r;
      int32_t vis_hi = p.causal ? min(q.len, pos + 1) : q.len;
      const int32_t vis_lo = p.window ? (int32_t)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
      if (!in || pos < 0) vis_hi = 0;
      // tiles of keys between these are seen whole by every row of the tile
      const uint32_t ra = r0 + t * 128, rb = r0 + min(n_rows, t * 128 + 128u) - 1u;
      const int32_t pos_a = q.start + (int32_t)(ra / p.G), pos_b = q.start + (int32_t)(rb / p.G);
      const int32_t full_hi = min(hi, pos_a < 0 ? 0 : p.causal ? min(q.len, pos_a + 1) : q.len);
      const int32_t full_lo = p.window ? (int32_t)max((int64_t)0, (int64_t)pos_b - p.window + 1) : 0;
      for (int32_t j = 0; j < n_steps && fine; ++j) {
        const int32_t tok0 = lo + j * kKeys;
        const uint32_t rec = j & 3;
        const float* ks = reinterpret_cast<const float*>(smem + S::kScale + rec * S::kScaleStage);
        const float* vs = ks + kKeys;
        fine = mbar_wait(c_full + 8 * rec, (j >> 2) & 1, stop) && mbar_wait(s_full + 8 * t, j & 1, stop);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        __syncwarp();
        tc_fence_after();
        // holes of K (a token without a page has the scale 0), the largest scale of V
        const uint32_t nan_w = nan_seen[rec];
        float vt = ks[3 * kKeys];
        bool hole = ks[3 * kKeys + 1] != 0.0f;
        if (!PAGED16) {
          vt = 0.0f;
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) {
            vt = fmaxf(vt, vs[32 * i + lane]);
            hole |= ks[32 * i + lane] == 0.0f;
          }
#pragma unroll
          for (int d = 1; d < 32; d *= 2) vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, d));
          hole = __any_sync(0xffffffffu, hole);
        }
        const bool masked = hole || tok0 + kKeys > full_hi || tok0 < full_lo;
        // among what the row sees: another page's scale must not push its weights out of FP16's range
        if (masked) {
          vt = 0.0f;
          if (PAGED16) {
#pragma unroll
            for (int g = 0; g < kKeys / 16; ++g)
              if (tok0 + 16 * g < vis_hi && tok0 + 16 * g + 16 > vis_lo) vt = fmaxf(vt, vs[g]);
          } else {
            for (int32_t c = max(0, vis_lo - tok0); c < min(kKeys, vis_hi - tok0); ++c) vt = fmaxf(vt, vs[c]);
            __syncwarp();
          }
        }
        // columns [lo_c, hi_c) of the tile are seen
        const int32_t hi_c = vis_hi - tok0, lo_c = vis_lo - tok0;
        // (whole pages) K's scale times the row's factor, -1 without a page; V's scale as a logarithm
        float f8[8], l8[8];
        if (PAGED16) {
#pragma unroll
          for (int g = 0; g < 8; g += 4) {
            const float4 k = *reinterpret_cast<const float4*>(ks + g), v = *reinterpret_cast<const float4*>(vs + kKeys + g);
            f8[g] = __fmul_rn(k.x, rf); f8[g + 1] = __fmul_rn(k.y, rf);
            f8[g + 2] = __fmul_rn(k.z, rf); f8[g + 3] = __fmul_rn(k.w, rf);
            if (hole) {
              f8[g] = k.x == 0.0f ? -1.0f : f8[g]; f8[g + 1] = k.y == 0.0f ? -1.0f : f8[g + 1];
              f8[g + 2] = k.z == 0.0f ? -1.0f : f8[g + 2]; f8[g + 3] = k.w == 0.0f ? -1.0f : f8[g + 3];
            }
            l8[g] = v.x; l8[g + 1] = v.y; l8[g + 2] = v.z; l8[g + 3] = v.w;
          }
        }
        float mt = masked ? row_max<PAGED16, true>(s_at, ks, f8, rf, lo_c, hi_c)
                          : row_max<PAGED16, false>(s_at, ks, f8, rf, lo_c, hi_c);
        const bool grow = mt > m + kLag;
        if (__any_sync(0xffffffffu, grow || vt > vref)) {
          const float vn = fmaxf(vt, vref);
          const float mn = grow ? mt : m;
          const float f = m == kNegInf ? 0.0f : ex2(m - mn);
          l *= f;
          m = mn;
          if (j > 0) {  // the accumulator, once the products before are done
            fine = __all_sync(0xffffffffu, mbar_wait(pv_done + 8 * t, (j - 1) & 1, stop));
            if (!fine) break;
            __syncwarp();
            tc_fence_after();
            const float fo = f * (vref / vn);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t y[32];
              tm_ld32(o_at + 32 * c, y);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * fo);
              tm_st32(o_at + 32 * c, y);
            }
          }
          vref = vn;
          if (vn > 1.17549435e-38f) lref = kLift - lg2(vn);
        }
        const float base = m == kNegInf ? 0.0f : m;
        // (bits are kept by the loading warps that saw one: rows 8 w .. 8 w + 7 of a round of kVWarps * 8)
        auto tok_nan = [&](int32_t c) {
          constexpr int R = D >= 64 ? 8 : 16;
          return (nan_w >> (8 * ((c / R) % kVWarps))) & 1u;
        };
        if (masked && nan_w) {
          // V has NaN codes (laid out as 0): the dims that a token seen by this row has them at
          const uint32_t* bits = reinterpret_cast<const uint32_t*>(smem + S::kNan) + rec * kKeys * (D / 32);
          uint32_t* rn = reinterpret_cast<uint32_t*>(smem + S::kRowNan) + r * (D / 32);
          uint32_t any = 0;
          for (int32_t c = max(0, vis_lo - tok0); c < min(kKeys, vis_hi - tok0); ++c)
            if (tok_nan(c))
              for (int k = 0; k < D / 32; ++k) {
                const uint32_t b = bits[c * (D / 32) + k];
                any |= b;
                rn[k] |= b;
              }
          if (any) *any_row_nan = 1;
        } else if (nan_w) {
          const uint32_t* bits = reinterpret_cast<const uint32_t*>(smem + S::kNan) + rec * kKeys * (D / 32);
          uint32_t* rn = reinterpret_cast<uint32_t*>(smem + S::kRowNan) + r * (D / 32);
          for (int32_t c = 0; c < kKeys; ++c)
            if (tok_nan(c))
              for (int k = 0; k < D / 32; ++k) rn[k] |= bits[c * (D / 32) + k];
          *any_row_nan = 1;
        }
        __syncwarp();
        // 2^(s f - m) in one step, unless m is so large that its own rounding would show
        if (__any_sync(0xffffffffu, fabsf(base) >= 1048576.0f))
          l += row_weights<PAGED16, true, true>(s_at, ks, vs + kKeys, f8, l8, rf, lref, base, lo_c, hi_c);
        else if (masked)
          l += row_weights<PAGED16, true, false>(s_at, ks, vs + kKeys, f8, l8, rf, lref, base, lo_c, hi_c);
        else
          l += row_weights<PAGED16, false, false>(s_at, ks, vs + kKeys, f8, l8, rf, lref, base, lo_c, hi_c);
        tm_wait_st();
        tc_fence_before();
        mbar_arrive_warp(p_full + 8 * t);
      }
      // ---- outputs
      if (n_steps > 0 && fine) {
        fine = __all_sync(0xffffffffu, mbar_wait(pv_done + 8 * t, (n_steps - 1) & 1, stop));
        tc_fence_after();
      }
      if (fine) {
        const float inv = l == 0.0f ? 0.0f : vref / (l * 2048.0f);
        uint16_t* out = p.b + ((int64_t)q.row + tok_r) * p.b_row + (int64_t)hd * p.b_head;
        const uint32_t* rn = reinterpret_cast<const uint32_t*>(smem + S::kRowNan) + r * (D / 32);
        const bool fix = *any_row_nan != 0u;
        const bool out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          __syncwarp();
          if (n_steps > 0) {
            tm_ld32(o_at + 32 * c, x);
            tm_wait_ld();
          }
          if (in) {
            if (fix && rn[c]) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((rn[c] >> i) & 1u) x[i] = 0x7fffffffu;
            }
            uint4 y4[4];
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = inv == 0.0f ? 0.0f : __uint_as_float(x[i + k]) * inv;
              y4[i / 8] = pack8<DT>(y);
            }
            if (out32) {
              st32(out + 32 * c, y4[0], y4[1]);
              st32(out + 32 * c + 16, y4[2], y4[3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) st16(out + 32 * c + 8 * i, y4[i]);
            }
          }
        }
        if (p.lse && in)
          st4(p.lse + ((int64_t)q.row + tok_r) * p.HQ + hd,
              __float_as_uint(l == 0.0f ? kNegInf : (m + log2f(l)) * 0.693147180559945309f));
      }
    }
  } else if (warp < kSoftWarps + kVWarps) {
    // ================================================================ V's codes to FP16 tiles
    regs_dec();
    load_tiles<D, PAGED16, false, kVWarps>(p, q, smem, head, lo, hi, n_steps, v_full, v_empty, c_full, stop, nan_seen);
  } else {
    regs_dec();  // (both roles of this warpgroup)
    if (warp == kMmaWarp) {
      // ============================================================== products
      if (n_steps > 0) {
        // The whole warp walks, one lane issues: what the instructions take is uniform.
        // (All 512 columns are allocated, so TMEM starts at column 0.)
        const bool one = elect_one();
        bool fine = true;
        constexpr uint64_t kDescK = tc_desc(0, 16, 1024), kDescV = tc_desc(0, kKeys * 128, 1024);
        const uint32_t q_lo = (sbase + S::kQ) >> 4, k_lo = (sbase + S::kK) >> 4, v_lo = (sbase + S::kV) >> 4;
        auto scores = [&](uint32_t t, int32_t j) {
          const uint64_t a = kDescK | (q_lo + t * (S::kQTile >> 4)), b = kDescK | (k_lo + (j & 1) * (S::kTile >> 4));
          if (one) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc_mma_ss(S::kS + t * 128, a + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                        b + (((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4), tc_idesc(kKeys, 0), k > 0);
            tc_commit(s_full + 8 * t);
          }
        };
        auto wait = [&](uint32_t at, uint32_t parity) {
          fine = __all_sync(0xffffffffu, mbar_wait(at, parity, stop));
          __syncwarp();
          tc_fence_after();
          return fine;
        };
        if (wait(q_full, 0) && wait(k_full, 0)) {
          for (uint32_t t = 0; t < n_tiles; ++t) scores(t, 0);
          if (one) tc_commit(k_empty);
        }
        for (int32_t j = 0; j < n_steps && fine; ++j) {
          const uint32_t st = j & 1;
          if (!wait(v_full + 8 * st, (j >> 1) & 1)) break;
          for (uint32_t t = 0; t < n_tiles; ++t) {
            if (!wait(p_full + 8 * t, j & 1)) break;
            const uint64_t b = kDescV | (v_lo + st * (S::kTile >> 4));
            if (one) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                tc_mma_ts(S::kO + t * D, S::kS + t * 128 + 8 * k, b + ((k * 2048) >> 4), tc_idesc(D, 1), j > 0 || k > 0);
              tc_commit(pv_done + 8 * t);
              if (t + 1 == n_tiles) tc_commit(v_empty + 8 * st);
            }
            if (j + 1 < n_steps) {
              if (t == 0 && !wait(k_full + 8 * ((j + 1) & 1), ((j + 1) >> 1) & 1)) break;
              scores(t, j + 1);
              if (one && t + 1 == n_tiles) tc_commit(k_empty + 8 * ((j + 1) & 1));
            }
          }
        }
        if (!fine && one) {
          // products still in flight end before their memory goes
          const uint32_t sb = (uint32_t)__cvta_generic_to_shared(smem + S::kBar + 136);
          mbar_init(sb, 1);
          tc_commit(sb);
          *stop = 0u;  // the others have given up or will at their own limit
          mbar_wait(sb, 0, stop);
          *stop = 1u;
        }
      }
    } else {
      // ============================================================== K's codes
      load_tiles<D, PAGED16, true, kKWarps>(p, q, smem, head, lo, hi, n_steps, k_full, k_empty, 0u, stop, nan_seen);
    }
  }
  __syncwarp();
  tc_fence_before();
  // (counts threads: the roles' loops may leave a warp diverged)
  asm volatile("barrier.sync 0;" ::: "memory");
  if (tid == 0 && *stop) c8_error(p, q.s, KV_CACHE8_STALLED);  // whichever role gave up
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

template <int DT, int D, bool PAGED16>
int prompt_launch(const C8Params& p, void* stream) {
  constexpr int bytes = PromptShape<D>::kBytes;
  const auto kernel = c8_prompt_kernel<DT, D, PAGED16>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kernel, bytes, done)) return KV_ERR_CUDA;
  const uint64_t gx = (uint64_t)p.n_units * p.H;
  if (gx > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        kernel<<<(unsigned)gx, kPromptThreads, bytes, (cudaStream_t)stream>>>(p);
        return cudaGetLastError();
      },
      p);
}

template <int DT, int D>
int prompt_d(const C8Params& p, void* stream) {
  return p.T % 16 == 0 ? prompt_launch<DT, D, true>(p, stream) : prompt_launch<DT, D, false>(p, stream);
}

}  // namespace

int launch_c8_prompt(const C8Params& p, void* stream) {
  switch (p.D) {
    case 32: return p.dtype == KV_DT_FP16 ? prompt_d<0, 32>(p, stream) : prompt_d<1, 32>(p, stream);
    case 64: return p.dtype == KV_DT_FP16 ? prompt_d<0, 64>(p, stream) : prompt_d<1, 64>(p, stream);
    case 128: return p.dtype == KV_DT_FP16 ? prompt_d<0, 128>(p, stream) : prompt_d<1, 128>(p, stream);
  }
  return KV_ERR_UNSUPPORTED_HEAD_DIM;
}

}  // namespace kvc
