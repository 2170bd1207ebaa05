// cache16_append.cu -- new tokens into the 16-bit pages, keys turned by their
// positions on the way, and the same tokens' queries.
//
// Bound by memory: every value is read and written once (4 bytes a value of K, V and
// queries; the tables' rows come from L2 for all heads but the first).  A warp takes a
// row, or the part of its heads that keeps 128 bytes a lane in flight; it asks for the
// row's values first, and finds the row's sequence, position and page (three dependent
// trips to memory) while these are on their way.  K, V and queries are one launch.
// Measured on a GB300, 4 x 8192 tokens with 8 KV heads and 32 query heads of 128 in FP16: 125 us,
// 6.5 TB/s (a plain copy 6.7).
#include "rotate.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kQueries = 4;     // iterations of a queries' warp: 128 bytes of loads in flight a lane
constexpr uint32_t kIterations = 2;  // of K and V each: 128 bytes of loads in flight a lane

struct Append16 : AppendParams {
  RowMap kv, qm;
  uint32_t kv_blocks;
};

#ifdef KVC_BOUNDS_CHECK
inline void dbg_ranges(DbgRanges& r, const Append16& p) {
  const uint64_t last = (uint64_t)p.sb * (p.num_blocks - 1u) + (uint64_t)p.st * (p.T - 1u) +
                        (uint64_t)p.sh * (p.H - 1u) + 2u * p.D;
  dbg_add(r, p.k, dbg_slot_bytes(last));
  dbg_add(r, p.v, dbg_slot_bytes(last));
  dbg_add(r, p.tables, 4ull * ((uint64_t)p.table_stride * (p.n_seqs - 1u) + p.table_width));
  dbg_add(r, p.lens, 4ull * p.n_seqs);
  if (p.cu) dbg_add(r, p.cu, 4ull * (p.n_seqs + 1u));
  if (p.errors) dbg_add(r, p.errors, 4ull * p.n_seqs);
  dbg_rows(r, p.a, p.a_row, p.a_head, p, p.H);
  dbg_rows(r, p.b, p.b_row, p.b_head, p, p.H);
  dbg_append(r, p);
}
#endif

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) c16_append_kernel(const __grid_constant__ Append16 p) {
  constexpr uint32_t U = D / 16, C = D / 8, I = kIterations;
  const uint32_t lane = threadIdx.x & 31u;
  if (blockIdx.x >= p.kv_blocks)
    return append_queries<DT, D, kQueries>(p, p.qm, (blockIdx.x - p.kv_blocks) * kWarps + (threadIdx.x >> 5));
  const RowMap& m = p.kv;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (warp >= m.warps) return;
  const uint32_t per = 32u >> m.log2, l = lane & ((1u << m.log2) - 1u);
  const uint32_t group = warp / m.slabs, slab = warp - group * m.slabs;
  const uint32_t row0 = group * per, row = row0 + (lane >> m.log2);
  const uint32_t first = slab * m.span + l, units = p.H * U;
  const RotUnit r = rot_unit<D>(p.R, p.neighbours, first % U);  // the same for all iterations
  // V is not turned: its chunks are dealt in their order, chunk vc + i 2^log2
  const uint32_t vc = 2u * slab * m.span + l;
  uint4 k[I][2], v[2 * I];
#pragma unroll
  for (uint32_t i = 0; i < I; ++i) {
    const uint32_t u = first + (i << m.log2);
    const bool in = row < p.n_new && u < units;
    const uint16_t* src = p.a + (int64_t)row * p.a_row + (int64_t)(u / U) * p.a_head;
    k[i][0] = in ? ld_stream16<true>(src + r.c0) : make_uint4(0, 0, 0, 0);
    k[i][1] = in ? ld_stream16<true>(src + r.c1) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (uint32_t i = 0; i < 2 * I; ++i) {
    const uint32_t c = vc + (i << m.log2);
    const bool in = row < p.n_new && c < 2u * units;
    v[i] = in ? ld_stream16<true>(p.b + (int64_t)row * p.b_row + (int64_t)(c / C) * p.b_head + (c % C) * 8u)
              : make_uint4(0, 0, 0, 0);
  }
  const RowPlace at = row_place(p, row0, row);
  if (!at.in || at.pos < 0) return;
  const uint32_t page = c8_div_t(p, (uint32_t)at.pos);
  const int32_t id = c8_page(p, at.s, page);
  RotAngles a;
  if (p.R) a = rot_angles(p, r, at.pos);
  if (slab == 0u && l == 0u) {
    uint32_t bits = id < 0 ? KV_CACHE8_BAD_PAGE : 0u;
    if (p.R && (uint32_t)at.pos >= p.positions) bits |= KV_CACHE8_BAD_POSITION;
    if (bits) c8_error(p, at.s, bits);
  }
  if (id < 0) return;
  const int64_t off = (int64_t)id * p.sb + (int64_t)((uint32_t)at.pos - page * p.T) * p.st;
#pragma unroll
  for (uint32_t i = 0; i < I; ++i) {
    const uint32_t u = first + (i << m.log2);
    if (u < units) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(p.k + off + (int64_t)(u / U) * p.sh);
      if (p.R) rot_row<DT>(r, a, k[i][0], k[i][1]);
      st16(dst + r.c0, k[i][0]);
      st16(dst + r.c1, k[i][1]);
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < 2 * I; ++i) {
    const uint32_t c = vc + (i << m.log2);
    if (c < 2u * units) st16(p.v + off + (int64_t)(c / C) * p.sh + (c % C) * 16u, v[i]);
  }
}

template <int DT, int D>
int append_d(const AppendParams& p, void* stream) {
  Append16 a;
  static_cast<AppendParams&>(a) = p;
  a.kv = row_map(p.n_new, p.H * (D / 16), kIterations);
  a.qm = row_map(p.q ? p.n_new : 0u, p.HQ * (D / 16), kQueries);
  if (a.kv.warps == 0xffffffffu || a.qm.warps == 0xffffffffu) return KV_ERR_INVALID_ARG;
  a.kv_blocks = (a.kv.warps + kWarps - 1u) / kWarps;
  const uint64_t grid = a.kv_blocks + (uint64_t)((a.qm.warps + kWarps - 1u) / kWarps);
  if (grid > 0x7fffffffull) return KV_ERR_INVALID_ARG;
  return dbg_launch(
      stream,
      [&] {
        c16_append_kernel<DT, D><<<(unsigned)grid, kWarps * 32, 0, (cudaStream_t)stream>>>(a);
        return cudaGetLastError();
      },
      a);
}

}  // namespace

int launch_c16_append(const AppendParams& p, void* stream) { KVC_C8_DISPATCH(append_d, p, stream); }

}  // namespace kvc
