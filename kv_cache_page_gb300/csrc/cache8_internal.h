// cache8_internal.h -- launch parameters of the live 8-bit KV cache, and of the
// live 16-bit cache that shares its batches and rows; for the host library and
// the kernels.
#pragma once
#include <stdint.h>

#include "kv_cache8.h"

namespace kvc {

constexpr uint32_t kC8Sms = 152;  // SMs of a GB300: what the split rules count on

// Row tiles of the attention: consecutive (token, query head of the group)
// pairs r = i * G + g of one sequence and KV head.
constexpr uint32_t kStepRows = 16;
constexpr uint32_t kMaxSplits = 256;  // ranges of a row tile's keys (the joining CTA holds 8 bytes a range and row)
constexpr uint32_t kPromptRows = 256;
// Row tiles (times KV heads) whose keys may be split, of one call.  Their tickets take this much of every
// workspace whatever the batch, so that what a call leaves behind them is never another call's ticket.
constexpr uint32_t kTickets = 4096;
constexpr uint32_t kC16Ctas = 2u * kC8Sms;  // CTAs of 16-bit attention at most: two an SM

struct C8Params {
  // ---- registered geometry ----
  uint32_t dtype, D, H, HQ, G, T;
  uint32_t t_magic, t_shift;    // n / T = (umulhi(t_magic, n) + n) >> t_shift, n < 2^31
  uint32_t num_blocks;
  int64_t sb, st, sh;           // code strides, bytes
  int64_t st2, stv;             // 2 tokens; the token rows that a warp's 16-byte copies cover (512 / D)
  // ---- layer ----
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  // ---- batch ----
  uint32_t n_seqs, n_new, table_width;
  int64_t table_stride;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* cu;            // NULL: one new token per sequence
  uint32_t* errors;             // may be NULL
  // ---- 16-bit rows: write k, v; read k, v; attend q, out ----
  uint16_t* a;
  uint16_t* b;
  int64_t a_row, a_head, b_row, b_head;
  // ---- attend ----
  float* lse;                   // may be NULL
  float scale_log2;             // softmax scale * log2(e)
  uint32_t window;              // 0: none
  uint32_t causal;
  uint32_t splits;              // ranges a row tile's keys are split into, at most
  uint32_t step_warps;          // warps of a step CTA: 4, or as many as an SM holds (12; 8 for D = 256)
  uint32_t chunk;               // keys of a range (more where splits ranges of it do not reach)
  uint32_t min_rows, max_rows;  // sequences this launch serves: G * new within [min_rows, max_rows]
  uint32_t rows8;               // step: every row tile has at most 8 rows
  uint32_t both_roles;          // write, read: a warp takes K and V of its page and head
  uint32_t per_seq;             // step: units of a sequence, 0: by cu_new
  uint32_t n_units;             // row tiles (step, prompt) or page units (write, read), an upper bound
  uint32_t* tickets;            // [kTickets], of which [n_units][H] are used; 0 between calls
  float* partials;              // [n_units][H][splits][kStepRows][D + 2]
};

// Appending with the position rotation, to 8-bit and (k, v: 16-bit pages, strides in bytes) 16-bit pages.
struct AppendParams : C8Params {
  const float* cos;             // [positions][R / 2]
  const float* sin;
  int64_t rot_stride;           // floats between positions
  uint32_t R;                   // channels turned, a multiple of 16; 0: none
  uint32_t positions;
  uint32_t neighbours;          // pairs (2 i, 2 i + 1), else (i, i + R / 2)
  const uint16_t* q;            // may be NULL, or q_out itself
  uint16_t* q_out;
  int64_t q_row, q_head, q_out_row, q_out_head;
};

// Attention over 16-bit pages (strides in bytes, scales NULL).
struct C16Params : C8Params {
  uint32_t tile_rows;           // rows of a tile: 8 where one token's query heads fit, else 16
  uint32_t even;                // the jobs may be few enough to split each into even parts
  uint32_t g_magic, g_shift;    // n / G = (umulhi(g_magic, n) + n) >> g_shift, n < 2^31
};

int launch_c8_append(const AppendParams& p, void* stream);
int launch_c16_append(const AppendParams& p, void* stream);
int launch_c16_attend(const C16Params& p, uint64_t jobs, uint64_t keys, void* stream);  // at most so many
int launch_c8_write(const C8Params& p, void* stream);
int launch_c8_read(const C8Params& p, void* stream);
int launch_c8_step(const C8Params& p, void* stream);
int launch_c8_prompt(const C8Params& p, void* stream);

}  // namespace kvc
