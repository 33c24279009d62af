// Which form of the products on MXFP4 weights a call takes: rules on its sizes alone.  The
// runs themselves are known on the device only.  Plain constexpr functions, for launches and
// host alike.
#pragma once

#include <stdint.h>

#include "row_runs.h"

namespace moe {
namespace mx {

enum class Form {
  kSplit16, kSplit32, kSplit32By2,                   // depth split over waves: 16 rows by 16 or 32 columns
  k32x64, k32x128, k64x64, k64x128, k128x128, k256x256,  // staged tiles: rows by weight rows (SwiGLU: of both weights)
};

struct Sizes {
  int64_t rows;
  int E;
  bool dense;      // one expert that holds every row
  int N, K, parts; // parts: 2 for two weights
  bool rows4_out;  // MXFP4 rows out, whose blocks hold 32 columns
};

// Rows per expert on average, of the matrix's height, in which the alignment's padding
// counts: runs far below the block size can get tiles that are too large.  SwiGLU of 2 x 768 x
// 2048 over 128 experts, 16 and 32 tokens top-8 aligned to 16 rows and to 64 (128-row tiles):
// bf16 rows 49 and 61 us, 59 and 80; MXFP4 rows 31 and 35, 39 and 47; the gradient 51 and 75,
// 70 and 100.
constexpr int64_t mean_rows(const Sizes& a) { return (a.rows + a.E - 1) / a.E; }

// Square tiles of `edge` that the rows and `cols` columns make.
constexpr int64_t tiles(const Sizes& a, int64_t cols, int64_t edge) {
  return (a.rows + edge - 1) / edge * ((cols + edge - 1) / edge);
}

// The depth-split form: few tiles in all (of 16 rows and 32 columns), which the staged forms
// walk one memory trip after another.  Dense rows of bf16 by 2048 x 2048: 16 rows 8.6 us,
// 12.9 in 32 x 64 tiles; 64 rows 9.1 and 13.0; 256 rows 24.5 and 13.8; 16 rows by 8192 x
// 7168 25 and 36 (MXFP4 rows: 15 and 15).  Over many experts it is the slower one, 64 rows on
// 51 of 128, SwiGLU of 2 x 768 x 2048: 33 us, 30 in 32 x 128 tiles (MXFP4 rows: 28 and 19).
constexpr int64_t split_tiles(const Sizes& a) { return row_tiles_bound(a.rows, a.E, a.dense, 16) * (((int64_t)a.N + 31) / 32); }
constexpr bool few_tiles(const Sizes& a) {
  const int64_t mean = mean_rows(a);
  return split_tiles(a) <= (mean <= 32 ? 1024 : mean <= 64 ? 256 : 0);
}

// 8 waves along the depth while its tiles are fewer than 512, of half the columns where the
// result allows it (8 dense rows, 2048 x 7168: 10 us, 16 on 32 columns); else 2 (16384
// columns: 30 us, 31 with 8).
constexpr Form split_form(const Sizes& a) {
  if (split_tiles(a) >= 512) return Form::kSplit32By2;
  return a.rows4_out ? Form::kSplit32 : Form::kSplit16;
}

// 256-wide tiles read each operand byte half as often as 128-wide ones and are four times the
// work: taken where they fill the GPU and the runs fill most of them.  SwiGLU of 2 x 768 x
// 2048 over 128 experts, rows an expert on average, 256- and 128-wide tiles, us:
//                        96          128          256       16384 rows, 16 experts, 2 x 2048 x 7168
//   MXFP4 rows        77   73      83   83     113   123       303   354
//   bf16 rows        138  135     152  158     222   242       766   913
//   their gradient   163  163     176  187     267   301       837  1121
constexpr int kWideRuns = 120;
constexpr bool wide_tiles(const Sizes& a, int64_t cols) { return tiles(a, cols, 256) >= 256 && mean_rows(a) >= kWideRuns; }

// Rows per expert on average up to which tiles have 32 rows: SwiGLU of 2 x 768 x 2048 over
// 128 experts, MXFP4 rows, in 32 x 128 and 128 x 128 tiles: 8 rows an expert 42 and 50 us,
// 24 52 and 56, 48 64 and 62 (bf16 rows: 61 and 82, 83 and 91, 111 and 110).  Over few experts
// it is not as good a rule: 40 and 41 dense rows by 4096 x 4096 take 32 and 23 us with bf16
// rows, 10 and 13 with MXFP4 ones.
constexpr int64_t kShortRuns = 40;

constexpr Form rows4_form(const Sizes& a) {
  if (few_tiles(a)) return split_form(a);
  const int64_t cols = a.parts * (int64_t)a.N;
  if (wide_tiles(a, cols)) return Form::k256x256;
  if (mean_rows(a) <= kShortRuns) return Form::k32x128;
  // few 128-wide tiles: smaller ones (1024 dense rows by 4096 x 2048: 13.1 us, 14.8; 2048 x
  // 2048: 12.8 and 14.7; in 64 x 64 16.7)
  return tiles(a, cols, 128) < 256 ? Form::k64x128 : Form::k128x128;
}

constexpr Form rows16_form(const Sizes& a) {
  if (few_tiles(a)) return split_form(a);
  const int64_t cols = a.parts * (int64_t)a.N;
  if (wide_tiles(a, cols)) return Form::k256x256;
  if (mean_rows(a) <= kShortRuns) return Form::k32x128;
  // few tiles: smaller ones, of which more than one shares a compute unit (dense rows by 2048 x
  // 2048, in 32 x 64, 64 x 64 and 128 x 128: 256 rows 13.8, 16.5 and 28.5 us; 512 15.2, 16.8 and
  // 26; 2048 35, 26 and 28)
  if (tiles(a, cols, 128) >= 256) return Form::k128x128;
  return tiles(a, cols, 64) <= 256 ? Form::k32x64 : Form::k64x64;
}

// The rows' gradient, [rows, K].
constexpr Form back_form(const Sizes& a) {
  if (wide_tiles(a, a.K)) return Form::k256x256;
  // 2 x 768 x 2048, 16 rows an expert: 85 us, 109 in 128 x 128 tiles; 48 rows 130 and 128
  if (mean_rows(a) <= kShortRuns) return Form::k32x128;
  // few tiles: 64 rows on each of 8 experts 20 us, 25; 1024 dense rows by 2 x 2048 x 2048 43, 54
  return tiles(a, a.K, 128) < 256 ? Form::k64x128 : Form::k128x128;
}

}  // namespace mx
}  // namespace moe
