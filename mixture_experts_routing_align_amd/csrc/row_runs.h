// Arithmetic of row runs and their tiles for any row count below 2^31: no sum or product
// on the way passes an int.  Plain constexpr functions, for kernels and host alike.
#pragma once

#include <stdint.h>

namespace moe {

// a >= 0, b > 0: the sum stays below 2^32
constexpr int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// Length of the run of `cnt` rows from row `off` on, cut off at `rows`; a negative or
// far offset leaves an empty run.
constexpr int run_length(int off, int cnt, int rows) {
  if (off < 0 || off >= rows || cnt <= 0) return 0;
  return cnt < rows - off ? cnt : rows - off;
}

// Row tiles all runs can need: one partly filled tile per expert on top of the full ones.
constexpr int64_t row_tiles_bound(int64_t rows, int E, bool dense, int bq) {
  return dense ? (rows + bq - 1) / bq : rows / bq + (E < rows ? E : rows);
}

// Part `split` of `splits` of a run of `count` rows: equal parts, in whole stages of
// `depth` rows; the last ones may be shorter or empty.
struct RowRange {
  int begin, rows;
};
constexpr RowRange split_rows(int count, int split, int splits, int depth) {
  const int64_t share = (int64_t)ceil_div(ceil_div(count, splits), depth) * depth;
  const int64_t begin = share * split < count ? share * split : count;
  return RowRange{(int)begin, (int)(share < count - begin ? share : count - begin)};
}

// Rows left of `rows` from stage s of `depth` rows on, no more than a stage.
constexpr int rows_left(int rows, int s, int depth) {
  const int64_t left = rows - (int64_t)s * depth;
  return left < depth ? (int)left : depth;
}

}  // namespace moe
