"""The products' arithmetic of row runs, on the host: right for every row count below
2^31.  It runs as constant expressions, in which a sum or product that passes its
type is a compile error."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_routing_align_amd", "csrc")

SOURCE = r"""
#include <stdint.h>
#include <initializer_list>
#include "row_runs.h"
using namespace moe;

constexpr int kMax = 0x7fffffff;

constexpr bool ceil_divs() {
  for (int back = 0; back < 600; ++back)
    for (int b : {1, 16, 32, 64, 128, 256}) {
      const int64_t a = (int64_t)kMax - back;
      if (ceil_div((int)a, b) != (a + b - 1) / b) return false;
      if (ceil_div(back, b) != (back + b - 1) / b) return false;
    }
  return true;
}
static_assert(ceil_divs(), "");

// the parts follow each other without a gap, cover the run, and only the last has a ragged end
constexpr bool parts(int count, int splits, int depth) {
  int64_t at = 0;
  for (int s = 0; s < splits; ++s) {
    const RowRange r = split_rows(count, s, splits, depth);
    if (r.begin != at || r.rows < 0) return false;
    at += r.rows;
    if (at < count && r.rows % depth != 0) return false;
  }
  return at == count;
}
static_assert(parts(kMax, 512, 32) && parts(kMax, 1, 32) && parts(kMax, 2, 32) && parts(kMax, 511, 64), "");
static_assert(parts(kMax - 8000, 512, 32) && parts(kMax - 7, 512, 32) && parts(kMax - 16352, 512, 32), "");
static_assert(parts(0, 3, 32) && parts(1, 3, 32) && parts(100, 3, 32) && parts(8192, 32, 32) && parts(70, 512, 32), "");

constexpr bool stages(int rows, int depth) {
  const int n = ceil_div(rows, depth);
  return rows_left(rows, 0, depth) == (rows < depth ? rows : depth) && (n == 0 || rows_left(rows, n - 1, depth) > 0) &&
         rows_left(rows, n, depth) <= 0 && rows_left(rows, n + 2, depth) <= 0;
}
static_assert(stages(kMax, 32) && stages(kMax - 31, 32) && stages(0, 32) && stages(1, 32) && stages(64, 32), "");

static_assert(run_length(0, kMax, kMax) == kMax && run_length(5, kMax, kMax) == kMax - 5 && run_length(kMax - 1, 9, kMax) == 1, "");
static_assert(run_length(-1, 9, 50) == 0 && run_length(50, 9, 50) == 0 && run_length(3, -2, 50) == 0 && run_length(3, 0, 50) == 0, "");
static_assert(run_length(-kMax - 1, kMax, kMax) == 0 && run_length(3, -kMax - 1, kMax) == 0 && run_length(0, 9, 0) == 0, "");
"""


def test_row_arithmetic(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "row_runs_test.cpp"
    src.write_text(SOURCE)
    res = subprocess.run([gxx, "-std=c++17", "-Wall", "-fconstexpr-ops-limit=1000000000", "-fsyntax-only", "-I", CSRC, str(src)],
                         stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout
