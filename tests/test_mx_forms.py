"""Which form the products on MXFP4 weights take, on the host: the cases of the GPU tests take
the forms they are named for, and between them every form that is built."""

import os
import shutil
import subprocess

import pytest

import mixture_experts_routing_align_amd as moe
from mx_forms_cases import BACKWARD, DEPTHS, FORWARD

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_routing_align_amd", "csrc")

SOURCE = r"""
#include <stdio.h>
#include "mx_forms.h"
using namespace moe::mx;
int main() {
  long long kind, rows, E, dense, N, K, parts, out;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &kind, &rows, &E, &dense, &N, &K, &parts, &out) == 8) {
    const Sizes a{rows, (int)E, dense != 0, (int)N, (int)K, (int)parts, out != 0};
    const Form f = kind == 0 ? rows16_form(a) : kind == 1 ? rows4_form(a) : back_form(a);
    const char* const names[] = {"split16", "split32", "split32by2", "32x64", "32x128", "64x64", "64x128", "128x128", "256x256"};
    puts(names[(int)f]);
  }
}
"""


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """The forms of a list of (kind, rows, N, K, parts, MXFP4 rows out)."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("forms")
    (at / "forms.cpp").write_text(SOURCE)
    res = subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "forms.cpp"), "-o", str(at / "forms")],
                         stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout

    def ask(calls):
        lines = []
        for kind, rows, N, K, parts, out in calls:
            M, E, k, BS = (rows, 1, 1, 1) if isinstance(rows, int) else rows[:4]
            total = rows if isinstance(rows, int) else moe.moe_align_max_total(M * k, E, BS)
            lines.append(f"{kind} {total} {E} {int(isinstance(rows, int))} {N} {K} {parts} {int(out)}")
        out = subprocess.run([str(at / "forms")], input="\n".join(lines), stdout=subprocess.PIPE, text=True, check=True).stdout.split()
        assert len(out) == len(calls)
        return out

    return ask


def test_forward_forms(forms):
    calls, named = [], []
    for form, rows, N, which in FORWARD:
        for kind in (0, 1):
            if which not in ("both", "bf16" if kind == 0 else "mxfp4"):
                continue
            for K in DEPTHS:
                for parts in (1, 2):
                    for out in (False, True):
                        calls.append((kind, rows, N, K, parts, out))
                        named.append(("split32" if out else "split16") if form == "split" else form)
    got = forms(calls)
    wrong = [(c, n, g) for c, n, g in zip(calls, named, got) if n != g]
    assert not wrong, wrong
    # everything that is built runs: each form with one and two weights, staged ones at aligned and other depths
    ran = {(c[0], g, c[4], None if "split" in g else c[3] % 128 == 0) for c, g in zip(calls, got)}
    staged = {0: ("32x64", "32x128", "64x64", "128x128", "256x256"), 1: ("32x128", "64x128", "128x128", "256x256")}
    want = {(kind, f, parts, aligned) for kind in (0, 1) for f in staged[kind] for parts in (1, 2) for aligned in (True, False)}
    want |= {(kind, f, parts, None) for kind in (0, 1) for f in ("split16", "split32", "split32by2") for parts in (1, 2)}
    assert ran == want, (want - ran, ran - want)


def test_backward_forms(forms):
    calls = [(2, rows, N, K, parts, False) for _, rows, N, K in BACKWARD for parts in (1, 2)]
    got = forms(calls)
    assert got == [f for f, *_ in BACKWARD for _ in (1, 2)], got
    assert set(got) == {"32x128", "64x128", "128x128", "256x256"}
