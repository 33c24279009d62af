"""Every form of the products on MXFP4 weights, with all of the epilogue and partly filled
tiles on both sides (which form a case takes is held to the rules by test_mx_forms.py)."""

import pytest

from mx_forms_cases import BACKWARD, DEPTHS, FORWARD
from test_gpu_ops_mxfp4 import backward_case, forward_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.mark.parametrize("form,rows,N,rows4", [(f, r, n, q) for f, r, n, which in FORWARD for q in (False, True)
                                               if which in ("both", "mxfp4" if q else "bf16")], ids=str)
@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("out4", [False, True])
def test_forward(moe, form, rows, N, rows4, K, act, out4):
    forward_case(moe, rows, act, True, True, True, rows4, out4, N, K)


@pytest.mark.parametrize("form,rows,N,K", BACKWARD, ids=str)
@pytest.mark.parametrize("gated", [False, True])
def test_backward_x(moe, form, rows, N, K, gated):
    backward_case(moe, rows, gated, N, K)
