"""8-bit rows out of every form of the products: the tiles with two scale blocks (a block's
maximum shared by two waves, the last tile half filled), those with one, and the
depth-split kernel, for bf16 and 8-bit operands."""

import pytest
import torch

import test_gpu_ops_linear as linear

pytestmark = pytest.mark.gpu

moe = linear.moe
SKEW = (1500, 16, 4, 16, "skew", 0.0)  # 6000 slots, runs of every length
FEW = (60, 8, 2, 16, "random", 0.0)


# 256 x 256 tiles without SwiGLU: at least 256 of them, rows of 160 and more an expert;
# 4224 columns are 16 tiles and a half
@pytest.mark.parametrize("rows,N,K", [(4100, 4224, 136), (SKEW, 4224, 72), (1100, 2176, 264), (40, 1152, 520), (FEW, 384, 136)],
                         ids=str)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_bf16_operands(moe, rows, N, K, act):
    linear.test_bf16_operands_to_8bit_rows(moe, rows, act, N, K)


@pytest.mark.parametrize("rows,N,K", [(1100, 1024, 256), (2100, 2176, 128), (SKEW, 1152, 384), (40, 1152, 512), (FEW, 384, 128)],
                         ids=str)
@pytest.mark.parametrize("act,bias,res", [("none", False, True), ("gelu", True, True), ("swiglu", True, True)])
def test_8bit_operands(moe, rows, N, K, act, bias, res):
    linear.test_forward_8bit(moe, rows, act, bias, res, True, N, K)
