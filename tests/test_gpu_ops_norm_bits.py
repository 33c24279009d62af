"""A row of the norm has the same bits in a batch of any size, also where the batch
size picks the kernel's layout (rows of 513 to 1024 columns: a wave per row from 2048
rows on)."""

import pytest
import torch

from moe_testlib import log
from ops_testlib import gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routing_align_amd as m

    return m


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [512, 520, 896, 1000, 1024, 1032])
def test_rows_in_batches_of_any_size(moe, H, res):
    log(f"norm bits H={H} residual={res}")
    M = 2300
    g = gen(H)
    x, w = randn(g, M, H), randn(g, H, scale=0.2) + 1.0
    r = None if res is None else randn(g, M, H, scale=3.0, dtype=res)
    for fp8 in (False, True) if H % 128 == 0 else (False,):
        whole = moe.moe_add_rms_norm(x, w, 1e-6, residual=r, fp8=fp8, save_rstd=True)
        for at, n in ((0, 1), (7, 40), (100, 2047), (253, 2047), (252, 2048)):
            part = slice(at, at + n)
            some = moe.moe_add_rms_norm(x[part].contiguous(), w, 1e-6, residual=None if r is None else r[part].contiguous(),
                                        fp8=fp8, save_rstd=True)
            for name, a, b in zip(("y", "scale", "z", "rstd"), whole, some):
                if b is not None:
                    same = a[part].contiguous().view(torch.uint8) == b.view(torch.uint8)
                    assert bool(same.all()), (name, fp8, at, n, int((~same).sum()))
