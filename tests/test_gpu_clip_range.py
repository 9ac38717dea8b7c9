"""The clip where the norm passes fp32's range, and with no limit."""
import math

import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block

pytestmark = pytest.mark.gpu
DEV = "cuda"


def clip(grads, max_norm, outs=None):
    glist = block.grad_list(grads, outs)
    norm = torch.full((2,), -1.0, device=DEV)
    block.moe_grad_clip(glist, max_norm, norm, block.grad_workspace(glist, DEV))
    return norm.tolist()


@pytest.mark.parametrize("count", [2, 130])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_factor_is_of_the_norm_that_is_returned(dt, count):
    """Finite gradients whose norm is above the largest fp32: the norm is +inf,
    and the factor max_norm / (inf + 1e-6) = 0."""
    for in_place in (False, True):
        g = [torch.full((33,), 3e38, device=DEV).to(dt) for _ in range(count)]
        outs = g if in_place else [torch.full_like(t, 7.0) for t in g]
        norm, factor = clip(g, 1.0, None if in_place else outs)
        assert norm == math.inf and factor == 0.0
        assert all(not t.any() for t in outs)


def test_the_largest_norm_that_fits():
    g = [torch.full((4,), 1.5e38, device=DEV)]
    norm, factor = clip(g, 3.0)
    assert abs(norm - 3e38) <= 4 * R.U * 3e38 and abs(factor - 1e-38) <= 4 * R.U * 1e-38
    assert bool(((g[0].double() - 1.5).abs() <= 8 * R.U * 1.5).all())


@pytest.mark.parametrize("value", [1.0, 3e38, math.inf])
def test_no_limit_changes_nothing(value):
    g = [torch.full((100,), value, device=DEV)]
    out = [torch.zeros(100, device=DEV)]
    norm, factor = clip(g, math.inf, out)
    assert norm == (10.0 if value == 1.0 else math.inf) and factor == 1.0
    assert torch.equal(out[0], g[0])
