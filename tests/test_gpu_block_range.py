"""The block operators where values lie far from one, or leave fp32's range on
the way to a result that does not."""
import pytest
import torch

import block_ref as R
from test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scale", [1e-12, 1e12, 1e14, 1e16])
@pytest.mark.parametrize("n,d,dtype,tokens,shift", [
    (40, 192, "f32", 0, 0), (40, 1024, "bf16", 3, 0), (21, 7168, "f32", 1, 0),
    (9, 16384, "bf16", 0, 0), (33, 1001, "bf16", 8, 1), (600, 64, "f32", 100, 0)])
def test_norm_backward_of_large_and_small_rows(n, d, dtype, tokens, shift, scale):
    """The bounds are relative to the terms, as everywhere: r1 scales with 1 / y,
    and so does dy, however large y is."""
    for both in (False, True):
        c = Case(n, d, dtype, tokens, shift=shift, seed=d)
        c.y.mul_(scale)
        if both:
            c.x.mul_(scale)
        c.forward()
        c.check_forward(c.x, c.y)
        c.backward()
        c.check_backward(c.reference(), c.reference(magnitudes=True))


@pytest.mark.parametrize("eps", [1e-26, 1e-30, 1e-35])
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (2048, "bf16"), (7168, "bf16"), (131, "bf16")])
def test_norm_backward_of_zero_rows_under_a_small_eps(d, dtype, eps):
    """eps^-1/2 is finite, and so are the gradients; eps^-3/2 is not."""
    c = Case(12, d, dtype, 2, seed=4)
    c.cfg.eps = eps
    c.y[3:5] = 0
    c.x[8] = 0
    c.y[8] = 0
    c.forward()
    assert abs(c.r1[3].item() * eps ** 0.5 - 1) < 1e-6
    c.backward()
    for t in (c.dx, c.dy, c.dgate, c.dw_post, c.dw_next):
        assert torch.isfinite(t).all()
    c.check_backward(c.reference(), c.reference(magnitudes=True))


def test_a_block_output_that_is_not_finite_does_not_reach_dy_without_its_norm():
    """Without w_post dy = b g D: y is no part of it."""
    c = Case(6, 96, "f32", 2, post=False, nxt=False, b=0.5, seed=3)
    c.y[2, 5] = float("inf")
    c.y[3, 7] = float("nan")
    c.forward()
    c.backward()
    ref = 0.5 * c.dout.double() * R.gate_of(c.gate, 6, 2)
    assert bool(((c.dy.double() - ref).abs() <= 3 * R.U * ref.abs()).all())
