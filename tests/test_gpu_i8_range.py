"""8-bit products whose scales lie far from one: the two scales' product may
leave fp32's range where the result does not."""
import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import moe
from test_gpu_i8 import Gemm

pytestmark = pytest.mark.gpu

# rows, k, channels: the tile kernels, then K split in four and in two
SHAPES = [(300, 1024, 272), (70, 2048, 272), (3, 4096, 4112)]


def wide(rows, k, o, act, dtype, xs, ws, s3, seed):
    """Sums of one sign, so that none of them is small."""
    c = Gemm(rows, k, o, act, dtype, seed=seed)
    c.x.copy_(c.x.abs().clamp(min=64))
    c.w.copy_(c.w.abs().clamp(min=64))
    c.xs.mul_(xs)
    c.ws.copy_(c.ws / c.ws.max() * ws)
    if act == "swiglu":
        c.w3.copy_(c.w3.abs().clamp(min=64))
        c.s3.copy_(c.s3 / c.s3.max() * s3)
    return c


def products(c):
    x, xs = c.x.double(), c.xs.double()[:, None]
    u = (x @ c.w[0].double().T) * xs * c.ws[0].double()
    v = None if c.w3 is None else (x @ c.w3[0].double().T) * xs * c.s3[0].double()
    return u, v


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,o", SHAPES)
def test_scales_whose_product_underflows(rows, k, o, dtype, act):
    # u about 1e-37 to 1e-34, from scales of 1e-24 and 1e-18; v about 10 and more
    c = wide(rows, k, o, act, dtype, 1e-24, 1e-18, 1e20, rows + k)
    c.run()
    u, v = products(c)
    want = R.act(c.act, u, v)
    assert want.abs().min() > 2 ** -126  # all of them are normal numbers
    # the sum, two products; the activation is u / 2 (1 + 1e-34), a product or two
    # (and a reciprocal) more, and v's three; then the output's rounding
    tol = (R.half_step(c.dt) + 10 * R.U) * want.abs()
    off = (c.out.double() - want).abs() - tol
    assert bool((off <= 0).all()), (off.max().item(), want.abs().max().item())
    assert moe.moe_read_error(c.space) == (moe.MOE_OK, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,o", SHAPES)
def test_scales_whose_product_overflows(rows, k, o, dtype):
    """Scales of 1e25 and 1e18: a sum of zero is zero."""
    c = wide(rows, k, o, "none", dtype, 1e25, 1e18, 0, rows + k)
    c.x.zero_()
    c.run()
    assert not c.out.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,o", SHAPES)
def test_silu_of_large_negative_sums(rows, k, o, dtype):
    """silu(u) = u e^u / (1 + e^u) from u = -80 down to -100 is 1e-33 to 1e-42,
    and counts where v is large."""
    c = wide(rows, k, o, "swiglu", dtype, 1.0, 1.0, 1.0, rows + k)
    c.w.neg_()
    c.xs.fill_(1.0)
    total = (c.x.double() @ c.w[0].double().T)[0]  # row 0's sums set the channels' scales
    c.x.copy_(c.x[:1].expand_as(c.x))
    c.ws.copy_((torch.linspace(-80, -100, o, device="cuda", dtype=torch.float64) / total)[None])
    c.s3.fill_(1e25)
    c.run()
    u, v = products(c)
    # e^u with u rounded three times and e^x's own error relative to |u| (see
    # Gemm.check); below 2^-126 a value keeps steps of 2^-149, some of them
    # (e^u, u e^u) before v multiplies them
    want = R.act("swiglu", u, v)
    tol = R.half_step(c.dt) * want.abs() + (20 + 5 * u.abs()) * R.U * want.abs() + \
        (u.abs() + 2) * 2.0 ** -149 * v.abs()
    off = (c.out.double() - want).abs() - tol
    assert bool((off <= 0).all()), (off.max().item(), want.abs().max().item())
    assert bool((c.out[:, u[0] > -87] != 0).all())
