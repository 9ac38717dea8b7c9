"""Buffers of more than 2^31 elements: the block operators' offsets are 64-bit.
Only the rows at both ends are compared."""
import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block, moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def randn(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(shape, dtype=BF, device=DEV)
    for part in t.split(1 << 16):  # (fp32 draws of a slice at a time)
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    return t


def near(got, want, mag):
    assert bool(((got.double() - want).abs() <=
                 R.half_step(got.dtype) * want.abs() + 3 * R.ROW * mag + 1e-30).all())


def test_residual_norm():
    n, d = 270_000, 8192
    assert n * d > 1 << 31
    x, y = randn(n, d, seed=1), randn(n, d, seed=2)
    w = torch.ones(d, device=DEV)
    cfg = block.norm_config(n, d, BF, 1e-6)
    out, h = torch.empty_like(x), torch.empty_like(x)
    r1, r2 = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    block.moe_residual_norm_forward(cfg, x, y, w, None, w, out, h, r1, r2)
    ends = torch.tensor([0, 1, n - 2, n - 1], device=DEV)
    want = R.residual_norm(x[ends].double(), y[ends].double(), w, None, w, eps=1e-6)
    mag = x[ends].double().abs() + (want[0] - x[ends].double()).abs()
    near(out[ends], want[0], mag)
    near(h[ends], want[1], mag + want[1].abs())
    # backward, dx and dy over the gradients that came in
    ws = block.norm_workspace(cfg, DEV)
    dw1, dw2 = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ins = [t[ends].double() for t in (x, h, out, y)]
    block.moe_residual_norm_backward(cfg, x, h, out, y, w, None, w, r1, r2, x, h, dw1, None, dw2,
                                     ws)
    args = (*ins, w, None, w, r1[ends].double(), r2[ends].double())
    ref = R.residual_norm_backward(*args)
    big = R.residual_norm_backward(*args, magnitudes=True)
    near(x[ends], ref[0], big[0])
    near(h[ends], ref[1], big[1])
    assert torch.isfinite(dw1).all() and torch.isfinite(dw2).all()


def test_clip():
    g = randn(34_000, 1 << 16, seed=3)
    assert g.numel() > 1 << 31
    glist = block.grad_list([g])
    norm = torch.empty(2, device=DEV)
    total = sum(float((p.double() ** 2).sum()) for p in g.split(1024)) ** 0.5
    ends = [(g[i].clone(), i) for i in (0, 33_999)]
    block.moe_grad_clip(glist, 1.0, norm, block.grad_workspace(glist, DEV))
    assert abs(norm[0].item() - total) <= 10 * R.U * total
    for before, i in ends:
        near(g[i], before.double() / (total + 1e-6), before.double().abs() / total)


def test_quantize_and_product():
    rows, k, o = 300_000, 8192, 8192
    assert rows * k > 1 << 31
    x = randn(rows, k, seed=4)
    q, s = torch.empty((rows, k), dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    block.moe_quantize_rows(x, q, s)
    ends = torch.tensor([0, 255, rows - 300, rows - 1], device=DEV)
    ws, wq = R.quantize(x[ends])
    assert torch.equal(q[ends].double(), wq) and torch.equal(s[ends].double(), ws)
    del x
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.randint(-127, 128, (1, o, k), generator=g, device=DEV, dtype=torch.int8)
    wsc = torch.rand((1, o), generator=g, device=DEV)
    cfg = block.gemm_i8_config(1, rows, k, o)
    out, sp = torch.empty((rows, o), dtype=BF, device=DEV), block.gemm_i8_workspace(cfg, DEV)
    block.moe_gemm_i8(cfg, q, s, None, None, w, wsc, None, None, out, sp)
    ref = (wq @ w[0].double().T) * ws[:, None] * wsc.double()
    got = out[ends].double()
    assert bool(((got - ref).abs() <= (2 ** -8 + 4 * R.U) * ref.abs() + 1e-30).all())
    assert moe.moe_read_error(sp) == (moe.MOE_OK, 0)
