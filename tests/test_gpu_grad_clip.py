"""Gradient norm and clip on the GPU against float64."""
import math

import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def tensors(sizes, dtypes, seed, scale=1.0, shift=0):
    g = gen(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (scale * torch.randn(n + shift, generator=g, device=DEV)).to(dtypes[i % len(dtypes)])
        out.append(t[shift:])
    return out


def reference(grads):
    total = 0.0
    for t in grads:
        total += float((t.double() ** 2).sum())
    return math.sqrt(total)


def check(grads, max_norm, outs=None):
    raw = [t.clone() for t in grads]
    want = reference(raw)
    glist = block.grad_list(grads, outs)
    ws = block.grad_workspace(glist, DEV)
    ws.fill_(0xff)
    norm = torch.full((2,), -1.0, device=DEV)
    block.moe_grad_norm(glist, norm, ws)
    only = norm[0].item()
    block.moe_grad_clip(glist, max_norm, norm, ws)
    got, factor = norm.tolist()
    assert got == only  # the same sums in both calls
    # eight squares in a chain of fp32, the rest in fp64, one rounding of the root
    assert abs(got - want) <= 10 * R.U * want
    f = min(1.0, max_norm / (want + 1e-6))
    assert abs(factor - f) <= 12 * R.U * f
    for r, o in zip(raw, grads if outs is None else outs):
        w = r.double() * f
        tol = (R.half_step(r.dtype) + 14 * R.U) * w.abs() + torch.finfo(r.dtype).smallest_normal
        assert bool(((o.double() - w).abs() <= tol).all())
    if outs is not None:
        for r, t in zip(raw, grads):
            assert torch.equal(r, t)
    return factor


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("sizes,dtypes", [
    ([1], [F32]), ([1], [BF]), ([7, 1, 3], [BF, F32]), ([8192], [BF]), ([8193, 8191], [F32]),
    ([0, 5, 0, 0, 9, 0], [BF]), ([100_003, 17, 65_536], [BF, F32]), ([3_000_001], [BF]),
    ([13 + 7 * i for i in range(300)], [BF, F32, BF]), ([5] * 1203, [F32, BF]),
    ([0] * 130, [BF]), ([16_384 * 900], [F32])])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_sizes(sizes, dtypes, max_norm):
    g = tensors(sizes, dtypes, 1)
    check(g, max_norm, [torch.full_like(t, 9) for t in g])
    check(g, max_norm)  # in place


@pytest.mark.parametrize("shift,other", [(1, 1), (3, 3), (1, 2), (0, 5)])
def test_views_at_any_element(shift, other):
    for dt in (BF, F32):
        g = tensors([1000, 30_011, 4], [dt], 2, shift=shift)
        check(g, 0.25, tensors([1000, 30_011, 4], [dt], 3, shift=other))
        check(g, 0.25)


def test_neighbours_in_one_buffer():
    flat = torch.randn(50_000, generator=gen(4), device=DEV).to(BF)
    sizes = [129 * 33, 1, 7, 20_001, 50_000 - 129 * 33 - 8 - 20_001]
    check(list(flat.split(sizes)), 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
def test_squares_that_leave_fp32(dt, scale):
    g = tensors([5000, 77], [dt], 5, scale)
    raw = [t.clone() for t in g]
    want = reference(raw)
    glist = block.grad_list(g, [torch.empty_like(t) for t in g])
    norm = torch.empty(2, device=DEV)
    block.moe_grad_clip(glist, 1.0, norm, block.grad_workspace(glist, DEV))
    assert abs(norm[0].item() - want) <= 10 * R.U * want
    f = min(1.0, 1.0 / (want + 1e-6))
    assert abs(norm[1].item() - f) <= 4 * R.U * f


def test_mixed_magnitudes():
    t = torch.tensor([3e-23, 4e-23, 0, 0, 0, 0, 0, 0] + [0.0] * 64, device=DEV)
    norm = torch.empty(1, device=DEV)
    glist = block.grad_list([t])
    block.moe_grad_norm(glist, norm, block.grad_workspace(glist, DEV))
    assert abs(norm.item() - 5e-23) <= 4 * R.U * 5e-23


def test_not_finite():
    for dt in (BF, F32):
        for bad, want in ((float("inf"), math.inf), (float("nan"), math.nan)):
            for at in (0, 3, 4999):
                g = tensors([5000, 8], [dt], 6)
                g[0][at] = bad
                raw = [t.clone() for t in g]
                glist = block.grad_list(g)
                norm = torch.empty(2, device=DEV)
                block.moe_grad_clip(glist, 1.0, norm, block.grad_workspace(glist, DEV))
                n, f = norm.tolist()
                assert n == want or (math.isnan(n) and math.isnan(want))
                assert math.isnan(f) if math.isnan(want) else f == 0.0
                for r, t in zip(raw, g):
                    assert torch.equal(torch.isnan(t), torch.isnan(r.double() * f))


def test_nothing_to_clip():
    norm = torch.full((2,), 9.0, device=DEV)
    for g in ([], [torch.empty(0, device=DEV)]):
        glist = block.grad_list(g)
        ws = block.grad_workspace(glist, DEV)
        block.moe_grad_clip(glist, 1.0, norm, ws)
        assert norm.tolist() == [0.0, 1.0]
        block.moe_grad_clip(glist, 0.0, norm, ws)
        assert norm.tolist() == [0.0, 0.0]
    zero = [torch.zeros(100, device=DEV)]
    glist = block.grad_list(zero)
    block.moe_grad_clip(glist, 1.0, norm, block.grad_workspace(glist, DEV))
    assert norm.tolist() == [0.0, 1.0] and not zero[0].any()


def test_captured_on_a_stream():
    g = tensors([100_000, 33], [BF, F32], 7)
    outs = [torch.empty_like(t) for t in g]
    glist = block.grad_list(g, outs)
    ws, norm = block.grad_workspace(glist, DEV), torch.empty(2, device=DEV)
    block.moe_grad_clip(glist, 1.0, norm, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.moe_grad_clip(glist, 1.0, norm, ws)
    for seed in (8, 9):
        for t, f in zip(g, tensors([100_000, 33], [BF, F32], seed, 0.5 * seed)):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = reference(g)
        assert abs(norm[0].item() - want) <= 10 * R.U * want
        f = 1.0 / (want + 1e-6)
        for t, o in zip(g, outs):
            w = t.double() * f
            assert bool(((o.double() - w).abs() <=
                         (R.half_step(t.dtype) + 14 * R.U) * w.abs() + 1e-38).all())
    del graph
