"""Calls that include/moe_block.h allows beside the usual ones: outputs over inputs,
long gradient lists in a graph, a whole training step in a graph, a backward pass run
twice."""
import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl
from test_gpu_block import gen, make, near
from test_gpu_block_norm import EPS, Case
from test_gpu_grad_clip import reference, tensors

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDTHS = [(256, "bf16"), (1000, "bf16"), (1001, "bf16"), (7168, "bf16"), (4096, "f32"), (9216, "f32")]


@pytest.mark.parametrize("tokens", [0, 1, 8])
@pytest.mark.parametrize("d,dtype", WIDTHS)
def test_out_over_y_and_h_over_x(d, dtype, tokens):
    n = 700
    c = Case(n, d, dtype, tokens, seed=3)
    x, y = c.x.clone(), c.y.clone()
    c.forward()
    want = c.out.clone(), c.h.clone()
    c.x.copy_(x)
    c.y.copy_(y)
    c.forward(out=c.y, h=c.x)
    assert torch.equal(c.y, want[0]) and torch.equal(c.x, want[1])
    c.check_forward(x, y)


@pytest.mark.parametrize("d,dtype", WIDTHS)
def test_pre_norm_in_place(d, dtype):
    n = 700
    c = Case(n, d, dtype, 0, seed=5)
    x, r = c.x.clone(), torch.empty(n, device=DEV)
    h = torch.empty_like(x)
    block.moe_norm_forward(c.cfg, x, c.w_next, h, r)
    block.moe_norm_forward(c.cfg, c.x, c.w_next, c.x, r)
    assert torch.equal(c.x, h)
    want, _ = R.norm(x.double(), c.w_next, 0.0, EPS)
    near(h, want, 2 * R.ROW * want.abs(), R.half_step(c.dt), "h")
    ws = block.norm_workspace(c.cfg, DEV)
    got = []
    for over in (None, "dres", "dh"):
        dres, dh, dw = c.dout.clone(), c.dh.clone(), torch.empty(d, device=DEV)
        dx = {None: torch.empty_like(x), "dres": dres, "dh": dh}[over]
        block.moe_norm_backward(c.cfg, dres, dh, x, c.w_next, r, dx, dw, ws)
        got.append((dx, dw))
    for dx, dw in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dw, got[0][1])


def test_long_lists_in_a_graph():
    """More tensors than the small parameter block holds, and than the large one does."""
    for count in (300, 1203):
        sizes = [13 + 7 * (i % 90) for i in range(count)]
        kinds = [torch.bfloat16, torch.float32]
        g = tensors(sizes, kinds, 7)
        glist = block.grad_list(g, [torch.empty_like(t) for t in g])
        ws, norm = block.grad_workspace(glist, DEV), torch.empty(2, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block.moe_grad_clip(glist, 1.0, norm, ws)
        for seed in (8, 9):
            for t, f in zip(g, tensors(sizes, kinds, seed, 0.5 * seed)):
                t.copy_(f)
            graph.replay()
            torch.cuda.synchronize()
            want = reference(g)
            assert abs(norm[0].item() - want) <= 10 * R.U * want
            f = 1.0 / (want + 1e-6)
            for t, o in zip(g, glist.outs):
                w = t.double() * f
                assert bool(((o.double() - w).abs() <=
                             (R.half_step(t.dtype) + 14 * R.U) * w.abs() + 1e-38).all())
        del graph


@pytest.mark.parametrize("w", [wl.EC_FP32, wl.SMALL[3]], ids=lambda w: w.name)
def test_train_step_in_a_graph(w):
    """Forward, backward and clip captured once and replayed on other inputs, beside
    the same calls one after another; and a second backward pass of one forward."""
    b, p, x, dout, dh = make(w, tokens=1)

    def results(g, norm):
        own = [g[k] for k in ("dx", "dy", "dw_pre", "dw_post", "dgate", "dw_next")]
        return [t.clone() for t in [b.out, b.h_next, norm] + own +
                [t for k, t in g["layer"].items() if t is not None and k != "dL"]]

    def step():
        b.forward_train(x)
        g = b.backward_train(dout, dh)
        return g, b.clip_grads(0.5)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, norm = step()
    for seed in (31, 32):
        for t in (x, dout, dh):
            t.copy_(torch.randn(t.shape, generator=gen(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = results(g, norm)
        want = results(*step())
        assert all(torch.equal(s, t) for s, t in zip(got, want))
        b.forward_train(x)
        once = results(b.backward_train(dout, dh), norm)
        again = results(b.backward_train(dout, dh), norm)
        assert all(torch.equal(s, t) for s, t in zip(once, again))
    assert moe.moe_read_error(b.layer._bws) == (moe.MOE_OK, 0)
    del graph
