"""Blocks in a row: the first one's fused next pre-norm is the second one's input."""
import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl
from test_gpu_block import gen, near

pytestmark = pytest.mark.gpu
DEV = "cuda"


def chain(w, kind=moe.Layer):
    """Two blocks that hand h over, and two that each norm their own input."""
    g = gen(5)
    f = lambda: 1 + 0.1 * torch.randn(w.d, generator=g, device=DEV)  # noqa: E731
    first, second = {"w_pre": f(), "w_post": f()}, {"w_post": f()}
    w_mid = f()
    inp = [wl.make_inputs(w.replace(seed=s), DEV) for s in (1, 2)]
    one = block.Block(kind(w, inp[0], DEV), {**first, "w_next": w_mid}, eps=1e-5)
    two = block.Block(kind(w, inp[1], DEV), second, eps=1e-5)
    one_own = block.Block(kind(w, inp[0], DEV), first, eps=1e-5)
    two_own = block.Block(kind(w, inp[1], DEV), {**second, "w_pre": w_mid}, eps=1e-5)
    x = torch.randn((w.n, w.d), generator=g, device=DEV).to(w.torch_dtype)
    dout = torch.randn((w.n, w.d), generator=g, device=DEV).to(w.torch_dtype)
    return one, two, one_own, two_own, x, dout


@pytest.mark.parametrize("w", [wl.EC_FP32, wl.SMALL[3]], ids=lambda w: w.name)
def test_two_blocks_train_with_one_norm_between_them(w):
    one, two, one_own, two_own, x, dout = chain(w)
    mid, h = one.forward_train(x)
    out, none = two.forward_train(mid, h=h)
    assert none is None
    g2 = {k: t for k, t in two.backward_train(dout).items()}
    g1 = one.backward_train(g2["dx"], g2["dh"])
    # the second block: its layer's gradient is dh, the residual's dx
    layer = moe.Layer(w, two.layer.inp, DEV)
    layer.forward_train(X=h)
    assert torch.equal(g2["dh"], layer.backward_train(g2["dy"], X=h)["dX"])
    y = two.layer.out.double()
    step = R.half_step(w.torch_dtype)
    want = R.residual_norm_backward(dout.double(), None, None, y, two.p["w_post"], None, None,
                                    two.r_post.double(), None)
    near(g2["dx"], want[0], 2 * R.ROW * want[0].abs(), step, "dx of the second")
    # the first: gradients of <dx, out> + <dh, h>
    args = [t.double() for t in (g2["dx"], g2["dh"], mid, one.layer.out)] + \
        [one.p["w_post"], None, one.p["w_next"], one.r_post.double(), one.r_next.double()]
    ref = R.residual_norm_backward(*args)
    mag = R.residual_norm_backward(*args, magnitudes=True)
    chain_err = R.ROW + (w.n + 4000) * R.U
    near(g1["dy"], ref[1], 3 * R.ROW * mag[1], step, "dy")
    near(g1["dw_next"], ref[4], chain_err * mag[4], R.U, "dw_next")
    assert two.clip_grads(1e-3)[1].item() < 1.0  # no pre-norm's gradient among them
    # beside the blocks that norm for themselves: in fp32 out is not rounded between
    # the two forms, and the second block's inputs and gradients are the same bits
    if w.torch_dtype is torch.float32:
        mid_own, _ = one_own.forward_train(x)
        out_own, _ = two_own.forward_train(mid_own)
        assert torch.equal(mid, mid_own) and torch.equal(two_own.h, h)
        assert torch.equal(out, out_own)
        g2_own = two_own.backward_train(dout)
        assert torch.equal(g2["dy"], g2_own["dy"])
        # dw_next of the first is dw_pre of the second
        near(g1["dw_next"], g2_own["dw_pre"].double(), 2 * chain_err * mag[4], R.U, "dw_pre")
        near(g1["dy"], one_own.backward_train(g2_own["dx"])["dy"].double(), 6 * R.ROW * mag[1],
             2 * R.U, "dy of the first")


def test_decoding_through_two_blocks_in_a_graph():
    w = wl.SMALL[4].replace(name="decode", n=5)
    one, two, _, _, x, _ = chain(w, block.QuantizedLayer)

    def step():
        out, h = one.forward(x)
        return two.forward(out, h=h)[0]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = two.out.clone()
        assert torch.equal(got, step())
    del graph
