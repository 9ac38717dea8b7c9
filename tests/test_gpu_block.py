"""A block (pre-norm, layer, post-norm with gate and residual, next pre-norm)
run as a user runs it: serving, training with the clip, and in a graph."""
import math
import os
import subprocess
import sys

import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def near(got, want, rel_mag, rounding, name):
    tol = rounding * want.abs() + rel_mag + 1e-37
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), (name, off.max().item())


def make(w, seed=3, tokens=100, gate=True):
    inp = wl.make_inputs(w, DEV)
    g = gen(seed)
    f = lambda: 1 + 0.1 * torch.randn(w.d, generator=g, device=DEV)  # noqa: E731
    p = {"w_pre": f(), "w_post": f(), "w_next": f()}
    if gate:
        p["gate"] = (0.5 * torch.randn((-(-w.n // tokens) if tokens else 1, w.d), generator=g,
                                       device=DEV)).to(w.torch_dtype)
    b = block.Block(moe.Layer(w, inp, DEV), p, eps=1e-5, gate_tokens=tokens, block_scale=0.5)
    x = torch.randn((w.n, w.d), generator=g, device=DEV).to(w.torch_dtype)
    dout = torch.randn((w.n, w.d), generator=g, device=DEV).to(w.torch_dtype)
    dh = torch.randn((w.n, w.d), generator=g, device=DEV).to(w.torch_dtype)
    return b, p, x, dout, dh


@pytest.mark.parametrize("w", [wl.EC_FP32, wl.SMALL[2], wl.SMALL[3], wl.SMALL[4]],
                         ids=lambda w: w.name)
def test_train_step(w):
    b, p, x, dout, dh = make(w)
    out, h_next = b.forward_train(x)
    g = b.backward_train(dout, dh)
    torch.cuda.synchronize()
    step = R.half_step(w.torch_dtype)
    kw = dict(b=0.5, tokens=100)
    # forward: each step from what the one before it stored
    h, r = R.norm(x.double(), p["w_pre"], 0.0, 1e-5)
    near(b.h, h, 2 * R.ROW * h.abs(), step, "h")
    y = b.layer.out
    ref, hn, r1, r2 = R.residual_norm(x.double(), y.double(), p["w_post"], p["gate"],
                                      p["w_next"], eps=1e-5, **kw)
    terms = x.double().abs() + (ref - x.double()).abs()
    near(out, ref, R.ROW * terms, step, "out")
    scale = r2[:, None] * p["w_next"].double().abs()
    mix = 1 + (terms * ref.abs()).mean(1, keepdim=True) / (ref * ref).mean(1, keepdim=True)
    near(h_next, hn, R.ROW * (terms * scale + mix * hn.abs()), step, "h_next")
    # backward
    rows = b.p["gate"].shape[0]
    args = [t.double() for t in (dout, dh, out, y)] + [p["w_post"], p["gate"], p["w_next"],
                                                       b.r_post.double(), b.r_next.double()]
    want = R.residual_norm_backward(*args, gate_rows=rows, **kw)
    mag = R.residual_norm_backward(*args, gate_rows=rows, magnitudes=True, **kw)
    chain = R.ROW + (w.n + 4000) * R.U
    near(g["dy"], want[1], 3 * R.ROW * mag[1], step, "dy")
    near(g["dw_post"], want[2], (2 * R.ROW + chain) * mag[2], R.U, "dw_post")
    near(g["dgate"], want[3], (2 * R.ROW + chain) * mag[3], step, "dgate")
    near(g["dw_next"], want[4], chain * mag[4], R.U, "dw_next")
    # the layer's own gradient is what moe.Layer gives for dy
    lg = {k: None if t is None else t.clone() for k, t in g["layer"].items()}
    layer2 = moe.Layer(w, b.layer.inp, DEV)
    layer2.forward_train(X=b.h)
    again = layer2.backward_train(g["dy"], X=b.h)
    for k in ("dX", "dW1", "dWg"):
        assert torch.equal(lg[k], again[k]), k
    # dx: the residual's share was rounded once before the pre-norm's was added
    args = (want[0], lg["dX"].double(), x.double(), torch.zeros_like(h), None, None, p["w_pre"],
            None, b.r_pre.double())
    dx = R.residual_norm_backward(*args)
    dmag = R.residual_norm_backward(*args, magnitudes=True)
    near(g["dx"], dx[0], step * want[0].abs() + 4 * R.ROW * (dmag[0] + mag[0]), step, "dx")
    near(g["dw_pre"], dx[4], chain * dmag[4] + 2 * R.ROW * dmag[4], R.U, "dw_pre")
    # clip: every parameter's gradient, in place
    names = ["dw_pre", "dw_post", "dgate", "dw_next"]
    params = [g[k] for k in names] + [t for k, t in g["layer"].items()
                                      if t is not None and k not in ("dX", "dL")]
    before = [t.clone() for t in params]
    total = math.sqrt(sum(float((t.double() ** 2).sum()) for t in before))
    norm, factor = b.clip_grads(0.25 * total).tolist()
    assert abs(norm - total) <= 10 * R.U * total
    for t, o in zip(params, before):
        near(t, o.double() * (0.25 * total / (total + 1e-6)), 14 * R.U * o.double().abs(), step,
             "clipped")
    assert abs(factor - 0.25) < 1e-6
    # one more clip finds the norm inside the limit (or a rounding above it)
    norm2, factor2 = b.clip_grads(0.2501 * total).tolist()
    assert norm2 <= 0.2501 * total and factor2 == 1.0


def test_block_without_optional_parts():
    w = wl.SMALL[3]
    inp = wl.make_inputs(w, DEV)
    p = {"w_pre": torch.ones(w.d, device=DEV)}
    b = block.Block(moe.Layer(w, inp, DEV), p)
    x = inp["X"]
    out, h_next = b.forward_train(x)
    assert h_next is None
    want = x.double() + b.layer.out.double()
    near(out, want, 2 * R.U * (x.double().abs() + b.layer.out.double().abs()),
         R.half_step(out.dtype), "out")
    dout = torch.randn_like(out)
    g = b.backward_train(dout)
    assert torch.equal(g["dy"], dout)
    assert b.clip_grads(1.0)[1].item() < 1.0


@pytest.mark.parametrize("tokens", [1, 100])
def test_gate_that_is_a_slice_of_wider_rows(tokens):
    """A gate with a stride (one of several parts of a modulation's rows): the
    same bits as its dense copy gives, backward and clip included."""
    w = wl.SMALL[3]
    res = []
    for wide in (False, True):
        b, p, x, dout, dh = make(w, tokens=tokens)
        rows = p["gate"].shape[0]
        if wide:
            parts = torch.full((rows, 3 * w.d), float("nan"), dtype=w.torch_dtype, device=DEV)
            parts[:, w.d:2 * w.d] = p["gate"]
            p["gate"] = parts[:, w.d:2 * w.d]
            b = block.Block(moe.Layer(w, b.layer.inp, DEV), p, eps=1e-5, gate_tokens=tokens,
                            block_scale=0.5, gate_stride=3 * w.d)
        out, h_next = b.forward_train(x)
        g = b.backward_train(dout, dh)
        own = [g[k] for k in ("dx", "dy", "dw_pre", "dw_post", "dgate", "dw_next")]
        res.append([out.clone(), h_next.clone()] + [t.clone() for t in own])
        total = math.sqrt(sum(float((t.double() ** 2).sum()) for t in own[2:] + [
            t for k, t in g["layer"].items() if t is not None and k not in ("dX", "dL")]))
        norm, factor = b.clip_grads(0.25 * total).tolist()
        # (the list's squares are added in fp64; 10 roundings as in test_train_step)
        assert abs(norm - total) <= 10 * R.U * total
        near(g["dgate"], res[-1][6].double() * (0.25 * total / (total + 1e-6)),
             14 * R.U * res[-1][6].double().abs(), R.half_step(w.torch_dtype), "clipped gate")
    for i, (s, t) in enumerate(zip(*res)):
        assert torch.equal(s, t), i


def test_serving_with_8_bit_experts():
    w = wl.SMALL[4]
    inp = wl.make_inputs(w, DEV)
    p = {"w_pre": torch.ones(w.d, device=DEV), "w_post": torch.ones(w.d, device=DEV),
         "w_next": torch.ones(w.d, device=DEV)}
    exact = block.Block(moe.Layer(w, inp, DEV), p)
    fast = block.Block(block.QuantizedLayer(w, inp, DEV), p)
    x = inp["X"]
    a, ha = exact.forward(x)
    b, hb = fast.forward(x)
    for s, t in ((a, b), (ha, hb)):
        # the layer's 6% (see the quantised layer's test) before a residual of equal size
        assert (s.double() - t.double()).norm() / s.double().norm() < 0.06


def test_decode_step_in_a_graph():
    """Two blocks in a row on one token batch, the first one's fused next
    pre-norm feeding a layer, captured and replayed on new tokens."""
    w = wl.SMALL[4].replace(name="decode", n=5)
    inp = wl.make_inputs(w, DEV)
    p = {k: torch.ones(w.d, device=DEV) for k in ("w_pre", "w_post", "w_next")}
    one = block.Block(block.QuantizedLayer(w, inp, DEV), p)
    two = block.QuantizedLayer(w, inp, DEV)
    x = inp["X"].clone()

    def step():
        _, h = one.forward(x)
        return two.forward(h)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = two.out.clone(), one.out.clone()
        want = step().clone(), one.out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del graph


CHECKED = os.environ.get("MOE_LIBRARY") == "checked"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(args, **env):
    r = subprocess.run([sys.executable, *args], env=dict(os.environ, **env), cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout


@pytest.mark.skipif(CHECKED, reason="the driver of the checked run")
def test_checked_build():
    """The same products and layers in the checked build, where every group that
    does not fit its buffers is reported; the test below plants one."""
    out = _run(["-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                "tests/test_gpu_i8.py", "tests/test_gpu_block.py", "-k",
                "one_group or many_groups or split_reduction or quantized_layer or train_step "
                "or serving or reports_groups"], MOE_LIBRARY="checked")
    assert " passed" in out and "failed" not in out


@pytest.mark.skipif(not CHECKED, reason="runs under the checked build (MOE_LIBRARY=checked)")
def test_checked_build_reports_groups_that_do_not_fit():
    cfg = block.gemm_i8_config(2, 64, 32, 16)
    i8 = dict(dtype=torch.int8, device=DEV)
    x, w = torch.ones((64, 32), **i8), torch.ones((2, 16, 32), **i8)
    xs, s = torch.ones(64, device=DEV), torch.ones((2, 16), device=DEV)
    out = torch.zeros((64, 16), dtype=torch.bfloat16, device=DEV)
    ws = block.gemm_i8_workspace(cfg, DEV)
    at = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    for counts, code in (([40, 24], 0), ([40, 30], 0x221)):
        n = torch.tensor(counts, dtype=torch.int32, device=DEV)
        block.moe_gemm_i8(cfg, x, xs, at, n, w, s, None, None, out, ws)
        torch.cuda.synchronize()
        assert moe.moe_read_error(ws)[1] == code
        assert bool((out == 32.0).all())  # cut to the rows that are there


FIRST_CALLS = """
import torch
from expert_dispatch_gemm_b200 import block
dev, bf = "cuda", torch.bfloat16
n, d, o = 40, 256, 256
x = torch.randn(n, d, device=dev).to(bf)
y, dout, dh = x * 2, x.clone(), x.clone()
w = torch.ones(d, device=dev)
out, h, dx, dy = (torch.empty_like(x) for _ in range(4))
r1, r2 = torch.empty(n, device=dev), torch.empty(n, device=dev)
dw1, dw2 = torch.empty(d, device=dev), torch.empty(d, device=dev)
cfg = block.norm_config(n, d, bf, 1e-6)
ws = block.norm_workspace(cfg, dev)
g = [torch.ones(1000, device=dev), torch.ones(333, device=dev, dtype=bf)]
glist = block.grad_list(g)
gws, norm = block.grad_workspace(glist, dev), torch.empty(2, device=dev)
q, qs = torch.empty((n, d), dtype=torch.int8, device=dev), torch.empty(n, device=dev)
wq = torch.ones((1, o, d), dtype=torch.int8, device=dev)
wsc = torch.ones((1, o), device=dev)
c = block.gemm_i8_config(1, n, d, o)
prod, iws = torch.empty((n, o), device=dev, dtype=bf), block.gemm_i8_workspace(c, dev)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    block.moe_residual_norm_forward(cfg, x, y, w, None, w, out, h, r1, r2)
    block.moe_residual_norm_backward(cfg, dout, dh, out, y, w, None, w, r1, r2, dx, dy, dw1, None,
                                     dw2, ws)
    block.moe_grad_clip(glist, 1.0, norm, gws)
    block.moe_quantize_rows(h, q, qs)
    block.moe_gemm_i8(c, q, qs, None, None, wq, wsc, None, None, prod, iws)
graph.replay()
torch.cuda.synchronize()
ref = (q.double().sum(1) * qs.double())[:, None].expand(n, o)
assert ((prod.double() - ref).abs() <= 2 ** -8 * ref.abs() + 1e-30).all()
assert abs(norm[0].item() - 1333 ** 0.5) < 1e-4
assert torch.isfinite(dx).all() and torch.isfinite(dw1).all()
print("replayed")
"""


@pytest.mark.skipif(CHECKED, reason="once is enough")
def test_first_calls_of_a_process_inside_a_capture():
    assert "replayed" in _run(["-c", FIRST_CALLS])


def test_wrong_use_is_refused():
    w = wl.SMALL[3]
    inp = wl.make_inputs(w, DEV)
    p = {"w_pre": torch.ones(w.d, device=DEV), "w_next": torch.ones(w.d, device=DEV)}
    fast = block.Block(block.QuantizedLayer(w, inp, DEV), p)
    with pytest.raises(TypeError):  # 8-bit experts have no backward pass
        fast.grads()
    b = block.Block(moe.Layer(w, inp, DEV), p)
    out, _ = b.forward_train(inp["X"])
    with pytest.raises(ValueError):  # h_next's gradient is missing
        b.backward_train(torch.ones_like(out))
    with pytest.raises(moe.MoeError):  # d is not a multiple of 16
        v = wl.EC_FP32.replace(d=24, h=40)
        block.QuantizedLayer(v, wl.make_inputs(v, DEV), DEV)
    t = torch.ones(100, device=DEV)
    with pytest.raises(ValueError):  # the same tensor twice, in place
        block.grad_list([t, t])
    with pytest.raises(ValueError):  # an output over another gradient
        block.grad_list([t[:50], t[50:]], [t[50:], torch.empty(50, device=DEV)])
    with pytest.raises(ValueError):
        block.grad_list([t[::2]])
    glist = block.grad_list([t, t], [torch.empty_like(t), torch.empty_like(t)])  # read twice: fine
    norm = torch.empty(2, device=DEV)
    block.moe_grad_clip(glist, 1.0, norm, block.grad_workspace(glist, DEV))
    assert abs(norm[0].item() - 200 ** 0.5) < 1e-5
    with pytest.raises(ValueError):
        block.moe_grad_clip(glist, 1.0, norm[:1], block.grad_workspace(glist, DEV))
    cfg = block.norm_config(4, 64, torch.bfloat16, 1e-6, gate_tokens=2)
    x = torch.ones(4, 64, device=DEV, dtype=torch.bfloat16)
    o, one = torch.empty_like(x), torch.ones(64, device=DEV)
    for bad in (x.float(), x[:3], x.t(), x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            block.moe_residual_norm_forward(cfg, x, bad, one, None, None, o)
    with pytest.raises(ValueError):  # two gate rows are wanted
        block.moe_residual_norm_forward(cfg, x, x, one, x[:1], None, o)
    with pytest.raises(moe.MoeError):  # w_next without h
        block.moe_residual_norm_forward(cfg, x, x, one, None, one, o)
