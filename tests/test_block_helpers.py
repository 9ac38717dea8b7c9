"""Host logic of block.Block and block.QuantizedLayer (no GPU): on which device
and stream their steps run, and what they refuse before the first of them.

The library's calls are replaced by a log, and the tensors are host tensors:
`_device_of` names their device, another one is current."""
import contextlib
import types

import pytest
import torch

from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl

HERE = -1  # what a host tensor's get_device() says


class Calls:
    """The entry points called, each with the device and stream it ran on."""

    def __init__(self, monkeypatch):
        self.device, self.stream, self.log = 0, "device 0's", []
        monkeypatch.setattr(block, "_device_of", lambda t: HERE)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(torch.cuda, "device", self.on_device)
        monkeypatch.setattr(torch.cuda, "stream", self.on_stream)
        monkeypatch.setattr(block, "_call", self.call)
        monkeypatch.setattr(moe, "workspace", lambda cfg, device, layer=True, stream=None:
                            self.made("moe.workspace"))
        monkeypatch.setattr(block, "grad_workspace",
                            lambda *a: self.made("grad_workspace"))
        for name in ("moe_route", "moe_combine", "moe_layer_forward", "moe_layer_forward_train",
                     "moe_layer_backward_train"):
            monkeypatch.setattr(moe, name, lambda *a, name=name, **k: self.note(name))
        monkeypatch.setattr(moe, "backward_workspace",
                            lambda cfg, device, stream=None: (self.made("backward_workspace"), 1))
        # a gradient list takes host tensors here
        monkeypatch.setattr(block, "grad_list", lambda g: types.SimpleNamespace(
            grads=g, device=None, c=None, count=len(g)))

    def call(self, what, dev, stream, *args):
        with self.on_device(dev) if self.device != dev else contextlib.nullcontext():
            self.log.append((what, self.device, stream or self.stream))

    def note(self, what):
        self.log.append((what, self.device, self.stream))

    def made(self, what):
        self.note(what)
        return torch.empty(512, dtype=torch.uint8)

    @contextlib.contextmanager
    def on_device(self, dev):
        old = self.device, self.stream
        self.device, self.stream = HERE, "the tensors'"
        yield
        self.device, self.stream = old

    @contextlib.contextmanager
    def on_stream(self, s):
        old = self.device, self.stream
        self.device, self.stream = HERE, s
        yield
        self.device, self.stream = old

    def names(self):
        return [c[0] for c in self.log]


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


W = wl.SMALL[3].replace(name="host", n=40)
SERVE = ["moe_route", "moe_dispatch_i8", "moe_gemm_i8", "moe_quantize_rows", "moe_gemm_i8",
         "moe_combine"]
TAIL = "moe_residual_norm_forward"


class Stream:
    def __init__(self, dev=HERE):
        self.device = types.SimpleNamespace(index=dev)


def params():
    return {k: torch.ones(W.d) for k in ("w_pre", "w_post", "w_next")}


def test_quantized_layer_runs_on_its_tensors_device(calls):
    inp = wl.make_inputs(W)
    q = block.QuantizedLayer(W, inp, "cpu")
    assert "moe.workspace" in calls.names() and "moe_quantize_rows" in calls.names()
    assert all(c[1] == HERE for c in calls.log)
    calls.log.clear()
    q.forward(inp["X"])
    assert calls.names() == SERVE and {c[1:] for c in calls.log} == {(HERE, "the tensors'")}
    assert calls.device == 0
    calls.log.clear()
    s = Stream()
    q.forward(inp["X"], s)
    assert {c[1:] for c in calls.log} == {(HERE, s)}


def test_block_runs_on_its_tensors_device(calls):
    inp = wl.make_inputs(W)
    for s in (None, Stream()):
        calls.log.clear()
        b = block.Block(moe.Layer(W, inp, "cpu"), params())
        calls.log.clear()  # (a layer is made on the current device, as ever)
        x = inp["X"]
        out, _ = b.forward(x, stream=s)
        out, _ = b.forward_train(x, stream=s)
        b.backward_train(out, out, stream=s)
        b.clip_grads(1.0, stream=s)
        want = ["moe_norm_forward", "moe_layer_forward", TAIL, "moe_norm_forward",
                "backward_workspace", "moe_layer_forward_train", TAIL,
                "moe_residual_norm_backward", "moe_layer_backward_train", "moe_norm_backward",
                "grad_workspace", "moe_grad_clip"]
        assert calls.names() == want
        assert {c[1:] for c in calls.log} == {(HERE, s or "the tensors'")}


def test_quantized_layer_refuses_before_the_first_step(calls):
    inp = wl.make_inputs(W)
    q = block.QuantizedLayer(W, inp, "cpu")
    calls.log.clear()
    x = inp["X"]
    for bad, error in ((x[:-1], ValueError), (x.float(), TypeError), (x[:, :-16], ValueError),
                       (x.t().contiguous().t(), ValueError), (None, ValueError)):
        with pytest.raises(error):
            q.forward(bad)
    assert not calls.log
    # the router's operands are the call's too
    for k, t in (("Wg", inp["Wg"][:, :-1].contiguous()), ("Wg", inp["Wg"].to(torch.bfloat16)),
                 ("logit_bias", torch.zeros(W.E - 1)), ("sel_bias", torch.zeros(W.E + 1)),
                 ("Wg", None)):
        with pytest.raises((TypeError, ValueError)):
            block.QuantizedLayer(W, {**inp, k: t}, "cpu")


def test_streams_of_another_device_are_refused(calls):
    inp = wl.make_inputs(W)
    b = block.Block(moe.Layer(W, inp, "cpu"), params())
    q = block.QuantizedLayer(W, inp, "cpu")
    calls.log.clear()
    for call in (lambda: b.forward(inp["X"], Stream(0)), lambda: b.clip_grads(1.0, Stream(0)),
                 lambda: q.forward(inp["X"], Stream(0))):
        with pytest.raises(ValueError):
            call()
    assert not calls.log


def test_backward_needs_the_forward_that_kept_its_inputs(calls):
    """After forward(), the layer's saved activations are of an earlier step, or none."""
    inp = wl.make_inputs(W)
    b = block.Block(moe.Layer(W, inp, "cpu"), params())
    x = inp["X"]
    with pytest.raises(RuntimeError, match="forward_train"):
        b.backward_train(x, x)
    b.forward(x)
    with pytest.raises(RuntimeError, match="forward_train"):
        b.backward_train(x, x)
    b.forward_train(x)
    b.backward_train(x, x)
    b.backward_train(x, x)  # again, with other gradients
    b.forward(x)
    with pytest.raises(RuntimeError, match="forward_train"):
        b.backward_train(x, x)
    # a forward that fails leaves nothing to go back through
    b.forward_train(x)
    with pytest.raises(ValueError):
        b.forward_train(x[:-1])
    with pytest.raises(RuntimeError, match="forward_train"):
        b.backward_train(x, x)


def test_training_of_8_bit_experts_is_refused(calls):
    inp = wl.make_inputs(W)
    b = block.Block(block.QuantizedLayer(W, inp, "cpu"), params())
    calls.log.clear()
    with pytest.raises(TypeError, match="no backward pass"):
        b.forward_train(inp["X"])
    with pytest.raises(TypeError, match="no backward pass"):
        b.clip_grads(1.0)
    assert not calls.log


def test_a_block_that_takes_its_normed_input(calls):
    inp = wl.make_inputs(W)
    p = {k: torch.ones(W.d) for k in ("w_post", "w_next")}
    b = block.Block(moe.Layer(W, inp, "cpu"), p)
    own = block.Block(moe.Layer(W, inp, "cpu"), {**p, "w_pre": torch.ones(W.d)})
    x, h = inp["X"], inp["X"].clone()
    calls.log.clear()
    for bad, error in (((x, None), ValueError), ((x, h[:-1]), ValueError),
                       ((x[:-1], h), ValueError), ((x.float(), h), TypeError),
                       ((x, h.float()), TypeError)):
        with pytest.raises(error):
            b.forward_train(bad[0], h=bad[1])
    with pytest.raises(ValueError):  # which norm?
        own.forward(x, h=h)
    assert not calls.log
    out, _ = b.forward_train(x, h=h)
    g = b.backward_train(out, out)
    assert calls.names() == ["backward_workspace", "moe_layer_forward_train", TAIL,
                             "moe_residual_norm_backward", "moe_layer_backward_train"]
    assert g["dh"] is g["layer"]["dX"] and g["dw_pre"] is None


def test_training_on_the_blocks_own_outputs_is_refused(calls):
    """They are overwritten by the forward that should be gone back through; without
    a backward pass a block may take them."""
    inp = wl.make_inputs(W)
    b = block.Block(moe.Layer(W, inp, "cpu"), params())
    two = block.Block(moe.Layer(W, inp, "cpu"), {"w_next": torch.ones(W.d)})
    x = inp["X"]
    out, h = b.forward_train(x)
    out2, h2 = two.forward_train(out, h=h)
    calls.log.clear()
    for call in (lambda: b.forward_train(out), lambda: b.forward_train(h),
                 lambda: two.forward_train(out2, h=h), lambda: two.forward_train(out, h=h2)):
        with pytest.raises(ValueError, match="overwritten"):
            call()
    assert not calls.log
    b.forward(out)
    two.forward(out2, h=h2)


def test_a_layer_in_two_blocks_goes_back_through_the_last_one_only(calls):
    """The layer keeps one forward's activations: the other block's are gone."""
    inp = wl.make_inputs(W)
    layer = moe.Layer(W, inp, "cpu")
    one, two = block.Block(layer, params()), block.Block(layer, params())
    x = inp["X"]
    one.forward_train(x)
    two.forward_train(x)
    two.backward_train(x, x)
    with pytest.raises(RuntimeError, match="another block"):
        one.backward_train(x, x)
    one.forward_train(x)
    one.backward_train(x, x)
    two.forward(x)  # serving through the same layer overwrites them too
    with pytest.raises(RuntimeError, match="another block"):
        one.backward_train(x, x)
