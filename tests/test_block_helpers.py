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
