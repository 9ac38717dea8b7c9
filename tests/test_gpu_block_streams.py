"""Block and QuantizedLayer on a stream of their own while the current one is busy."""
import pytest
import torch

from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_train_step_on_another_stream():
    """Nothing of the step waits for, or is left on, the current stream: buffers
    that the first call makes and clears included."""
    w = wl.SMALL[4]
    inp = wl.make_inputs(w, DEV)
    p = {k: torch.ones(w.d, device=DEV) for k in ("w_pre", "w_post", "w_next")}
    x, dout = inp["X"], torch.randn((w.n, w.d), device=DEV).to(w.torch_dtype)

    def step(b, s):
        out, h = b.forward_train(x, stream=s)
        g = b.backward_train(dout, dout, stream=s)
        norm = b.clip_grads(0.5, stream=s)
        return [out, h, norm, g["dx"], g["dw_post"], g["dw_next"], g["dw_pre"],
                g["layer"]["dW1"], g["layer"]["dW2"]]

    want = [t.clone() for t in step(block.Block(moe.Layer(w, inp, DEV), p), None)]
    b = block.Block(moe.Layer(w, inp, DEV), p)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = step(b, s)
    s.synchronize()
    busy = not torch.cuda.current_stream().query()
    for a, t in zip(want, [t.cpu() for t in got]):
        assert torch.equal(a.cpu(), t)
    assert busy
    assert moe.moe_read_error(b.layer._bws, s) == (moe.MOE_OK, 0)


def test_serving_on_another_stream():
    w = wl.SMALL[4]
    inp = wl.make_inputs(w, DEV)
    q = block.QuantizedLayer(w, inp, DEV)
    want = q.forward(inp["X"]).clone()
    q.out.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    q.forward(inp["X"], stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    assert torch.equal(q.out, want)
