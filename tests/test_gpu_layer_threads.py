"""Two host threads in the layer's calls at once, each with its own stream,
buffers and workspace, of sizes that take different amounts of shared memory."""
import ctypes
import subprocess
import threading

import pytest
import torch

from expert_dispatch_gemm_b200 import moe
from expert_dispatch_gemm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"

# The loop is C, so that the interpreter's lock does not keep the threads apart.
HAMMER = r"""
typedef int (*fn)(long, long, long, long, long, long, long);
int hammer(fn f, const long* a, int n) {
  for (int i = 0; i < n; ++i) {
    int st = f(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
    if (st) return st;
  }
  return 0;
}
"""


def at_once(tmp_path, name, argss, n):
    src, so = tmp_path / "hammer.c", str(tmp_path / "hammer.so")
    src.write_text(HAMMER)
    subprocess.check_call(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", so])
    hammer = ctypes.CDLL(so).hammer
    hammer.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_long), ctypes.c_int]
    call = ctypes.cast(getattr(moe.lib(), name), ctypes.c_void_p)
    start, status = threading.Barrier(len(argss)), {}

    def run(i):
        torch.cuda.set_device(0)
        start.wait()
        a = (ctypes.c_long * 7)(*(argss[i] + [0] * (7 - len(argss[i]))))
        status[i] = hammer(call, a, n)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(argss))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert set(status.values()) == {0}, status


class Side:
    def __init__(self, w):
        self.w, self.cfg = w, moe.config(w)
        self.S = wl.random_scores(w.n, w.E, 3, DEV)
        self.route = moe.RouteBuffers(self.cfg, DEV)
        self.ws = moe.workspace(self.cfg, DEV, layer=False)
        self.stream = torch.cuda.Stream()
        moe.moe_route_from_scores(self.cfg, self.S, None, self.route, self.ws)
        self.idx = self.route.idx.clone()

    def route_args(self):
        return [ctypes.addressof(self.cfg), self.S.data_ptr(), 0, ctypes.addressof(self.route.c),
                self.ws.data_ptr(), self.ws.numel(), self.stream.cuda_stream]

    def dispatch_args(self):
        self.X = torch.randn((self.w.n, self.w.d), device=DEV).to(self.w.torch_dtype)
        self.P = torch.zeros((self.route.sizes.rows, self.w.d), dtype=self.X.dtype, device=DEV)
        return [ctypes.addressof(self.cfg), self.X.data_ptr(), ctypes.addressof(self.route.c),
                self.P.data_ptr(), self.stream.cuda_stream]


EC = wl.EC_BF16.replace(name="threads", n=4096, d=256, h=256)


@pytest.mark.parametrize("a,b", [
    (EC.replace(n=16384, E=4), EC.replace(n=16384, E=8)),    # 8,192 picks an expert, and 4,096
    (EC.replace(E=256), EC.replace(E=200)),                  # experts of a token's list
], ids=["picks", "experts"])
def test_expert_choice_from_two_threads(tmp_path, a, b):
    sides = [Side(a), Side(b)]
    torch.cuda.synchronize()
    at_once(tmp_path, "moe_route_from_scores", [s.route_args() for s in sides], 3000)
    for s in sides:
        assert torch.equal(s.route.idx, s.idx)
        assert moe.moe_read_error(s.ws) == (moe.MOE_OK, 0)


def test_dispatch_from_two_threads(tmp_path):
    w = wl.TC_DROPLESS.replace(name="threads", n=1000, h=256)
    sides = [Side(w.replace(d=7168)), Side(w.replace(d=256))]
    args = [s.dispatch_args() for s in sides]
    torch.cuda.synchronize()
    at_once(tmp_path, "moe_dispatch", args, 10_000)
    for s in sides:  # (on the host: row_token holds nothing behind the last segment)
        rows = s.route.tok_row.cpu().long()
        assert int(rows.min()) >= 0 and int(rows.max()) < s.P.shape[0]  # dropless
        assert torch.equal(s.P.cpu()[rows], s.X.cpu()[:, None].expand(-1, rows.shape[1], -1))
