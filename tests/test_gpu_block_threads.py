"""Two host threads in the block operators at once, each with its own stream,
buffers and workspace."""
import ctypes
import subprocess
import threading

import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block

pytestmark = pytest.mark.gpu
DEV = "cuda"

# The loop is C, so that the interpreter's lock does not keep the threads apart.
HAMMER = r"""
typedef int (*fn)(const void*, const void*, const void*, void*, void*, void*);
int hammer(fn f, const void* cfg, const void* x, const void* w, void* h, void* r, void* s, int n) {
  for (int i = 0; i < n; ++i) {
    int st = f(cfg, x, w, h, r, s);
    if (st) return st;
  }
  return 0;
}
"""


def test_norms_of_two_widths_from_two_threads(tmp_path):
    """One kernel, with more shared memory in one thread's launches than in the
    other's: neither may take away what the other was about to use."""
    src, so = tmp_path / "hammer.c", str(tmp_path / "hammer.so")
    src.write_text(HAMMER)
    subprocess.check_call(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", so])
    hammer = ctypes.CDLL(so).hammer
    P = ctypes.c_void_p
    hammer.argtypes = [P] * 7 + [ctypes.c_int]
    call = ctypes.cast(block.lib().moe_norm_forward, P)
    n = 1000  # a ring of four rows: 64 and 56 KB
    work, status = [], {}
    for d in (8192, 7168):
        x = torch.randn((n, d), device=DEV).to(torch.bfloat16)
        w, r = torch.ones(d, device=DEV), torch.empty(n, device=DEV)
        work.append((block.norm_config(n, d, x.dtype, 1e-6), x, w, torch.empty_like(x), r,
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def run(i):
        cfg, x, w, h, r, s = work[i]
        torch.cuda.set_device(x.device)
        start.wait()
        status[i] = hammer(call, ctypes.addressof(cfg), x.data_ptr(), w.data_ptr(), h.data_ptr(),
                           r.data_ptr(), s.cuda_stream, 30_000)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == {0: 0, 1: 0}
    for _, x, w, h, r, _ in work:
        want, rw = R.norm(x.double(), w, 0.0, 1e-6)
        assert bool(((h.double() - want).abs() <=
                     (R.half_step(h.dtype) + 2 * R.ROW) * want.abs()).all())
