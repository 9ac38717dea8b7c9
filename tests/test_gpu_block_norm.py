"""Residual norms on the GPU against their 64-bit form (block_ref), at the
sizes, gates and layouts where the kernels change their path. Tolerances count
roundings (see block_ref) and were fixed before the first run."""
import itertools

import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Case:
    def __init__(self, n, d, dtype, tokens, post=True, gate=True, nxt=True, off=0.0, a=1.0,
                 b=1.0, stride=None, shift=0, seed=1):
        g, dt = gen(seed), DT[dtype]
        self.n, self.d, self.dt, self.tokens = n, d, dt, tokens
        self.kw = dict(off=off, a=a, b=b, tokens=tokens)
        self.cfg = block.norm_config(n, d, dt, EPS, off, a, b, tokens, stride)
        self.rows = block.norm_gate_rows(self.cfg)
        self.shift = shift
        self.x = self.make(g, n, d, 2.0)
        self.y = self.make(g, n, d, 1.5)
        w = lambda: (1 - off + 0.2 * torch.randn(d, generator=g, device=DEV))  # noqa: E731
        self.w_post = w() if post else None
        self.w_next = w() if nxt else None
        self.gate = None
        if gate:
            pitch = stride or d
            store = (0.5 * torch.randn((max(self.rows, 1), pitch), generator=g, device=DEV)).to(dt)
            self.gate = store[:self.rows, :d]
        self.dout, self.dh = self.make(g, n, d, 1.0), self.make(g, n, d, 1.0) if nxt else None

    def make(self, g, n, d, s):
        """[n, d], `shift` elements behind an aligned address."""
        t = (s * torch.randn(n * d + self.shift, generator=g, device=DEV)).to(self.dt)
        return t[self.shift:].view(n, d)

    def empty(self):
        return torch.full((self.n * self.d + self.shift,), 7.0, dtype=self.dt,
                          device=DEV)[self.shift:].view(self.n, self.d)

    def forward(self, out=None, h=None):
        f = dict(dtype=torch.float32, device=DEV)
        self.out = self.empty() if out is None else out
        self.h = None if self.w_next is None else self.empty() if h is None else h
        self.r1 = torch.full((self.n,), -1.0, **f) if self.w_post is not None else None
        self.r2 = torch.full((self.n,), -1.0, **f) if self.w_next is not None else None
        block.moe_residual_norm_forward(self.cfg, self.x, self.y, self.w_post, self.gate,
                                        self.w_next, self.out, self.h, self.r1, self.r2)

    def check_forward(self, x, y):
        """x, y: copies of the inputs (the call may have overwritten them)"""
        x, y = x.double(), y.double()
        out, h, r1, r2 = R.residual_norm(x, y, self.w_post, self.gate, self.w_next, eps=EPS,
                                         **self.kw)
        v = y if r1 is None else R.norm(y, self.w_post, self.kw["off"], EPS)[0]
        terms = (self.kw["a"] * x).abs() + (
            self.kw["b"] * R.gate_of(self.gate, self.n, self.tokens) * v).abs()
        step = R.half_step(self.dt)
        near(self.out, out, step * out.abs() + R.ROW * terms, "out")
        if r1 is not None:
            near(self.r1, r1, R.ROW * r1, "rstd_post")
        if h is not None:
            # out enters h with its terms' error, and through its own norm
            rel = R.ROW * (1 + (terms * out.abs()).mean(1) / (out * out).mean(1).clamp(min=EPS))
            near(self.r2, r2, rel * r2, "rstd_next")
            w = (self.w_next.double() + self.kw["off"]).abs()
            near(self.h, h, step * h.abs() + R.ROW * terms * r2[:, None] * w +
                 rel[:, None] * h.abs(), "h")

    def backward(self, dx=None, dy=None, dout=True, poison=False):
        """gradients from the stored forward results"""
        f = dict(dtype=torch.float32, device=DEV)
        self.dx = self.empty() if dx is None else dx
        self.dy = self.empty() if dy is None else dy
        self.dw_post = torch.full((self.d,), 7.0, **f) if self.w_post is not None else None
        self.dw_next = torch.full((self.d,), 7.0, **f) if self.w_next is not None else None
        self.dgate = None
        if self.gate is not None:
            self.dgate = torch.full((max(self.rows, 1), int(self.cfg.gate_stride)), 7.0,
                                    dtype=self.dt, device=DEV)[:self.rows, :self.d]
        self.ws = block.norm_workspace(self.cfg, DEV)
        if poison:
            self.ws.fill_(0xff)  # NaNs
        block.moe_residual_norm_backward(
            self.cfg, self.dout if dout else None, self.dh,
            self.out if self.w_next is not None else None, self.y, self.w_post, self.gate,
            self.w_next, self.r1, self.r2, self.dx, self.dy, self.dw_post, self.dgate,
            self.dw_next, self.ws)

    def reference(self, dout=True, **more):
        dbl = lambda t: None if t is None else t.double()  # noqa: E731
        return R.residual_norm_backward(
            dbl(self.dout) if dout else None, dbl(self.dh), dbl(self.out), dbl(self.y),
            self.w_post, self.gate, self.w_next, dbl(self.r1), dbl(self.r2),
            gate_rows=self.rows, **self.kw, **more)

    def check_backward(self, ref, mag):
        step = R.half_step(self.dt)
        # sums over tokens: a chain of a worker's rows, then of the workers,
        # each term off by a row's error
        chain = R.ROW + (self.n + 2 * 148 * 12) * R.U
        for name, got, want, m, rounding, err in (
                ("dx", self.dx, ref[0], mag[0], step, 2 * R.ROW),
                ("dy", self.dy, ref[1], mag[1], step, 3 * R.ROW),
                ("dw_post", self.dw_post, ref[2], mag[2], R.U, 2 * R.ROW + chain),
                ("dgate", self.dgate, ref[3], mag[3], step, 2 * R.ROW + chain),
                ("dw_next", self.dw_next, ref[4], mag[4], R.U, chain)):
            assert (got is None) == (want is None), name
            if got is not None:
                near(got, want, rounding * want.abs() + err * m, name)


def near(got, want, tol, name):
    assert got.shape == want.shape, name
    if got.numel() == 0:
        return
    off = (got.double() - want).abs() - tol
    assert bool((off <= 1e-40).all()), (
        f"{name}: off by {(got.double() - want).abs().max().item():.3g}, over its bound by "
        f"{off.max().item():.3g}")


SIZES = [(1, 1), (3, 7), (5, 8), (2, 31), (37, 64), (300, 192), (129, 256), (65, 257), (33, 520),
         (19, 1000), (41, 1024), (7, 2048), (301, 2048), (13, 7168), (9, 8192), (3, 8200),
         (2, 16384), (2, 16383)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", SIZES)
def test_sizes(n, d, dtype):
    """Every path of the kernels: warp and block rows, vectors or not, staged or not."""
    c = Case(n, d, dtype, 0, a=0.75, b=1.5, seed=n * 31 + d)
    c.forward()
    c.check_forward(c.x, c.y)
    c.backward()
    c.check_backward(c.reference(), c.reference(magnitudes=True))


@pytest.mark.parametrize("tokens", [0, 1, 2, 3, 16, 64, 250, 1000, 5000])
@pytest.mark.parametrize("n,d,dtype", [(1, 64, "f32"), (1000, 128, "bf16"), (997, 72, "f32"),
                                       (3000, 40, "bf16"), (250, 9, "f32")])
def test_gate_rows(n, d, dtype, tokens):
    """Gate rows shared by any number of tokens, the last one by fewer; their
    gradients sum over a worker's rows, over many workers', or over both."""
    c = Case(n, d, dtype, tokens, seed=tokens + n)
    c.forward()
    c.check_forward(c.x, c.y)
    c.backward()
    c.check_backward(c.reference(), c.reference(magnitudes=True))


@pytest.mark.parametrize("post,gate,nxt", [p for p in itertools.product([0, 1], repeat=3)])
def test_optional_parts(post, gate, nxt):
    for dtype, shift in (("bf16", 0), ("f32", 0), ("bf16", 1), ("f32", 3)):
        c = Case(77, 320, dtype, 10, bool(post), bool(gate), bool(nxt), off=1.0, a=1.25, b=0.5,
                 shift=shift, seed=5)
        c.forward()
        c.check_forward(c.x, c.y)
        c.backward()
        c.check_backward(c.reference(), c.reference(magnitudes=True))
        if nxt:  # nothing reaches out but through the norm
            c.backward(dout=False)
            c.check_backward(c.reference(dout=False), c.reference(dout=False, magnitudes=True))


def test_strided_gate_leaves_the_rest_of_its_rows():
    for dtype, d, stride in (("bf16", 192, 576), ("f32", 100, 301)):
        c = Case(50, d, dtype, 7, stride=stride, seed=9)
        c.forward()
        c.check_forward(c.x, c.y)
        c.backward()
        c.check_backward(c.reference(), c.reference(magnitudes=True))
        whole = c.dgate.as_strided((c.rows, stride), (stride, 1))
        assert bool((whole[:, d:] == 7.0).all())


@pytest.mark.parametrize("d", [256, 1000, 7168])
def test_in_place(d):
    c = Case(40, d, "bf16", 8, seed=3)
    x, y = c.x.clone(), c.y.clone()
    c.forward(out=c.x, h=c.y)  # out over x, h over y
    c.check_forward(x, y)
    c = Case(40, d, "bf16", 8, seed=3)
    c.forward()
    ref, mag = c.reference(), c.reference(magnitudes=True)
    c.backward(dx=c.dout, dy=c.dh)  # dx over dout, dy over dh
    c.check_backward(ref, mag)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 5), (6, 64), (130, 1000), (257, 2048), (11, 7168)])
def test_pre_norm(n, d, dtype):
    c = Case(n, d, dtype, 0, off=1.0, seed=n + d)
    x, h, r = c.x.double(), c.empty(), torch.empty(n, device=DEV)
    block.moe_norm_forward(c.cfg, c.x, c.w_next, h, r)
    want, rw = R.norm(x, c.w_next, 1.0, EPS)
    near(r, rw, R.ROW * rw, "rstd")
    near(h, want, (R.half_step(c.dt) + 2 * R.ROW) * want.abs(), "h")
    ws = block.norm_workspace(c.cfg, DEV)
    for dres in (None, c.dout):
        dx, dw = c.empty(), torch.empty(d, device=DEV)
        block.moe_norm_backward(c.cfg, dres, c.dh, c.x, c.w_next, r, dx, dw, ws)
        args = (None if dres is None else dres.double(), c.dh.double(), x,
                torch.zeros_like(x), None, None, c.w_next, None, r.double())
        ref = R.residual_norm_backward(*args, off=1.0)
        mag = R.residual_norm_backward(*args, off=1.0, magnitudes=True)
        near(dx, ref[0], R.half_step(c.dt) * ref[0].abs() + 2 * R.ROW * mag[0], "dx")
        near(dw, ref[4], (2 * R.ROW + (n + 4000) * R.U) * mag[4], "dw")


def test_rows_of_zeros_and_no_rows():
    c = Case(6, 64, "f32", 2, seed=4)
    c.x[2:4] = 0
    c.y[3:5] = 0
    c.forward()
    c.check_forward(c.x, c.y)
    assert torch.isfinite(c.h).all()
    c.backward()
    for t in (c.dx, c.dy, c.dgate, c.dw_post, c.dw_next):
        assert torch.isfinite(t).all()
    c.check_backward(c.reference(), c.reference(magnitudes=True))
    for tokens in (0, 5):
        c = Case(0, 64, "bf16", tokens)
        c.forward()
        c.backward()
        assert not c.dw_post.any() and not c.dw_next.any() and not c.dgate.any()


def test_a_row_that_is_not_finite_stays_alone():
    c = Case(9, 96, "f32", 1, seed=8)
    c.y[4, 5] = float("nan")
    c.x[6, 0] = float("inf")
    c.forward()
    bad = torch.zeros(9, dtype=torch.bool, device=DEV)
    bad[4] = bad[6] = True
    assert torch.isfinite(c.h[~bad]).all() and torch.isfinite(c.out[~bad]).all()
    assert torch.isnan(c.out[4]).all() and torch.isinf(c.out[6, 0])


def test_gradient_against_differences():
    """The gradient times a direction equals the change of the 64-bit forward
    along it (central differences, step 1e-4: error about 1e-8 of the terms)."""
    c = Case(11, 48, "f32", 4, a=0.5, b=2.0, off=1.0, seed=12)
    c.forward()
    c.backward()
    g = gen(77)
    names = ("x", "y", "w_post", "gate", "w_next")
    at = {k: getattr(c, k).double() for k in names}
    to = {k: torch.randn(v.shape, generator=g, device=DEV, dtype=torch.float64)
          for k, v in at.items()}

    def loss(t):
        p = {k: at[k] + t * to[k] for k in names}
        out, h, _, _ = R.residual_norm(p["x"], p["y"], p["w_post"], p["gate"], p["w_next"],
                                       eps=EPS, **c.kw)
        return ((c.dout.double() * out).sum() + (c.dh.double() * h).sum()).item()

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    grads = {"x": c.dx, "y": c.dy, "w_post": c.dw_post, "gate": c.dgate, "w_next": c.dw_next}
    terms = [(grads[k].double() * to[k]) for k in names]
    got = sum(t.sum().item() for t in terms)
    size = sum(t.abs().sum().item() for t in terms)
    # the forward's out and norms, stored in fp32, carry a row's error into the gradient
    assert abs(got - slope) <= 8 * R.ROW * size, (got, slope)


def test_same_sums_every_time_and_on_other_streams():
    c = Case(2000, 512, "bf16", 300, seed=6)
    c.forward()
    c.backward()
    first = [t.clone() for t in (c.dx, c.dy, c.dw_post, c.dgate, c.dw_next)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.backward()
    s.synchronize()
    for a, b in zip(first, (c.dx, c.dy, c.dw_post, c.dgate, c.dw_next)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [0, 1, 7])
@pytest.mark.parametrize("n,d,dtype", [(3000, 7168, "bf16"), (4000, 4096, "bf16"),
                                       (1500, 8192, "f32"), (6000, 1000, "bf16"),
                                       (5000, 130, "f32"), (700, 16384, "bf16")])
def test_every_worker_ends_well(n, d, dtype, tokens):
    """Many rows a worker, so that its warps reach the end of their range apart,
    several times over a poisoned workspace: the sums that are joined there are
    those of the reference, and the same each time."""
    c = Case(n, d, dtype, tokens, seed=n)
    c.forward()
    ref, mag = c.reference(), c.reference(magnitudes=True)
    first = None
    for _ in range(4):
        c.backward(poison=True)
        c.check_backward(ref, mag)
        got = [t.clone() for t in (c.dx, c.dy, c.dw_post, c.dgate, c.dw_next)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_captured_and_replayed():
    c = Case(100, 256, "bf16", 30, seed=2)
    c.forward()
    c.backward()  # buffers exist, kernels are loaded
    args = (c.cfg, c.x, c.y, c.w_post, c.gate, c.w_next, c.out, c.h, c.r1, c.r2)
    back = (c.cfg, c.dout, c.dh, c.out, c.y, c.w_post, c.gate, c.w_next, c.r1, c.r2, c.dx, c.dy,
            c.dw_post, c.dgate, c.dw_next, c.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.moe_residual_norm_forward(*args)
        block.moe_residual_norm_backward(*back)
    for seed in (21, 22):
        fresh = Case(100, 256, "bf16", 30, seed=seed)
        for k in ("x", "y", "gate", "w_post", "w_next", "dout", "dh"):
            getattr(c, k).copy_(getattr(fresh, k))
        for t in (c.dgate, c.dw_post, c.dw_next, c.dx, c.dy, c.out, c.h):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check_forward(c.x, c.y)
        c.check_backward(c.reference(), c.reference(magnitudes=True))
    del graph
