"""8-bit experts on the GPU: quantisation exactly, the grouped products against
float64, the layer they make against its own steps in float64."""
import pytest
import torch

import block_ref as R
from expert_dispatch_gemm_b200 import block, moe
from expert_dispatch_gemm_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F32}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def check_quantized(x, q, s, rows=None):
    ws, wq = R.quantize(x)
    sel = slice(None) if rows is None else rows
    assert torch.equal(q.double()[sel], wq[sel])
    a, b = s.double()[sel], ws[sel]
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 3), (3, 16), (700, 128), (33, 1000), (64, 1024),
                                       (17, 1040), (9, 2048), (5, 7168), (3, 16385), (2, 32776),
                                       (2, 40_000), (3000, 64), (0, 64)])
def test_quantize_rows(rows, cols, dtype):
    x = (3 * torch.randn((rows, cols), generator=gen(rows + cols), device=DEV)).to(DT[dtype])
    q = torch.empty((rows, cols), dtype=torch.int8, device=DEV)
    s = torch.empty(rows, device=DEV)
    block.moe_quantize_rows(x, q, s)
    check_quantized(x, q, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_borders_and_odd_rows(dtype):
    dt = DT[dtype]
    # every bf16 value between two steps, ties among them, at many scales
    top = torch.tensor([1.0, 127.0, 254.0, 1.9921875, 3e-30, 1e37, 0.37], device=DEV)
    steps = torch.arange(-254, 255, device=DEV) / 2
    x = (top[:, None] * steps[None] / 127).to(dt)
    x[:, 0] = top.to(dt)
    bits = torch.arange(0x3f00, 0x4000, device=DEV, dtype=torch.int32) << 16
    y = bits.view(F32).to(dt)[None].repeat(7, 1)
    y[:, 0] = top.to(dt).clamp(2, 300)
    for t in (x, y, x[:, 1:500].contiguous()):
        q = torch.empty(t.shape, dtype=torch.int8, device=DEV)
        s = torch.empty(t.shape[0], device=DEV)
        block.moe_quantize_rows(t, q, s)
        check_quantized(t, q, s)
    z = torch.randn((6, 200), generator=gen(1), device=DEV).to(dt)
    z[0] = 0
    z[1, 7] = float("nan")
    z[2, 0] = float("-inf")
    z[3] *= 1e-40  # denormal
    z[4, 1:] = 0
    z[4, 0] = -0.0
    q = torch.empty(z.shape, dtype=torch.int8, device=DEV)
    s = torch.empty(6, device=DEV)
    block.moe_quantize_rows(z, q, s)
    check_quantized(z, q, s)
    assert s[0] == 0 and s[4] == 0 and torch.isnan(s[1:3]).all() and not q[:3].any()


@pytest.mark.parametrize("exponent", [-90, -3, 0, 11, 100])
def test_quantize_every_bf16_quotient(exponent):
    """Every bf16 significand as the row's maximum, with every bf16 value from
    the maximum down to 2^-10 of it beside it, both signs: the quotients that lie on
    a border among them."""
    top = (128 + torch.arange(128, device=DEV, dtype=torch.float64)) * 2.0 ** exponent
    bits = (128 + torch.arange(128, device=DEV, dtype=torch.float64))[None] * \
        2.0 ** (exponent - torch.arange(11, device=DEV, dtype=torch.float64))[:, None]
    x = bits.reshape(1, -1).repeat(128, 1)
    x = torch.where(x <= top[:, None], x, torch.zeros_like(x))
    x = torch.cat([top[:, None], x, -x], 1).to(BF)
    x = torch.cat([x, torch.zeros(128, -x.shape[1] % 8, dtype=BF, device=DEV)], 1)
    for t in (x, x[:, :-1].contiguous()):
        q = torch.empty(t.shape, dtype=torch.int8, device=DEV)
        s = torch.empty(128, device=DEV)
        block.moe_quantize_rows(t, q, s)
        check_quantized(t, q, s)


def test_quantize_groups_leave_other_rows():
    x = torch.randn((1000, 96), generator=gen(3), device=DEV).to(BF)
    q = torch.full((1000, 96), 77, dtype=torch.int8, device=DEV)
    s = torch.full((1000,), -5.0, device=DEV)
    starts, counts = [0, 3, 3, 128, 640, 999], [3, 0, 60, 300, 128, 1]
    block.moe_quantize_rows(x, q, s, i32(starts), i32(counts))
    hit = torch.zeros(1000, dtype=torch.bool, device=DEV)
    for a, n in zip(starts, counts):
        hit[a:a + n] = True
    check_quantized(x, q, s, hit)
    assert bool((q[~hit] == 77).all()) and bool((s[~hit] == -5).all())
    # groups that pass the end are cut, ones outside are skipped
    q.fill_(77)
    block.moe_quantize_rows(x, q, s, i32([990, 2000, -4]), i32([100, 5, 3]))
    assert bool((q[:990] == 77).all())
    check_quantized(x, q, s, slice(990, None))


def test_quantize_views_off_alignment():
    for dt in (BF, F32):
        store = torch.randn(64 * 50 + 1, generator=gen(4), device=DEV).to(dt)
        x = store[1:].view(50, 64)
        q = torch.empty(64 * 50 + 3, dtype=torch.int8, device=DEV)[3:].view(50, 64)
        s = torch.empty(50, device=DEV)
        block.moe_quantize_rows(x, q, s)
        check_quantized(x, q, s)


class Gemm:
    """A grouped product and its reference over the groups' rows."""

    def __init__(self, rows, k, o, act, dtype, starts=None, counts=None, groups=1, seed=1):
        g = gen(seed)
        i8 = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV,  # noqa: E731
                                      dtype=torch.int8)
        self.x, self.xs = i8(rows, k), torch.rand(rows, generator=g, device=DEV) + 0.1
        self.w = i8(groups, o, k)
        self.ws = (torch.rand((groups, o), generator=g, device=DEV) + 0.1) / (5000 * k ** 0.5)
        self.w3, self.s3 = (i8(groups, o, k), self.ws.flip(1).contiguous()) \
            if act == "swiglu" else (None, None)
        self.starts = None if starts is None else i32(starts)
        self.counts = None if counts is None else i32(counts)
        self.segments = [(0, rows)] if starts is None else list(zip(starts, counts))
        self.act, self.dt, self.rows = act, DT[dtype], rows
        self.cfg = block.gemm_i8_config(groups, rows, k, o, act, self.dt)
        self.out = torch.full((rows, o), 7.0, dtype=self.dt, device=DEV)
        self.space = block.gemm_i8_workspace(self.cfg, DEV)

    def run(self, stream=None):
        block.moe_gemm_i8(self.cfg, self.x, self.xs, self.starts, self.counts, self.w, self.ws,
                          self.w3, self.s3, self.out, self.space, stream)

    def check(self):
        hit = torch.zeros(self.rows, dtype=torch.bool, device=DEV)
        for g, (a, n) in enumerate(self.segments):
            n = max(0, min(n, self.rows - a))
            if n == 0:
                continue
            hit[a:a + n] = True
            x, xs = self.x[a:a + n].double(), self.xs[a:a + n].double()[:, None]
            u = x @ self.w[g].double().T * xs * self.ws[g].double()
            # sum to fp32, the scales' product, the product: three half steps
            du = 3 * R.U * u.abs()
            if self.act == "swiglu":
                v = x @ self.w3[g].double().T * xs * self.s3[g].double()
                want = R.act("swiglu", u, v)
                # exp(-u) in fp32: two steps and u's own error (its argument's
                # rounding counts |u|); |d silu| <= 1.1 |du|
                tol = (1.1 * du + (6 + 2 * u.abs()) * R.U * u.abs()) * v.abs() + \
                    u.abs() * 3 * R.U * v.abs()
            else:
                want = R.act(self.act, u)
                # gelu' <= 1.13; erf is good to two steps of 1
                tol = 1.2 * du + (6 * R.U * u.abs() if self.act == "gelu" else 0)
            tol = tol + R.half_step(self.dt) * want.abs() + 1e-37
            off = (self.out[a:a + n].double() - want).abs() - tol
            assert bool((off <= 0).all()), (g, off.max().item(), want.abs().max().item())
        assert bool((self.out[~hit] == 7.0).all())
        assert moe.moe_read_error(self.space) == (moe.MOE_OK, 0)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,o", [(1, 16, 16), (1, 2048, 272), (3, 48, 48), (16, 128, 256),
                                      (33, 1040, 512), (257, 256, 1008), (300, 640, 240)])
def test_one_group(rows, k, o, dtype, act):
    c = Gemm(rows, k, o, act, dtype, seed=rows + k + o)
    c.run()
    c.check()


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("starts,counts,rows", [
    ([0, 128, 128, 256, 512], [100, 0, 128, 255, 1], 640),      # aligned segments, one empty
    ([5, 17, 18, 300], [12, 1, 257, 31], 331),                  # any start, up to the last row
    ([0], [0], 128),                                            # nothing at all
    ([0, 512, 1024], [512, 272, 33], 1100),                     # several chunks a group
    ([700, 0], [400, 300], 900),                                # cut at the end, out of order
])
def test_groups(starts, counts, rows, dtype, act):
    c = Gemm(rows, 320, 336, act, dtype, starts, counts, len(starts), seed=rows)
    c.run()
    c.check()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,o,starts,counts,rows", [
    (1024, 256, [0], [256], 256),                 # the longest tile, K in four
    (1040, 272, [0], [193], 193),                 # a K block that ends early
    (4096, 1024, [3, 40], [37, 230], 270),        # two groups, one of a few rows
    (2000, 528, [0, 128, 128], [128, 0, 97], 256),  # an empty group
    (512, 4096, [0], [70], 128),                  # K in two
    (640, 1936, [0, 100, 250], [100, 150, 33], 283),
    (1024, 64, [5], [0], 128),                    # no rows at all
])
def test_split_reduction(k, o, starts, counts, rows, dtype, act):
    """Few tiles: K is split over the pairs of a cluster, which join their sums."""
    c = Gemm(rows, k, o, act, dtype, starts, counts, len(starts), seed=rows + k)
    c.run()
    c.check()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,o,starts,counts,rows", [
    (2048, 256, [0], [256], 256),                   # the longest tile, K in four
    (2064, 272, [0], [193], 193),                   # a K block that ends early
    (2064, 3584, [3], [1], 4),                      # as many tiles as are split in four
    (2064, 3600, [0], [70], 128),                   # one more, K in two (SwiGLU: whole)
    (4112, 1936, [0, 100, 250], [100, 150, 33], 283),
    (4096, 8192, [2], [5], 9),                      # as many as are split in two
    (4096, 8208, [2], [5], 9),                      # one more
    (4096, 64, [5], [0], 128),                      # no rows at all
    (16384, 256, [0, 7], [7, 1], 8),
])
def test_split_of_a_long_reduction(k, o, starts, counts, rows, dtype, act):
    """Both sides of each limit within which K is split."""
    c = Gemm(rows, k, o, act, dtype, starts, counts, len(starts), seed=rows + k + o)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,cols", [("bf16", c) for c in (256, 264, 496, 504, 512, 1024)] +
                         [("f32", c) for c in (128, 132, 508, 512, 516)])
@pytest.mark.parametrize("rows", [1, 37, 5000])
def test_quantize_rows_about_a_warps_share(rows, cols, dtype):
    test_quantize_rows(rows, cols, dtype)


def test_many_groups():
    counts = [(7 * g) % 41 for g in range(260)]
    starts, at = [], 0
    for n in counts:
        starts.append(at)
        at += n
    c = Gemm(at, 64, 96, "gelu", "bf16", starts, counts, 260, seed=5)
    c.run()
    c.check()


def test_extreme_sums_are_exact():
    """127 * 127 * K at the largest K: the accumulator does not saturate or wrap."""
    k = block.MOE_I8_MAX_K
    c = Gemm(2, k, 16, "none", "f32", seed=6)
    c.x.fill_(127)
    c.x[1] = -127
    c.w.fill_(127)
    c.w[0, 3] = -127
    c.xs.fill_(1.0)
    c.ws.fill_(1.0)
    c.run()
    want = float(127 * 127 * k)
    ref = torch.full((2, 16), want, device=DEV, dtype=torch.float64)
    ref[1] *= -1
    ref[:, 3] *= -1
    assert torch.equal(c.out.double(), ref.float().double())


def test_dead_rows_and_scales():
    """A row that was not finite (scale NaN) poisons itself only; a row of zeros gives zeros."""
    for act in ("none", "relu", "gelu", "swiglu"):
        c = Gemm(40, 128, 64, act, "bf16", seed=7)
        c.xs[3] = float("nan")
        c.xs[5] = 0.0
        c.run()
        assert torch.isnan(c.out[3]).all() and not c.out[5].any()
        keep = torch.ones(40, dtype=torch.bool, device=DEV)
        keep[3] = False
        assert torch.isfinite(c.out[keep]).all()


def test_streams_and_graphs():
    c = Gemm(300, 512, 256, "swiglu", "bf16", [0, 128], [100, 172], 2, seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(s)
    s.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed, counts in ((9, [128, 1]), (10, [0, 172])):
        fresh = Gemm(300, 512, 256, "swiglu", "bf16", [0, 128], counts, 2, seed=seed)
        for k in ("x", "xs", "w", "ws", "w3", "s3", "counts"):
            getattr(c, k).copy_(getattr(fresh, k))
        c.segments = fresh.segments
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    del graph


def test_two_at_once():
    """Two products on two streams, each with its own workspace."""
    a = Gemm(2000, 512, 1024, "none", "bf16", seed=11)
    b = Gemm(1500, 1024, 768, "swiglu", "bf16", seed=12)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a.run(s)
        b.run(t)
    torch.cuda.synchronize()
    a.check()
    b.check()


LAYERS = [wl.EC_FP32, wl.SMALL[1], wl.SMALL[2], wl.SMALL[3], wl.SMALL[4],
          wl.SMALL[4].replace(name="decode-n1", n=1, n_shared=2),
          wl.SMALL[3].replace(name="relu-shared", n=130, act="relu", n_shared=1)]


@pytest.mark.parametrize("w", LAYERS, ids=lambda w: w.name)
def test_quantized_layer(w):
    """Each step of a layer with 8-bit experts against float64 on what the
    step before it left, and the whole against the layer it came from."""
    inp = wl.make_inputs(w, DEV)
    q = block.QuantizedLayer(w, inp, DEV)
    out = q.forward(inp["X"])
    torch.cuda.synchronize()
    assert moe.moe_read_error(q.ws) == (moe.MOE_OK, 0)
    sz, r, dt = q.route.sizes, q.route, w.torch_dtype
    n_pad = (w.n + 127) // 128 * 128
    # dispatch: each token's bytes and scale on its rows
    ws, wq = R.quantize(inp["X"])
    rows, toks = [], []
    for t, lst in enumerate(r.tok_row.tolist()):
        for x in lst:
            if x >= 0:
                rows.append(x)
                toks.append(t)
    for s in range(w.n_shared):
        rows += [sz.shared_row_base + s * n_pad + t for t in range(w.n)]
        toks += range(w.n)
    rows, toks = torch.tensor(rows, device=DEV), torch.tensor(toks, device=DEV)
    assert torch.equal(q.Xq[rows].double(), wq[toks])
    assert torch.equal(q.xs[rows].double(), ws[toks])
    assert torch.equal(q.starts[:w.E], r.offsets[:w.E])
    assert torch.equal(q.counts[:w.E], r.counts)
    # experts: up, quantise, down on each group's rows
    for g, (a, c) in enumerate(zip(q.starts.tolist(), q.counts.tolist())):
        if c == 0:
            continue
        x, xs = q.Xq[a:a + c].double(), q.xs[a:a + c].double()[:, None]
        # the integer sums are exact in float64 (a sum of scaled products would
        # not be: where the integers cancel it leaves 1e-17 instead of 0)
        u = x @ q.W1[g].double().T * xs * q.s1[g].double()
        v = x @ q.W3[g].double().T * xs * q.s3[g].double() if q.W3 is not None else None
        h = R.act(w.act, u, v)
        # the terms a rounding is relative to: u v for the gate, u itself otherwise
        # (gelu is u/2 + u/2 erf, and for u < 0 the two cancel: its error is a few
        # steps of u, however small the difference; relu's terms are u or 0)
        size = u.abs() if v is None else (u * v).abs()
        tol = R.half_step(dt) * h.abs() + 16 * R.U * (1 + u.abs()) * size + 1e-37
        assert bool(((q.H[a:a + c].double() - h).abs() <= tol).all()), g
        check_quantized(q.H[a:a + c], q.Hq[a:a + c], q.hs[a:a + c])
        y = (q.Hq[a:a + c].double() @ q.W2[g].double().T) * q.hs[a:a + c].double()[:, None] * \
            q.s2[g].double()
        assert bool(((q.Y[a:a + c].double() - y).abs() <=
                     (R.half_step(dt) + 4 * R.U) * y.abs() + 1e-37).all()), g
    # the whole: quantisation noise of three operands, each below
    # max / 127 / sqrt(12) of its row; for Gaussian rows of 128 to 4096 the
    # maximum is under 5 standard deviations: 1.2% each, about 2% together (the
    # activation passes a relative error on, at most doubled for a product)
    ref = moe.Layer(w, inp, DEV)
    want = ref.forward().double()
    err = (out.double() - want).norm() / want.norm()
    assert err < 0.06, err
