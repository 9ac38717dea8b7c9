"""Plain 64-bit forms of the block operators (include/moe_block.h), written from
their formulas on torch float64 tensors. Used by the tests only.

The error bounds beside them count roundings. u = 2^-24 is half an fp32 step;
an fp32 sum of the kernels is a chain of at most 32 elements a thread, 5
shuffle steps, 5 more over the warps, and a handful of products, so a row's sum
or a value made from a few of them is off by at most ROW = 64 u times the sum
of its terms' magnitudes.
"""
import torch

U = 2.0 ** -24
ROW = 64 * U


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gate_of(gate, n, tokens):
    """The gate row of each token, [n, d]; 1 without a gate."""
    if gate is None:
        return 1.0
    g = gate.double()
    if g.dim() == 1:
        g = g[None]
    t = torch.arange(n, device=g.device)
    return g[t // tokens if tokens else torch.zeros_like(t)]


def norm(v, w, off, eps):
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * r * (w.double() + off), r[:, 0]


def residual_norm(x, y, w_post, gate, w_next, *, eps, off=0.0, a=1.0, b=1.0, tokens=0):
    """out, h, r_post, r_next on float64 x, y (any of the last may be None)."""
    v, r1 = (y, None) if w_post is None else norm(y, w_post, off, eps)
    out = a * x + b * gate_of(gate, x.shape[0], tokens) * v
    h, r2 = (None, None) if w_next is None else norm(out, w_next, off, eps)
    return out, h, r1, r2


def residual_norm_backward(dout, dh, out, y, w_post, gate, w_next, r1, r2, *, off=0.0, a=1.0,
                           b=1.0, tokens=0, gate_rows=1, magnitudes=False):
    """dx, dy, dw_post, dgate, dw_next from the Jacobian of each norm,
    d(v r)/dv = r (I - v v^T r^2 / d); with `magnitudes` every term by its
    absolute value and every difference as a sum, which bounds the terms that
    the kernel adds up."""
    f = (lambda t: t.abs()) if magnitudes else (lambda t: t)
    minus = 1.0 if magnitudes else -1.0
    n, d = y.shape
    y = f(y)
    D = torch.zeros_like(y) if dout is None else f(dout)
    dw_next = dw_post = dgate = None
    if dh is not None:
        u = f(out) * r2[:, None]
        q = f(dh) * f(w_next.double() + off)
        D = D + r2[:, None] * (q + minus * u * (q * u).mean(1, keepdim=True))
        dw_next = (f(dh) * u).sum(0)
    g = gate_of(gate, n, tokens)
    g = f(g) if torch.is_tensor(g) else g
    a, b = (abs(a), abs(b)) if magnitudes else (a, b)
    v, w = y, 1.0
    if w_post is not None:
        w = f(w_post.double() + off)
        yr = y * r1[:, None]
        v = yr * w
        dw_post = (b * D * g * yr).sum(0)
    if gate is not None:
        which = torch.arange(n, device=y.device)
        which = which // tokens if tokens else torch.zeros_like(which)
        dgate = torch.zeros(gate_rows, d, dtype=torch.float64,
                            device=y.device).index_add_(0, which, b * D * v)
    dy = b * D * g
    if w_post is not None:
        p = dy * w
        dy = r1[:, None] * (p + minus * yr * (p * yr).mean(1, keepdim=True))
    return a * D, dy, dw_post, dgate, dw_next


def quantize(x):
    """scale (fp32 values) and integers of each row of a float tensor."""
    x = x.double()
    most = x.abs().amax(-1, keepdim=True)
    s = (most / 127).float().double()
    live = torch.isfinite(s) & (s > 0) & torch.isfinite(x).all(-1, keepdim=True)
    q = torch.where(live, torch.round(x / torch.where(live, s, 1.0)).clamp(-127, 127), 0.0)
    s = torch.where(torch.isfinite(x).all(-1, keepdim=True), s, torch.nan)
    return s[..., 0], q


def act(name, u, v=None):
    if name == "relu":
        return torch.where(u < 0, torch.zeros_like(u), u)
    if name == "gelu":
        return 0.5 * u * (1 + torch.erf(u / 2 ** 0.5))
    if name == "swiglu":
        return u / (1 + torch.exp(-u)) * v
    return u
