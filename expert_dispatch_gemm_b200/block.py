"""Thin Python binding of libmoe_block (include/moe_block.h): the operators of
the transformer block around the MoE layer, and the layer's experts in 8-bit
integers.

Argument checking and marshalling only, as in ``moe.py``, whose statuses,
errors, configs and workspaces it shares; every step runs in the library's CUDA
kernels on the stream given (default: the tensors' device's current stream). If
``libmoe_block.so`` is missing every call raises, there is no fallback.

``Block`` runs a layer between its norms, forward and backward, and clips its
gradients; ``QuantizedLayer`` serves a layer with 8-bit experts.
"""
from __future__ import annotations

import bisect
import contextlib
import ctypes
import os

import torch

from . import moe
from .moe import MOE_BF16, MOE_F32, MOE_OK, MoeError, RouteBuffers
from .workloads import Workload

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_LIBRARY=checked loads the checked build, as for libmoe
LIB_PATH = os.path.join(_PKG, "libmoe_block_checked.so"
                        if os.environ.get("MOE_LIBRARY") == "checked" else "libmoe_block.so")

# limits of include/moe_block.h
MOE_NORM_MAX_D = 16384
MOE_I8_MAX_GROUPS = 260
MOE_I8_MAX_K = 65536
MOE_WS_ERROR_BYTES = 256
I8_ACTS = {"relu": moe.MOE_ACT_RELU, "gelu": moe.MOE_ACT_GELU, "swiglu": moe.MOE_ACT_SWIGLU,
           "none": 3}

# every entry point include/moe_block.h declares
API_SYMBOLS = ["moe_norm_validate", "moe_norm_workspace_size", "moe_norm_forward",
               "moe_norm_backward", "moe_residual_norm_forward", "moe_residual_norm_backward",
               "moe_grad_workspace_size", "moe_grad_norm", "moe_grad_clip", "moe_quantize_rows",
               "moe_gemm_i8_validate", "moe_gemm_i8_workspace_size", "moe_gemm_i8",
               "moe_dispatch_i8"]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("gate_tokens", ctypes.c_int), ("gate_stride", ctypes.c_longlong)]


class MoeGradTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("numel", ctypes.c_longlong), ("dtype", ctypes.c_int)]


class MoeGemmI8Config(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int), ("rows", ctypes.c_int), ("k", ctypes.c_int),
                ("n_out", ctypes.c_int), ("act", ctypes.c_int), ("dtype", ctypes.c_int)]


class MoeDispatchI8Config(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("d", ctypes.c_int), ("E", ctypes.c_int),
                ("n_shared", ctypes.c_int), ("slots", ctypes.c_int), ("rows", ctypes.c_int),
                ("shared_row_base", ctypes.c_int), ("dtype", ctypes.c_int)]


_LIB = None
_FN = {}  # entry points by name, once loaded


def _functions() -> dict:
    L = lib()
    _FN.update({s: getattr(L, s) for s in API_SYMBOLS})
    return _FN


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _FN.clear()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m expert_dispatch_gemm_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, size, sizep = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        ncfg = ctypes.POINTER(MoeNormConfig)
        gcfg = ctypes.POINTER(MoeGemmI8Config)
        L.moe_norm_validate.argtypes = [ncfg]
        L.moe_norm_workspace_size.argtypes = [ncfg, sizep]
        L.moe_norm_forward.argtypes = [ncfg, P, P, P, P, P]
        L.moe_norm_backward.argtypes = [ncfg, P, P, P, P, P, P, P, P, size, P]
        L.moe_residual_norm_forward.argtypes = [ncfg] + [P] * 10
        L.moe_residual_norm_backward.argtypes = [ncfg] + [P] * 15 + [size, P]
        L.moe_grad_workspace_size.argtypes = [ctypes.c_int, sizep]
        tens = ctypes.POINTER(MoeGradTensor)
        L.moe_grad_norm.argtypes = [tens, ctypes.c_int, P, P, size, P]
        L.moe_grad_clip.argtypes = [tens, ctypes.c_int, ctypes.c_float, P, P, size, P]
        L.moe_quantize_rows.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, P, P, P,
                                        P, P, ctypes.c_int, P]
        L.moe_gemm_i8_validate.argtypes = [gcfg]
        L.moe_gemm_i8_workspace_size.argtypes = [gcfg, sizep]
        L.moe_gemm_i8.argtypes = [gcfg] + [P] * 10 + [size, P]
        L.moe_dispatch_i8.argtypes = [ctypes.POINTER(MoeDispatchI8Config), P,
                                      ctypes.POINTER(moe.MoeRouteOut), P, P, P, P, P]
        for s in API_SYMBOLS:
            getattr(L, s).restype = ctypes.c_int
        _LIB = L
    return _LIB


# ---------------------------------------------------------------------------
# argument checks
# ---------------------------------------------------------------------------

_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_TORCH = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _dtype(dt) -> int:
    if dt not in _DTYPES:
        raise TypeError(f"expected float32 or bfloat16, got {dt}")
    return _DTYPES[dt]


def _device_of(t) -> int:
    """The index of the CUDA device that a call's tensors have to be on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.get_device()


def _ptr(t, name, dtype, shape, dev, _Tensor=torch.Tensor):
    """The address of a tensor of this type, shape and device, or an error that
    says what is wrong with it. (One pass of cheap tests first: the calls of a
    decoded token take a few microseconds each.)"""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is missing")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _ptr(t, name, dtype, shape, dev)


def _ws(ws, dev):
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws: expected a torch.Tensor")
    return _ptr(ws, "ws", torch.uint8, (ws.numel(),), dev)


def _check_stream(stream, dev):
    if stream.device.index != dev:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on cuda:{dev}")


def _call(what, dev, stream, *args):
    """The entry point on the tensors' device and stream; raises MoeError."""
    fn = (_FN or _functions())[what]
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        _check_stream(stream, dev)
        raw = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != MOE_OK:
        raise MoeError(status, what)


_NOTHING = contextlib.nullcontext()


def _on(dev, stream):
    """The device and the stream of a sequence of calls, made current for it: the
    layer's calls (moe.py) take the current device as theirs, and a buffer made on
    the way belongs to the stream that it is used on."""
    if stream is not None:
        _check_stream(stream, dev)
        return torch.cuda.stream(stream)
    return _NOTHING if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _bytes(device, nbytes: int) -> torch.Tensor:
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


# ---------------------------------------------------------------------------
# residual norms
# ---------------------------------------------------------------------------

def norm_config(n: int, d: int, dtype, eps: float, weight_offset: float = 0.0,
                res_scale: float = 1.0, block_scale: float = 1.0, gate_tokens: int = 0,
                gate_stride: int | None = None) -> MoeNormConfig:
    return MoeNormConfig(n=n, d=d, dtype=_dtype(dtype), eps=eps, weight_offset=weight_offset,
                         res_scale=res_scale, block_scale=block_scale, gate_tokens=gate_tokens,
                         gate_stride=d if gate_stride is None else gate_stride)


def norm_gate_rows(cfg: MoeNormConfig) -> int:
    return -(-cfg.n // cfg.gate_tokens) if cfg.gate_tokens else 1


def norm_validate(cfg: MoeNormConfig) -> int:
    return lib().moe_norm_validate(cfg)


def norm_workspace(cfg: MoeNormConfig, device) -> torch.Tensor:
    """Workspace of the backward calls (one call at a time)."""
    nbytes = ctypes.c_size_t()
    _check(lib().moe_norm_workspace_size(cfg, ctypes.byref(nbytes)), "moe_norm_workspace_size")
    return _bytes(device, nbytes.value)


def _gate(t, name, cfg, dt, n, d, dev):
    """A gate or its gradient: [rows, d] (or [d] for one row) with unit column
    stride and cfg.gate_stride between rows."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    rows = -(-n // cfg.gate_tokens) if cfg.gate_tokens else 1
    if t.dtype is not dt:
        raise TypeError(f"{name}: expected {dt}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if t.shape != (rows, d) and not (rows == 1 and t.shape == (d,)):
        raise ValueError(f"{name}: expected shape {(rows, d)}, got {tuple(t.shape)}")
    if (d > 1 and t.stride(-1) != 1) or (rows > 1 and t.stride(0) != cfg.gate_stride):
        raise ValueError(f"{name}: strides {t.stride()} are not ({cfg.gate_stride}, 1)")
    return t.data_ptr()


_F32 = torch.float32


def moe_norm_forward(cfg: MoeNormConfig, x, w, h, rstd=None, stream=None):
    """h = norm(x): the pre-norm alone."""
    dev, dt, n, d = _device_of(x), _TORCH[cfg.dtype], cfg.n, cfg.d
    nd = (n, d)
    _call("moe_norm_forward", dev, stream, cfg, _ptr(x, "x", dt, nd, dev),
          _ptr(w, "w", _F32, (d,), dev), _ptr(h, "h", dt, nd, dev),
          _opt(rstd, "rstd", _F32, (n,), dev))


def moe_norm_backward(cfg: MoeNormConfig, dres, dh, x, w, rstd, dx, dw, ws, stream=None):
    """dx = dres + d<dh, norm(x)>/dx and dw (dres may be None)."""
    dev, dt, n, d = _device_of(x), _TORCH[cfg.dtype], cfg.n, cfg.d
    nd = (n, d)
    _call("moe_norm_backward", dev, stream, cfg, _opt(dres, "dres", dt, nd, dev),
          _ptr(dh, "dh", dt, nd, dev), _ptr(x, "x", dt, nd, dev), _ptr(w, "w", _F32, (d,), dev),
          _ptr(rstd, "rstd", _F32, (n,), dev), _ptr(dx, "dx", dt, nd, dev),
          _ptr(dw, "dw", _F32, (d,), dev), _ws(ws, dev), ws.numel())


def moe_residual_norm_forward(cfg: MoeNormConfig, x, y, w_post, gate, w_next, out, h=None,
                              rstd_post=None, rstd_next=None, stream=None):
    """out = res_scale x + block_scale gate * norm(y), h = norm(out); w_post,
    gate, w_next (with h) and the inverse norms may be None."""
    dev, dt, n, d = _device_of(x), _TORCH[cfg.dtype], cfg.n, cfg.d
    nd, n1, d1 = (n, d), (n,), (d,)
    _call("moe_residual_norm_forward", dev, stream, cfg, _ptr(x, "x", dt, nd, dev),
          _ptr(y, "y", dt, nd, dev), _opt(w_post, "w_post", _F32, d1, dev),
          _gate(gate, "gate", cfg, dt, n, d, dev), _opt(w_next, "w_next", _F32, d1, dev),
          _ptr(out, "out", dt, nd, dev), _opt(h, "h", dt, nd, dev),
          _opt(rstd_post, "rstd_post", _F32, n1, dev),
          _opt(rstd_next, "rstd_next", _F32, n1, dev))


def moe_residual_norm_backward(cfg: MoeNormConfig, dout, dh, out, y, w_post, gate, w_next,
                               rstd_post, rstd_next, dx, dy, dw_post, dgate, dw_next, ws,
                               stream=None):
    """Gradients of <dout, out> + <dh, h> (see include/moe_block.h for what may
    be None)."""
    dev, dt, n, d = _device_of(y), _TORCH[cfg.dtype], cfg.n, cfg.d
    nd, n1, d1 = (n, d), (n,), (d,)
    _call("moe_residual_norm_backward", dev, stream, cfg, _opt(dout, "dout", dt, nd, dev),
          _opt(dh, "dh", dt, nd, dev), _opt(out, "out", dt, nd, dev), _ptr(y, "y", dt, nd, dev),
          _opt(w_post, "w_post", _F32, d1, dev), _gate(gate, "gate", cfg, dt, n, d, dev),
          _opt(w_next, "w_next", _F32, d1, dev), _opt(rstd_post, "rstd_post", _F32, n1, dev),
          _opt(rstd_next, "rstd_next", _F32, n1, dev), _ptr(dx, "dx", dt, nd, dev),
          _ptr(dy, "dy", dt, nd, dev), _opt(dw_post, "dw_post", _F32, d1, dev),
          _gate(dgate, "dgate", cfg, dt, n, d, dev), _opt(dw_next, "dw_next", _F32, d1, dev),
          _ws(ws, dev), ws.numel())


# ---------------------------------------------------------------------------
# gradient norm and clip
# ---------------------------------------------------------------------------

class GradList:
    """The gradients of one moe_grad_norm / moe_grad_clip call, and where the
    clipped copies go (None: in place). Holds the tensors; their addresses are
    taken here, once. Outputs may not overlap, so a tensor that is listed twice needs
    two outputs of its own, for moe_grad_norm too, which leaves them alone."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients, {len(self.outs)} outputs")
        self.count = len(self.grads)
        self.device = self.grads[0].device if self.grads else None
        self.c = (MoeGradTensor * max(self.count, 1))()
        spans = []
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            for t in (g, o):
                if not isinstance(t, torch.Tensor) or not t.is_cuda:
                    raise ValueError(f"gradient {i}: expected CUDA tensors")
                if t.device != self.device:
                    raise ValueError(f"gradient {i} is on {t.device}, not on {self.device}")
                if not t.is_contiguous():
                    raise ValueError(f"gradient {i} must be contiguous")
            if o.dtype is not g.dtype or o.shape != g.shape:
                raise ValueError(f"gradient {i}: its output has another dtype or shape")
            n = g.numel()
            self.c[i] = MoeGradTensor(g.data_ptr(), o.data_ptr(), n, _dtype(g.dtype))
            if n:
                spans.append((o.data_ptr(), o.data_ptr() + n * o.element_size(), i))
        # what is written may meet nothing but its own gradient, whole
        spans.sort()
        for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"the outputs of gradients {i} and {j} overlap")
        firsts = [s[0] for s in spans]
        for i, g in enumerate(self.grads):
            a = g.data_ptr()
            b = a + g.numel() * g.element_size()
            for s in spans[max(bisect.bisect_right(firsts, a) - 1, 0):
                           bisect.bisect_left(firsts, b)]:
                if s[0] < b and a < s[1] and not (s[2] == i and s[:2] == (a, b)):
                    raise ValueError(f"the output of gradient {s[2]} overlaps gradient {i}")


def grad_list(grads, outs=None) -> GradList:
    return GradList(grads, outs)


def grad_workspace(grads: GradList, device) -> torch.Tensor:
    nbytes = ctypes.c_size_t()
    _check(lib().moe_grad_workspace_size(grads.count, ctypes.byref(nbytes)),
           "moe_grad_workspace_size")
    return _bytes(device, nbytes.value)


def _grad_call(what, grads: GradList, norm, ws, least, stream, *more):
    dev = _device_of(norm)
    if grads.device is not None and grads.device.index != dev:
        raise ValueError(f"norm is on {norm.device}, the gradients are on {grads.device}")
    if norm.numel() < least:
        raise ValueError(f"norm needs {least} elements")
    _call(what, dev, stream, grads.c, grads.count, *more,
          _ptr(norm, "norm", _F32, norm.shape, dev), _ws(ws, dev), ws.numel())


def moe_grad_norm(grads: GradList, norm, ws, stream=None):
    """norm[0] = the L2 norm over all gradients."""
    _grad_call("moe_grad_norm", grads, norm, ws, 1, stream)


def moe_grad_clip(grads: GradList, max_norm: float, norm, ws, stream=None):
    """norm[0] = the norm, norm[1] = the factor min(1, max_norm / (norm + 1e-6));
    the outputs receive the gradients times the factor."""
    _grad_call("moe_grad_clip", grads, norm, ws, 2, stream, max_norm)


# ---------------------------------------------------------------------------
# 8-bit experts
# ---------------------------------------------------------------------------

def gemm_i8_config(groups: int, rows: int, k: int, n_out: int, act: str = "none",
                   dtype=torch.bfloat16) -> MoeGemmI8Config:
    if act not in I8_ACTS:
        raise ValueError(f"unknown activation {act!r}")
    return MoeGemmI8Config(groups=groups, rows=rows, k=k, n_out=n_out, act=I8_ACTS[act],
                           dtype=_dtype(dtype))


def gemm_i8_validate(cfg: MoeGemmI8Config) -> int:
    return lib().moe_gemm_i8_validate(cfg)


def gemm_i8_workspace(cfg: MoeGemmI8Config, device, stream=None) -> torch.Tensor:
    """Workspace with a cleared error word (moe.moe_read_error reads it)."""
    nbytes = ctypes.c_size_t()
    _check(lib().moe_gemm_i8_workspace_size(cfg, ctypes.byref(nbytes)),
           "moe_gemm_i8_workspace_size")
    ws = _bytes(device, nbytes.value)
    with torch.cuda.device(ws.device):
        _check(moe.lib().moe_workspace_init(moe._ptr(ws), moe._stream(stream)),
               "moe_workspace_init")
    return ws


def _groups(starts, counts, dev):
    if (starts is None) != (counts is None):
        raise ValueError("starts and counts come together")
    if starts is None:
        return None, None, 0
    n = starts.numel()
    return (_ptr(starts, "starts", torch.int32, (n,), dev),
            _ptr(counts, "counts", torch.int32, (n,), dev), n)


def moe_quantize_rows(x, q, scale, starts=None, counts=None, stream=None):
    """q, scale = the rows of x [..., cols] in 8 bits with a scale each; with
    starts / counts only the groups' rows are read and written."""
    dev, shape, dt = _device_of(x), x.shape, x.dtype
    if not shape:
        raise ValueError("x needs at least one dimension")
    cols = shape[-1]
    rows = x.numel() // cols if cols else 0
    p0, p1, groups = _groups(starts, counts, dev)
    _call("moe_quantize_rows", dev, stream, rows, cols, _dtype(dt), _ptr(x, "x", dt, shape, dev),
          _ptr(q, "q", torch.int8, shape, dev), _ptr(scale, "scale", _F32, shape[:-1], dev), p0,
          p1, groups)


def moe_gemm_i8(cfg: MoeGemmI8Config, xq, x_scale, starts, counts, w, w_scale, w3, w3_scale, out,
                ws, stream=None):
    """out = act of the grouped 8-bit products (w3 / w3_scale only for SwiGLU;
    starts and counts None: one group of all rows)."""
    dev, i8 = _device_of(xq), torch.int8
    g, rows, k, o = cfg.groups, cfg.rows, cfg.k, cfg.n_out
    p0, p1, n = _groups(starts, counts, dev)
    if starts is not None and n != g:
        raise ValueError(f"starts and counts have {n} groups, the config {g}")
    wshape, sshape = (g, o, k), (g, o)
    _call("moe_gemm_i8", dev, stream, cfg, _ptr(xq, "xq", i8, (rows, k), dev),
          _ptr(x_scale, "x_scale", _F32, (rows,), dev), p0, p1, _ptr(w, "w", i8, wshape, dev),
          _ptr(w_scale, "w_scale", _F32, sshape, dev), _opt(w3, "w3", i8, wshape, dev),
          _opt(w3_scale, "w3_scale", _F32, sshape, dev),
          _ptr(out, "out", _TORCH[cfg.dtype], (rows, o), dev), _ws(ws, dev), ws.numel())


def dispatch_i8_config(cfg: moe.MoeConfig) -> MoeDispatchI8Config:
    """The dispatch of a layer config (sizes from moe_sizes)."""
    sz = moe.sizes(cfg)
    return MoeDispatchI8Config(n=cfg.n, d=cfg.d, E=cfg.E, n_shared=cfg.n_shared, slots=sz.slots,
                               rows=sz.rows, shared_row_base=sz.shared_row_base, dtype=cfg.dtype)


def moe_dispatch_i8(cfg: MoeDispatchI8Config, X, route: RouteBuffers, q, scale, starts, counts,
                    stream=None):
    """Each token quantised once and written to its dispatched rows (and its
    shared-expert rows); starts / counts = the groups of moe_gemm_i8."""
    dev, i32 = _device_of(X), torch.int32
    g = cfg.E + cfg.n_shared
    for name, shape in (("tok_row", (cfg.n, cfg.slots)), ("offsets", (cfg.E + 1,)),
                        ("counts", (cfg.E,))):
        _ptr(getattr(route, name), "route." + name, i32, shape, dev)
    _call("moe_dispatch_i8", dev, stream, cfg, _ptr(X, "X", _TORCH[cfg.dtype], (cfg.n, cfg.d), dev),
          ctypes.byref(route.c), _ptr(q, "q", torch.int8, (cfg.rows, cfg.d), dev),
          _ptr(scale, "scale", _F32, (cfg.rows,), dev), _ptr(starts, "starts", i32, (g,), dev),
          _ptr(counts, "counts", i32, (g,), dev))


# ---------------------------------------------------------------------------
# a layer with 8-bit experts, and a block
# ---------------------------------------------------------------------------

def quantize_weights(w, shared=None):
    """Expert weights [E, out, in] (and shared experts' [s, out, in], behind
    them) in 8 bits with a scale for each output channel."""
    total = w.shape[0] + (0 if shared is None else shared.shape[0])
    q = torch.empty((total, *w.shape[1:]), dtype=torch.int8, device=w.device)
    s = torch.empty((total, w.shape[1]), dtype=torch.float32, device=w.device)
    moe_quantize_rows(w, q[:w.shape[0]], s[:w.shape[0]])
    if shared is not None:
        moe_quantize_rows(shared, q[w.shape[0]:], s[w.shape[0]:])
    return q, s


class QuantizedLayer:
    """A layer for serving with its experts (routed and shared) in 8-bit
    integers: moe_route, moe_dispatch_i8, the up product with the activation,
    moe_quantize_rows on the hidden rows, the down product, moe_combine.
    The router stays in fp32. `inputs` as for moe.Layer; the expert weights are
    quantised here and not kept."""

    def __init__(self, w: Workload, inputs: dict, device, **cfg_override):
        self.w = w
        self.cfg = cfg = moe.config(w, **cfg_override)
        sz, dt, g = moe.sizes(cfg), w.torch_dtype, cfg.E + cfg.n_shared
        self.dispatch_cfg = dispatch_i8_config(cfg)
        self.up = gemm_i8_config(g, sz.rows, cfg.d, cfg.h, w.act, dt)
        self.down = gemm_i8_config(g, sz.rows, cfg.h, cfg.d, "none", dt)
        for c in (self.up, self.down):  # (d and h have to be multiples of 16)
            _check(gemm_i8_validate(c), "moe_gemm_i8_validate")
        self.Wg, self.logit_bias = inputs["Wg"], inputs.get("logit_bias")
        self.sel_bias = inputs.get("sel_bias")
        dev = _device_of(self.Wg)  # (moe_route's binding checks none of its operands)
        _ptr(self.Wg, "Wg", _F32, (cfg.d, cfg.E), dev)
        _opt(self.logit_bias, "logit_bias", _F32, (cfg.E,), dev)
        _opt(self.sel_bias, "sel_bias", _F32, (cfg.E,), dev)
        self.W1, self.s1 = quantize_weights(inputs["W1"], inputs.get("sW1"))
        self.W2, self.s2 = quantize_weights(inputs["W2"], inputs.get("sW2"))
        self.W3, self.s3 = (quantize_weights(inputs["W3"], inputs.get("sW3"))
                            if w.act == "swiglu" else (None, None))
        self.route = RouteBuffers(cfg, device)
        with _on(dev, None):
            self.ws = moe.workspace(cfg, device, layer=False)
        f32, i32, i8 = torch.float32, torch.int32, torch.int8
        self.Xq = torch.empty((sz.rows, cfg.d), dtype=i8, device=device)
        self.xs = torch.empty(sz.rows, dtype=f32, device=device)
        self.starts = torch.empty(g, dtype=i32, device=device)
        self.counts = torch.empty(g, dtype=i32, device=device)
        self.H = torch.empty((sz.rows, cfg.h), dtype=dt, device=device)
        self.Hq = torch.empty((sz.rows, cfg.h), dtype=i8, device=device)
        self.hs = torch.empty(sz.rows, dtype=f32, device=device)
        self.Y = torch.empty((sz.rows, cfg.d), dtype=dt, device=device)
        self.out = torch.empty((w.n, w.d), dtype=dt, device=device)

    def forward(self, X, stream=None):
        dev = _device_of(self.out)
        _ptr(X, "X", self.out.dtype, self.out.shape, dev)
        with _on(dev, stream):
            moe.moe_route(self.cfg, X, self.Wg, self.logit_bias, self.sel_bias, self.route,
                          self.ws, stream)
            moe_dispatch_i8(self.dispatch_cfg, X, self.route, self.Xq, self.xs, self.starts,
                            self.counts, stream)
            # the products share the routing workspace's error word
            moe_gemm_i8(self.up, self.Xq, self.xs, self.starts, self.counts, self.W1, self.s1,
                        self.W3, self.s3, self.H, self.ws, stream)
            moe_quantize_rows(self.H, self.Hq, self.hs, self.starts, self.counts, stream)
            moe_gemm_i8(self.down, self.Hq, self.hs, self.starts, self.counts, self.W2, self.s2,
                        None, None, self.Y, self.ws, stream)
            moe.moe_combine(self.cfg, self.Y, self.route, self.out, stream)
        return self.out


class Block:
    """A layer between its norms:

        h = norm(x; w_pre)                    pre-norm
        y = layer(h)                          moe.Layer (or QuantizedLayer: no backward)
        out = a x + b gate * norm(y; w_post)  residual norm
        h_next = norm(out; w_next)            the next block's pre-norm, fused

    params: optionally fp32 "w_pre" [d], "w_post" [d], "gate" (rows of the layer's
    dtype, see norm_config) and "w_next" [d]. A block without "w_pre" has no
    pre-norm of its own: it takes h beside x, as the block before it left it, and
    its backward pass gives "dx" (along the residual) and "dh" for that block:

        out, h = one.forward_train(x)              # one has "w_next"
        out, _ = two.forward_train(out, h=h)       # two has no "w_pre"
        g = two.backward_train(dout)
        g = one.backward_train(g["dx"], g["dh"])   # "dw_next" among its gradients

    A block keeps x and h themselves, not copies, until its backward pass; a layer
    keeps one forward's activations, so blocks that train have a layer each."""

    def __init__(self, layer, params: dict, eps: float = 1e-6, **norm):
        self.layer, self.p = layer, params
        w = layer.w
        self.cfg = norm_config(w.n, w.d, w.torch_dtype, eps, **norm)
        x = dict(dtype=w.torch_dtype, device=layer.out.device)
        f = dict(dtype=torch.float32, device=x["device"])
        self.pre = params.get("w_pre") is not None
        self.h = torch.empty((w.n, w.d), **x) if self.pre else None
        self.out = torch.empty((w.n, w.d), **x)
        self.h_next = torch.empty((w.n, w.d), **x) if params.get("w_next") is not None else None
        self.r_pre, self.r_post, self.r_next = (torch.empty(w.n, **f) for _ in range(3))
        self._g = None
        self._trained = False  # the last forward was forward_train()

    def _trains(self):
        if not hasattr(self.layer, "backward_train"):
            raise TypeError(f"a {type(self.layer).__name__} has no backward pass")

    def _tail(self, y, stream):
        p = self.p
        moe_residual_norm_forward(self.cfg, self.x, y, p.get("w_post"), p.get("gate"),
                                  p.get("w_next"), self.out, self.h_next,
                                  self.r_post if p.get("w_post") is not None else None,
                                  self.r_next if p.get("w_next") is not None else None, stream)
        return self.out, self.h_next

    def forward(self, x, stream=None, train=False, h=None):
        """(out, h_next). With train, the layer keeps what its backward needs."""
        if train:
            self._trains()
        self._trained = False
        if self.pre and h is not None:
            raise ValueError("h is given to a block that has a pre-norm of its own (w_pre)")
        dev = _device_of(self.out)
        if not self.pre:  # (the layer's binding checks no shapes)
            for name, t in (("x", x), ("h", h)):
                _ptr(t, name, self.out.dtype, self.out.shape, dev)
        if train:  # (the tail of this call writes them)
            mine = [t.data_ptr() for t in (self.out, self.h_next) if t is not None]
            for name, t in (("x", x), ("h", h)):
                if t is not None and t.numel() and t.data_ptr() in mine:
                    raise ValueError(f"{name} is an output of this block: it would be overwritten "
                                     "before the backward pass reads it")
        self.x = x
        if not self.pre:
            self.h = h
        self.layer._in_block = self  # whose forward its buffers hold
        with _on(dev, stream):
            if self.pre:
                moe_norm_forward(self.cfg, x, self.p["w_pre"], self.h, self.r_pre, stream)
            run = self.layer.forward_train if train else self.layer.forward
            res = self._tail(run(self.h, stream=stream), stream)
        self._trained = train
        return res

    def forward_train(self, x, stream=None, h=None):
        return self.forward(x, stream, train=True, h=h)

    def grads(self):
        """Gradient buffers (allocated once): "dx" ("dh" too, without a pre-norm), the
        norms' and the gate's, and the layer's own."""
        self._trains()
        if self._g is None:
            p, g = self.p, {"dx": torch.empty_like(self.out), "dy": torch.empty_like(self.out)}
            for k in ("w_pre", "w_post", "gate", "w_next"):
                t = p.get(k)  # (a gate's gradient has the gate's stride between rows)
                g["d" + k] = None if t is None else torch.empty_strided(
                    t.shape, t.stride(), dtype=t.dtype, device=t.device)
            self._nws = norm_workspace(self.cfg, self.out.device)
            with _on(_device_of(self.out), None):
                g["layer"] = self.layer.grads()
            g["dh"] = None if self.pre else g["layer"]["dX"]
            self._g = g
        return self._g

    def backward_train(self, dout, dh_next=None, stream=None):
        """Gradients of <dout, out> + <dh_next, h_next>, when the block's last forward
        was forward_train(). (A graph's replay is no call of this object's.)"""
        self._trains()
        if not self._trained:
            raise RuntimeError("backward_train() goes back through forward_train(): the last "
                               "forward of this block was none")
        if self.layer._in_block is not self:
            raise RuntimeError("another block has run this layer since: its activations are of "
                               "that forward")
        with _on(_device_of(self.out), stream):
            return self._backward(dout, dh_next, stream)

    def _backward(self, dout, dh_next, stream):
        p, g = self.p, self.grads()
        r_post = self.r_post if p.get("w_post") is not None else None
        r_next = self.r_next if p.get("w_next") is not None else None
        if p.get("w_next") is not None and dh_next is None:
            raise ValueError("dh_next is missing")
        moe_residual_norm_backward(self.cfg, dout, dh_next, self.out, self.layer.out,
                                   p.get("w_post"), p.get("gate"), p.get("w_next"), r_post,
                                   r_next, g["dx"], g["dy"], g["dw_post"], g["dgate"],
                                   g["dw_next"], self._nws, stream)
        lg = self.layer.backward_train(g["dy"], X=self.h, stream=stream)
        if self.pre:
            moe_norm_backward(self.cfg, g["dx"], lg["dX"], self.x, p["w_pre"], self.r_pre,
                              g["dx"], g["dw_pre"], self._nws, stream)
        return g

    def clip_grads(self, max_norm: float, stream=None):
        """Scales the parameters' gradients in place so that their global norm
        is at most max_norm; returns the device tensor [norm, factor], the same
        one at each call."""
        with _on(_device_of(self.out), stream):
            if not hasattr(self, "_clip"):
                g = self.grads()
                own = [g[k] for k in ("dw_pre", "dw_post", "dgate", "dw_next")]
                own += [t for k, t in g["layer"].items() if k not in ("dX", "dL")]
                own = [t for t in own if t is not None]
                # what lies between the rows of a strided gate's gradient is no gradient
                glist = grad_list([r for t in own
                                   for r in ([t] if t.is_contiguous() else t.unbind())])
                self._clip = (glist, torch.empty(2, dtype=torch.float32, device=self.out.device),
                              grad_workspace(glist, self.out.device))
            glist, norm, ws = self._clip
            moe_grad_clip(glist, max_norm, norm, ws, stream)
            return norm
