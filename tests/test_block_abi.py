"""Host-side checks of libmoe_block (no GPU needed): its symbols, its structs,
and what it refuses before any launch."""
import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch

from expert_dispatch_gemm_b200 import block
from expert_dispatch_gemm_b200 import build as build_mod
from expert_dispatch_gemm_b200 import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_block.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG,
                                       moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def test_every_declared_symbol_is_exported():
    syms = sorted(set(re.findall(r"^MOE_API\s+[^(]*?\b(moe_\w+)\s*\(", open(HEADER).read(),
                                 flags=re.M)))
    assert sorted(block.API_SYMBOLS) == syms
    out = subprocess.run(["nm", "-D", "--defined-only", block.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert sorted(re.findall(r" T (moe_\w+)", out)) == syms


def test_struct_layouts_and_limits_match_the_header():
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "moe_block.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu %zu %zu %d %d %d %d\n", sizeof(moe_norm_config),
             offsetof(moe_norm_config, gate_stride), sizeof(moe_grad_tensor),
             offsetof(moe_grad_tensor, dtype), sizeof(moe_gemm_i8_config),
             sizeof(moe_dispatch_i8_config), offsetof(moe_dispatch_i8_config, dtype),
             MOE_NORM_MAX_D, MOE_I8_MAX_GROUPS, MOE_I8_MAX_K, MOE_I8_NONE);
      return 0;
    }
    """
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = [int(v) for v in subprocess.check_output([exe]).split()]
    assert got == [ctypes.sizeof(block.MoeNormConfig), block.MoeNormConfig.gate_stride.offset,
                   ctypes.sizeof(block.MoeGradTensor), block.MoeGradTensor.dtype.offset,
                   ctypes.sizeof(block.MoeGemmI8Config), ctypes.sizeof(block.MoeDispatchI8Config),
                   block.MoeDispatchI8Config.dtype.offset, block.MOE_NORM_MAX_D,
                   block.MOE_I8_MAX_GROUPS, block.MOE_I8_MAX_K, block.I8_ACTS["none"]]


def norm(**kw):
    c = block.norm_config(8, 64, torch.bfloat16, 1e-6)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("field,value,status", [
    ("n", 0, OK), ("n", -1, INVALID), ("n", (1 << 30) + 1, UNSUPPORTED), ("d", 0, INVALID),
    ("d", 16384, INVALID), ("d", 1, OK), ("dtype", 2, INVALID), ("eps", 0.0, INVALID),
    ("eps", -1.0, INVALID), ("eps", float("nan"), INVALID), ("eps", float("inf"), INVALID),
    ("gate_tokens", -1, INVALID), ("gate_stride", 63, INVALID), ("gate_stride", 1 << 40, OK)])
def test_norm_configs(field, value, status):
    assert block.norm_validate(norm(**{field: value})) == status  # (d 16384: the stride is 64)
    assert block.norm_validate(norm(d=16385, gate_stride=16385)) == UNSUPPORTED


def fake(i):
    """A 256-aligned address that is never read: validation fails first."""
    return 0x10000000 + (i << 16)


host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="hands fake device pointers to the library")


@host_only
def test_norm_calls_are_refused():
    L, c = block.lib(), norm()
    f = [fake(i) for i in range(20)]
    fwd = lambda *a: L.moe_residual_norm_forward(c, *a, None)  # noqa: E731
    for i in (0, 1, 5):  # x, y, out
        a = f[:9].copy()
        a[i - 0 if i < 5 else 5] = None
        assert fwd(*a) == INVALID
    a = f[:9].copy()
    a[6] = None  # w_next without h
    assert fwd(*a) == INVALID
    a = f[:9].copy()
    a[4] = None  # h without w_next
    assert fwd(*a) == INVALID
    a = f[:9].copy()
    a[6] = a[5]  # h is out
    assert fwd(*a) == INVALID
    a = f[:9].copy()
    a[0] += 1  # not on an element
    assert fwd(*a) == INVALID
    assert L.moe_norm_forward(c, None, f[1], f[2], None, None) == INVALID
    need = ctypes.c_size_t()
    assert L.moe_norm_workspace_size(c, ctypes.byref(need)) == OK and need.value >= 256
    bwd = lambda a, ws=fake(30), n=need.value: L.moe_residual_norm_backward(  # noqa: E731
        c, *a, ws, n, None)
    full = f[:14]
    assert bwd(full, None) == WORKSPACE
    assert bwd(full, fake(30) + 16) == WORKSPACE
    assert bwd(full, n=need.value - 1) == WORKSPACE
    # dout dh out y w_post gate w_next r_post r_next dx dy dw_post dgate dw_next
    for missing in ([0, 1], [1], [2], [3], [6], [7], [8], [9], [10], [11], [12], [13]):
        a = full.copy()
        for m in missing:
            a[m] = None
        assert bwd(a) == INVALID, missing
    a = full.copy()
    a[10] = a[9]  # dx is dy
    assert bwd(a) == INVALID
    assert L.moe_norm_backward(c, None, None, f[1], f[2], f[3], f[4], f[5], f[6], need.value,
                               None) == INVALID


@host_only
def test_grad_calls_are_refused():
    L = block.lib()
    need = ctypes.c_size_t()
    assert L.moe_grad_workspace_size(-1, ctypes.byref(need)) == INVALID
    sizes = []
    for n in (0, 1, 120, 121, 1000, 1001):
        assert L.moe_grad_workspace_size(n, ctypes.byref(need)) == OK
        sizes.append(need.value)
    assert sizes == sorted(sizes) and sizes[0] > 0

    def clip(count=1, max_norm=1.0, norm=fake(1), ws=fake(2), ws_bytes=1 << 20, **kw):
        t = (block.MoeGradTensor * 1)(block.MoeGradTensor(fake(3), fake(4), 10, moe.MOE_F32))
        for k, v in kw.items():
            setattr(t[0], k, v)
        return L.moe_grad_clip(t, count, max_norm, norm, ws, ws_bytes, None)

    assert clip(count=-1) == INVALID
    assert clip(max_norm=-1.0) == INVALID and clip(max_norm=float("nan")) == INVALID
    assert clip(norm=None) == INVALID and clip(norm=fake(1) + 2) == INVALID
    assert clip(ws=None) == WORKSPACE and clip(ws_bytes=8) == WORKSPACE
    assert clip(grad=None) == INVALID and clip(out=None) == INVALID
    assert clip(grad=fake(3) + 2) == INVALID and clip(dtype=5) == INVALID
    assert clip(numel=-1) == INVALID and clip(numel=1 << 43) == UNSUPPORTED
    assert L.moe_grad_clip(None, 1, 1.0, fake(1), fake(2), 1 << 20, None) == INVALID


@pytest.mark.parametrize("field,value,status", [
    ("groups", 0, INVALID), ("groups", 261, UNSUPPORTED), ("groups", 260, OK), ("rows", -1, INVALID),
    ("rows", 0, OK), ("rows", (1 << 30) + 1, UNSUPPORTED), ("k", 0, INVALID), ("k", 24, UNSUPPORTED),
    ("k", 65536, OK), ("k", 65552, UNSUPPORTED), ("n_out", 0, INVALID), ("n_out", 8, UNSUPPORTED),
    ("act", 4, INVALID), ("act", -1, INVALID), ("dtype", 2, INVALID)])
def test_gemm_i8_configs(field, value, status):
    c = block.gemm_i8_config(4, 256, 64, 64)
    setattr(c, field, value)
    assert block.gemm_i8_validate(c) == status


@host_only
def test_i8_calls_are_refused():
    L = block.lib()
    f = [fake(i) for i in range(12)]
    c = block.gemm_i8_config(4, 256, 64, 64)

    def gemm(cfg=c, ws=fake(20), n=256, **kw):
        a = dict(xq=f[0], xs=f[1], starts=f[2], counts=f[3], w=f[4], s=f[5], w3=None, s3=None,
                 out=f[6])
        a.update(kw)
        return L.moe_gemm_i8(cfg, *a.values(), ws, n, None)

    for k in ("xq", "xs", "starts", "counts", "w", "s", "out"):
        assert gemm(**{k: None}) == INVALID, k
    assert gemm(starts=None, counts=None) == INVALID  # four groups need them
    assert gemm(w3=f[7]) == INVALID and gemm(s3=f[7]) == INVALID  # not SwiGLU
    up = block.gemm_i8_config(4, 256, 64, 64, "swiglu")
    assert gemm(up) == INVALID and gemm(up, w3=f[7]) == INVALID
    for k in ("xq", "w", "out"):
        assert gemm(**{k: f[0] + 8}) == INVALID, k
    assert gemm(ws=None) == WORKSPACE and gemm(n=255) == WORKSPACE
    assert gemm(block.gemm_i8_config(4, 0, 64, 64)) == OK  # no rows: nothing to do

    def quant(rows=4, cols=64, dtype=moe.MOE_BF16, x=f[0], q=f[1], s=f[2], starts=None,
              counts=None, groups=0):
        return L.moe_quantize_rows(rows, cols, dtype, x, q, s, starts, counts, groups, None)

    assert quant(rows=-1) == INVALID and quant(cols=0) == INVALID and quant(dtype=3) == INVALID
    assert quant(rows=0, x=None) == OK
    for k in ("x", "q", "s"):
        assert quant(**{k: None}) == INVALID
    assert quant(x=f[0] + 1) == INVALID and quant(s=f[2] + 2) == INVALID
    assert quant(starts=f[3]) == INVALID and quant(counts=f[3]) == INVALID
    assert quant(starts=f[3], counts=f[4], groups=0) == INVALID
    assert quant(starts=f[3], counts=f[4], groups=261) == INVALID

    d = dict(n=8, d=64, E=4, n_shared=1, slots=2, rows=640, shared_row_base=512,
             dtype=moe.MOE_BF16)
    route = moe.MoeRouteOut(*[fake(40 + i) for i in range(14)])
    run = lambda x=f[0], q=f[1], r=route, **kw: L.moe_dispatch_i8(  # noqa: E731
        block.MoeDispatchI8Config(**{**d, **kw}), x, ctypes.byref(r), q, f[2], f[3], f[4], None)
    for k, v in (("n", 0), ("d", 24), ("E", 0), ("slots", 0), ("n_shared", 5), ("rows", 0),
                 ("rows", 600), ("shared_row_base", 520), ("dtype", 4), ("shared_row_base", -1)):
        assert run(**{k: v}) == INVALID, (k, v)
    assert run(E=257) == UNSUPPORTED and run(slots=257) == UNSUPPORTED
    assert run(x=None) == INVALID and run(x=f[0] + 8) == INVALID and run(q=f[1] + 8) == INVALID
    bad = moe.MoeRouteOut(*[fake(40 + i) for i in range(14)])
    bad.tok_row = None
    assert run(r=bad) == INVALID


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(8, 64)
    with pytest.raises(ValueError):
        block.moe_norm_forward(norm(), x, x[0], x)
    with pytest.raises(ValueError):
        block.moe_quantize_rows(x, x, x)
    with pytest.raises(ValueError):
        block.grad_list([x])
    with pytest.raises(TypeError):
        block.norm_config(8, 64, torch.float16, 1e-6)
    with pytest.raises(ValueError):
        block.gemm_i8_config(1, 1, 16, 16, act="tanh")


def test_binding_refuses_to_run_without_library(monkeypatch, tmp_path):
    monkeypatch.setattr(block, "LIB_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(block, "_LIB", None)
    with pytest.raises(RuntimeError, match="missing"):
        block.lib()
