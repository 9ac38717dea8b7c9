"""8-bit products whose K is split over the pairs of a cluster: at least 16 blocks of
128 (SwiGLU in two: 32) and few tiles. (Of the shapes of test_gpu_i8's
test_split_reduction, those with K 2,000 and 4,096 are split; the shorter ones run
whole since the limits moved, though its comments say otherwise.)"""
import pytest
import torch

from test_gpu_block import CHECKED, _run
from test_gpu_i8 import Gemm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,o,groups,live,rows", [
    (2048, 256, 8, {3: 1}, 64),                       # in four: one live row of eight groups
    (2064, 272, 5, {0: 1, 4: 2}, 64),                 # the first and the last
    (4096, 512, 14, {13: 1, 2: 130}, 300),            # in two
    (4112, 336, 12, {}, 64),                          # no live row
    (4096, 4096, 2, {1: 61}, 64),                     # 32 tiles at most, 16 live
])
def test_split_reduction_of_few_live_groups(k, o, groups, live, rows, dtype, act):
    """The launch has a cluster for each tile that there could be; most have none."""
    counts = [live.get(g, 0) for g in range(groups)]
    starts, at = [], 0
    for n in counts:
        starts.append(at)
        at += n + 3  # (gaps between the groups, left as they are)
    assert at - 3 <= rows
    c = Gemm(rows, k, o, act, dtype, [min(s, rows) for s in starts], counts, groups,
             seed=k + groups)
    for _ in range(2):
        c.out.fill_(7.0)
        c.run()
        c.check()


@pytest.mark.skipif(CHECKED, reason="the driver of the checked run")
def test_checked_build_splits_too():
    """The split products in the checked build, in two and in four."""
    out = _run(["-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                "tests/test_gpu_i8.py", "tests/test_gpu_i8_split.py", "tests/test_gpu_i8_range.py",
                "-k", "split_of_a_long or few_live or scales_whose or silu"],
               MOE_LIBRARY="checked")
    assert " passed" in out and "failed" not in out


def test_scales_of_rows_behind_the_last_one_are_not_read():
    """Rows outside every group may hold anything: NaN scales, and bytes of no meaning."""
    for k in (1024, 2048, 4096):
        c = Gemm(70, k, 272, "none", "bf16", [2], [30], 1, seed=k)
        c.xs[:2] = float("nan")
        c.xs[32:] = float("nan")
        c.x[:2] = -128
        c.x[32:] = -128
        c.run()
        c.check()
        assert bool(torch.isfinite(c.out).all())
