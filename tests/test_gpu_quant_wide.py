"""The 8-bit norm on rows that a cluster of CTAs shares.

A CTA's threads are whole warps, so that those of all but the last CTA have slots
past its slice whose columns are the next CTA's: their parameters may not reach a
row's largest value.  Values and bounds are those of test_gpu_quant."""
from __future__ import annotations

import pytest
import torch

from test_gpu_drop import randn
from test_gpu_quant import BF16, F16, F32, _built, check_fwd, make, norm_quant  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = pytest.mark.parametrize("dtype,H", [(F32, 8200), (F32, 8201), (F32, 10000), (F32, 11008), (F32, 16383), (F16, 16001),
                                           (BF16, 16401), (F16, 20000), (BF16, 32767), (BF16, 32768)])


def opposed(rows, H, dtype, norm, seed):
    """Equal rows, with a beta that takes away most of every normalised value: each
    |y| is far below the |beta| beside it."""
    v = make((1, H), dtype, norm, residual=False, seed=seed)
    _, y, _, _, _ = norm_quant(v["x"], None, norm, v["gamma"], None, 1e-5)
    v["beta"] = (0.1 * randn((H,), seed=seed + 7).double() - y[0]).float()
    v["x"] = v["x"].expand(rows, H).contiguous()
    return v


@WIDE
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_betas_above_the_rows_values(dtype, H, norm):
    v = opposed(3, H, dtype, norm, H)
    for fmt, scaling, group in (("e4m3", "row", None), ("int8", "row", None), ("e5m2", "group", 128), ("int8", "pow2", 32)):
        check_fwd(v, norm, fmt, scaling, group, what=f"{H} {norm} {fmt} {scaling}", read=False)


@pytest.mark.parametrize("dtype,H", [(BF16, 16401), (F32, 8201), (F16, 20000)])
@pytest.mark.parametrize("norm,beta", [("rms", False), ("layer", True)])
def test_several_rounds_of_a_cluster(dtype, H, norm, beta):
    # more rows than clusters fit the GPU: their exchange buffers in turn
    v = make((500, H), dtype, norm, beta, seed=H)
    for fmt, scaling, group in (("e4m3", "row", None), ("int8", "group", 64)):
        check_fwd(v, norm, fmt, scaling, group, what=f"{H} {norm} {fmt} {scaling}", read=False)
