"""Rows that a cluster of CTAs shares, with biases and betas, through the
bounds-checked build."""
from __future__ import annotations

import pytest

import test_gpu_drop_wide as dw
import test_gpu_quant_wide as qw
from test_gpu_drop_quant_checked import chk  # noqa: F401

pytestmark = pytest.mark.gpu


@dw.WIDE
def test_boundary(chk, dtype, H):  # noqa: F811
    for norm, beta in (("rms", False), ("rms", True), ("layer", True)):
        v = dw.wide(3, H, dtype, norm, beta, H)
        dw.check_fwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}")
        dw.check_bwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}")


@pytest.mark.parametrize("dtype,H,a", [(dw.F32, 10000, 0), (dw.F16, 20000, 1), (dw.BF16, 32767, 3)])
def test_boundary_off_the_borders(chk, dtype, H, a):  # noqa: F811
    for norm in ("rms", "layer"):
        dw.test_off_the_borders(dtype, H, a, norm)


@qw.WIDE
def test_quant(chk, dtype, H):  # noqa: F811
    for norm in ("rms", "layer"):
        v = qw.opposed(3, H, dtype, norm, H)
        for scaling, group in (("row", None), ("group", 128)):
            qw.check_fwd(v, norm, "e4m3", scaling, group, what=f"{H} {norm} {scaling}", read=False)


def test_several_rounds_of_a_cluster(chk):  # noqa: F811
    dw.test_several_rounds_of_a_cluster(dw.BF16, 16401, "layer", True)
    qw.test_several_rounds_of_a_cluster(qw.BF16, 16401, "layer", True)
