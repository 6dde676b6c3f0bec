"""The dropout boundary's forward on rows that a cluster of CTAs shares.

A CTA's threads are whole warps, so that those of all but the last CTA have slots
past its slice whose columns are the next CTA's: nothing of them may reach the
row's statistics.  Values and bounds are those of test_gpu_drop."""
from __future__ import annotations

import pytest
import torch

from test_gpu_block import at_offset
from test_gpu_drop import BF16, F16, F32, _built, assert_within, check_bwd, check_fwd, drop_forward, make, mba, randn  # noqa: F401

pytestmark = pytest.mark.gpu

# widths of one to three CTAs a row, on 16-byte borders and off them
WIDE = pytest.mark.parametrize("dtype,H", [(F32, 8200), (F32, 8201), (F32, 10000), (F32, 11008), (F32, 16383), (F16, 14001),
                                           (F16, 16000), (BF16, 16401), (F16, 20000), (BF16, 32767), (BF16, 32768)])


def wide(rows, H, dtype, norm, beta, seed):
    v = make((rows, H), dtype, norm, True, beta, seed=seed)
    v["bias"] = randn((H,), seed=seed + 9, sc=2.0, loc=1.0)  # of the rows' own size
    return v


@WIDE
@pytest.mark.parametrize("norm,beta", [("rms", False), ("rms", True), ("layer", False), ("layer", True)])
def test_biases_of_the_rows_size(dtype, H, norm, beta):
    v = wide(3, H, dtype, norm, beta, H)
    for p in (0.0, 0.3):
        check_fwd(v, p, (3, 4), norm, what=f"{H} {norm}")
    check_bwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}")


@WIDE
def test_rows_of_equal_values(dtype, H):
    # their deviations are zero, so y is beta; x + bias is one value, rounded once
    x = torch.full((3, H), 100.25, dtype=dtype)
    f, bias, beta = torch.zeros(3, H, dtype=dtype), torch.full((H,), 200.7), randn((H,), seed=1)
    gamma = randn((H,), seed=2, sc=0.1, loc=1.0)
    h, y, st = mba.dropout_add_norm(f.cuda(), x.cuda(), p=0.0, rng=(0, 0), bias=bias.cuda(), norm="layer", gamma=gamma.cuda(),
                                    beta=beta.cuda(), want_stats=True)
    assert torch.equal(y.cpu(), beta.to(dtype).expand(3, H))
    assert torch.equal(st[1].cpu(), st[1][:1].cpu().expand(3)) and abs(float(st[1][0]) * 1e-5 ** 0.5 - 1) < 1e-6


@pytest.mark.parametrize("dtype,H,a", [(F32, 10000, 0), (F16, 20000, 1), (BF16, 32767, 3)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_off_the_borders(dtype, H, a, norm):
    v = wide(4, H, dtype, norm, True, H)
    h, y = (at_offset(torch.zeros(4, H, dtype=dtype), a + i)[0] for i in (1, 2))
    rstd = torch.empty(4, device="cuda")
    mba.dropout_add_norm_fwd(at_offset(v["f"], a)[0], at_offset(v["x"], a)[0], h, y, (None, rstd), p=0.3, rng=(5, 6), norm=norm,
                             bias=v["bias"].cuda(), gamma=v["gamma"].cuda(), beta=v["beta"].cuda())
    wh, wy, _, eh, ey = drop_forward(v["f"], v["x"], v["bias"], 0.3, (5, 6), norm, v["gamma"], v["beta"], 1e-5)
    assert_within(h, wh, eh, "h")
    assert_within(y, wy, ey, "y")


@pytest.mark.parametrize("dtype,H", [(BF16, 16401), (F32, 8201), (F16, 20000)])
@pytest.mark.parametrize("norm,beta", [("rms", False), ("layer", True)])
def test_several_rounds_of_a_cluster(dtype, H, norm, beta):
    # more rows than clusters fit the GPU: their exchange buffers in turn
    v = wide(500, H, dtype, norm, beta, H)
    check_fwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}")
    check_bwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}")
