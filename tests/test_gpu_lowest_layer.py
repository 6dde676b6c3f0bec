"""Layer norms of rows whose squared deviations pass fp32 (a mask's lowest values
among them): the variance is infinite, so 1 / sqrt is 0 and y is beta, as in the
framework's Add+LayerNorm; infinities and NaN make the row NaN."""
from __future__ import annotations

import pytest
import torch

from _block_ref import U
from test_gpu_drop import BF16, F32, _built, mba, randn  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5
# a warp, several, a CTA, and several CTAs a row; on and off 16-byte borders
WIDTHS = [(F32, 40), (F32, 264), (BF16, 264), (BF16, 1001), (F32, 4096), (BF16, 4097), (F32, 11008), (BF16, 20000), (BF16, 32767)]


def rows(dtype, H):
    """Row 0 and the last are ordinary; what stands in the others."""
    x = randn((6, H), dtype, H)
    x[1, 7] = torch.finfo(dtype).min
    x[2, -1] = torch.finfo(dtype).max
    x[3, H // 2:H // 2 + 3] = 1e25
    x[4, :H // 2] = -1e30  # whole warps of one value
    return x


def outputs(x, gamma, beta):
    """(name, y, mean, rstd) of every operator with a layer norm of x."""
    z = torch.zeros_like(x)
    h, y, st = mba.block_norm(z, x, pre="layer", pre_gamma=gamma, pre_beta=beta, eps=EPS, want_stats=True)
    yield "block, pre", y, st[2], st[3]
    h, _, st = mba.block_norm(x, z, post="layer", post_gamma=gamma, post_beta=beta, pre=None, eps=EPS, want_stats=True)
    yield "block, post", h, st[0], st[1]
    h, y, st = mba.dropout_add_norm(z, x, p=0.0, rng=(0, 0), norm="layer", gamma=gamma, beta=beta, eps=EPS, want_stats=True)
    assert torch.equal(h, x) or x.isnan().any()
    yield "dropout", y, st[0], st[1]
    for scaling in ("row", "group"):
        r = mba.norm_quant(x, norm="layer", gamma=gamma, beta=beta, eps=EPS, scaling=scaling, want_stats=True)
        yield "8 bits, " + scaling, mba.dequantise(r.q, r.scale, dtype=F32), r.mean, r.rstd


@pytest.mark.parametrize("dtype,H", WIDTHS)
def test_rows_beyond_fp32s_squares_are_beta(dtype, H):
    x, gamma, beta = rows(dtype, H).cuda(), randn((H,), seed=1, loc=1.0).cuda(), randn((H,), seed=2).cuda()
    plain = x.clone()
    plain[1:5] = 0
    big = torch.tensor([False, True, True, True, True, False], device="cuda")
    only = [y for _, y, _, _ in outputs(torch.zeros_like(x), gamma, beta)]  # of rows of zeros: beta
    for (name, y, mean, rstd), (_, want, wmean, wrstd), b in zip(outputs(x, gamma, beta), outputs(plain, gamma, beta), only):
        assert (rstd[big] == 0).all(), name
        assert torch.equal(y[big], b[big]), name
        for got, w in ((y, want), (mean, wmean), (rstd, wrstd)):
            assert torch.equal(got[~big], w[~big]), name
        # sums of up to 32 values a thread, 5 levels and 128 parts, in fp32
        d = x.double()
        assert ((mean.double() - d.mean(-1)).abs() <= 64 * U * d.abs().mean(-1))[big].all(), name


@pytest.mark.parametrize("dtype,H", WIDTHS[1:])
def test_their_gradients(dtype, H):
    # 1 / sqrt is 0, so only what reaches h from elsewhere passes
    x, gamma = rows(dtype, H).cuda(), torch.ones(H, device="cuda")
    dy, dh = randn((6, H), dtype, 3).cuda(), randn((6, H), dtype, 4).cuda()
    h, y, st = mba.dropout_add_norm(torch.zeros_like(x), x, p=0.0, rng=(0, 0), norm="layer", gamma=gamma, eps=EPS, want_stats=True)
    g = mba.dropout_add_norm_backward(dy, dh, h, st, p=0.0, rng=(0, 0), norm="layer", gamma=gamma)
    assert torch.equal(g.dx[1:5], dh[1:5]) and torch.equal(g.df[1:5], dh[1:5]) and g.dgamma.isfinite().all()


@pytest.mark.parametrize("dtype,H", WIDTHS)
def test_infinities_and_nan_are_nan(dtype, H):
    x = rows(dtype, H)
    for i, v in enumerate((float("inf"), float("-inf"), float("nan")), 1):
        x[i, (i * 13) % H] = v
    bad = [False, True, True, True, False, False]
    for name, y, mean, rstd in outputs(x.cuda(), torch.ones(H, device="cuda"), torch.ones(H, device="cuda")):
        assert y.isnan().all(-1).tolist() == bad and y.isnan().any(-1).tolist() == bad, name
        assert rstd.isnan().tolist() == bad, name
