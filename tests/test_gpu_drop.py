"""Dropout alone and at the block boundary, forward and backward, against the
plain 64-bit forms of _drop_ref, which derives the bounds."""
from __future__ import annotations

import pytest
import torch

from _block_ref import U, assert_within
from _drop_ref import drop_backward, drop_forward, dropped, keep, scale
from test_gpu_block import at_offset, cuda

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import build
    build()
    yield
    torch.cuda.synchronize()
    assert mba.addln_get_device_error() == 0


def randn(shape, dtype=F32, seed=0, sc=1.0, loc=0.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sc + loc).to(dtype)


def check_drop(x, p, rng, got, start=0):
    # one product, the scale's rounding and the output's
    want = dropped(x, p, rng, start)
    assert_within(got, want, 2 * U * want.abs(), "dropout")
    assert torch.equal((got.cpu() == 0) | keep(x.numel(), p, rng, start).view(x.shape), torch.ones(x.shape, dtype=torch.bool))


def make(shape, dtype, norm, bias, beta, seed=0):
    H = shape[-1]
    v = {"f": randn(shape, dtype, seed, 0.7, 0.1), "x": randn(shape, dtype, seed + 1, 1.5, 0.1)}
    v["bias"] = randn((H,), seed=seed + 2, sc=0.2) if bias else None
    v["gamma"] = randn((H,), seed=seed + 3, sc=0.1, loc=1.0) if norm else None
    v["beta"] = randn((H,), seed=seed + 4, sc=0.1) if norm and beta else None
    return v


def check_fwd(v, p, rng, norm, eps=1e-5, what="", with_x=True, as_tensor=False):
    x = v["x"] if with_x else None
    r = torch.tensor(rng, device="cuda") if as_tensor else rng
    d = cuda(v)
    h, y, st = mba.dropout_add_norm(d["f"], d["x"] if with_x else None, p=p, rng=r, bias=d["bias"], norm=norm,
                                    gamma=d["gamma"], beta=d["beta"], eps=eps, want_stats=True)
    torch.cuda.synchronize()
    wh, wy, wst, eh, ey = drop_forward(v["f"], x, v["bias"], p, rng, norm, v["gamma"], v["beta"], eps)
    assert_within(h, wh, eh, what + " h")
    if norm is None:
        assert y is None and st == (None, None)
        return h, y, st
    assert_within(y, wy, ey, what + " y")
    dev = (wh - wh.mean(-1, keepdim=True)).abs().amax(-1, keepdim=True)
    for i, (g, w) in enumerate(zip(st, wst)):
        assert (g is None) == (w is None)
        if w is not None:
            err = U * (wh.abs().amax(-1, keepdim=True) + 8 * dev) if i == 0 else U * 24 * w
            err = err + eh.amax(-1, keepdim=True) * (1 if i == 0 else w * w) * 2  # h itself is off by eh
            assert_within(g, w.reshape(-1), err.reshape(-1), what + f" stat {i}")
    return h, y, st


def check_bwd(v, p, rng, norm, dy=True, dh=True, eps=1e-5, what="", as_tensor=False, seed=50):
    shape, dt = v["f"].shape, v["f"].dtype
    h, _, st, _, _ = drop_forward(v["f"], v["x"], v["bias"], p, rng, norm, v["gamma"], v["beta"], eps)
    h, st = h.to(dt), [None if t is None else t.reshape(-1).float() for t in st]
    dyt = randn(shape, dt, seed) if dy and norm else None
    dht = randn(shape, dt, seed + 1, 0.5) if dh else None
    want, err = drop_backward(dyt, dht, h, st, p, rng, norm, v["gamma"])
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    r = torch.tensor(rng, device="cuda") if as_tensor else rng
    d = cuda(v)
    g = mba.dropout_add_norm_backward(c(dyt), c(dht), c(h) if norm else None, tuple(map(c, st)), p=p, rng=r, bias=d["bias"],
                                      norm=norm, gamma=d["gamma"], beta=d["beta"])
    torch.cuda.synchronize()
    for k, t in g._asdict().items():
        if t is not None:
            assert_within(t, want[k].reshape(t.shape), err[k].reshape(t.shape), f"{what} {k}")
    assert (g.dbias is None) == (v["bias"] is None) and (g.dgamma is None) == (norm is None)
    return g


# ------------------------------------------------------------- dropout alone
@DTYPES
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 1000, 8191, 8192, 8193, 100003])
def test_dropout_sizes(dtype, n):
    x = randn((n,), dtype, n)
    for i, (p, rng) in enumerate([(0.1, (5, 6)), (0.5, (-3, (1 << 63) + 5)), (0.9, ((1 << 64) - 1, 1 << 40))]):
        check_drop(x, p, rng, mba.dropout(x.cuda(), p, rng))
        if rng[1] < 1 << 63 and rng[0] < 1 << 63:
            assert torch.equal(mba.dropout(x.cuda(), p, torch.tensor(rng, device="cuda")), mba.dropout(x.cuda(), p, rng))


@DTYPES
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 0), (0, 5), (2, 6)])
def test_dropout_off_the_borders(dtype, a, b):
    for n in (3, 40, 5000):
        x = randn((n,), dtype, n + a)
        y, whole = at_offset(torch.zeros(n, dtype=dtype), b)
        before = whole.clone()
        mba.dropout_fwd(at_offset(x, a)[0], y, 0.25, (1, 2))
        check_drop(x, 0.25, (1, 2), y)
        # nothing beside y was written
        y.zero_()
        assert torch.equal(whole.view(torch.uint8), before.view(torch.uint8))


@DTYPES
def test_dropout_in_place_and_shapes(dtype):
    x = randn((3, 5, 17), dtype, 1)
    y = x.cuda()
    mba.dropout_fwd(y, y, 0.3, (9, 9))
    check_drop(x, 0.3, (9, 9), y)
    # the mask goes by the index alone
    assert torch.equal(mba.dropout(x.cuda().view(-1), 0.3, (9, 9)), y.view(-1))
    assert mba.dropout(torch.empty(0, 4, device="cuda", dtype=dtype), 0.3, (9, 9)).shape == (0, 4)
    assert mba.dropout(torch.ones((), device="cuda", dtype=dtype), 0.0, (9, 9)).item() == 1.0


@DTYPES
def test_p_of_zero_one_and_too_small(dtype):
    x = randn((1003,), dtype, 2)
    x[5], x[6], x[7] = float("inf"), float("nan"), -0.0
    c = x.cuda()
    for p in (0.0, 2.0 ** -18):
        assert torch.equal(mba.dropout(c, p, (1, 1)).cpu().view(torch.uint8), x.view(torch.uint8))
    for p in (1.0, 1 - 2.0 ** -18):
        assert torch.equal(mba.dropout(c, p, (1, 1)).cpu().double(), torch.zeros(1003, dtype=torch.float64))


@DTYPES
def test_dropped_infinities_and_nan_are_zero(dtype):
    n, p, rng = 4000, 0.4, (77, 3)
    k = keep(n, p, rng)
    for bad in (float("inf"), float("-inf"), float("nan"), torch.finfo(dtype).min):
        y = mba.dropout(torch.full((n,), bad, dtype=dtype, device="cuda"), p, rng).cpu().double()
        assert (y[~k] == 0).all()
        assert (y[k].isnan() if bad != bad else y[k] != 0).all()


@pytest.mark.slow
def test_dropout_past_32_bits():
    n = (1 << 32) + 13
    x = torch.ones(n, dtype=BF16, device="cuda")
    mba.dropout_fwd(x, x, 0.5, (3, 4))
    for start, m in ((0, 100), ((1 << 32) - 50, 63), ((1 << 31) - 5, 40)):
        assert torch.equal(x[start:start + m].cpu() != 0, keep(m, 0.5, (3, 4), start))


@pytest.mark.slow
def test_blocks_past_32_bits():
    # more than 2^32 blocks of 8 elements, alone and at the boundary
    rows, H = (1 << 20) + 8, 32768
    n = rows * H
    if torch.cuda.mem_get_info()[0] < 3 * n:
        pytest.skip("not enough device memory")
    x = torch.empty(rows, H, dtype=BF16, device="cuda")
    for f in (lambda: mba.dropout_fwd(x, x, 0.5, (3, 4)),
              lambda: mba.dropout_add_norm_fwd(x, None, x, p=0.5, rng=(3, 4), norm=None)):
        x.fill_(1)
        f()
        for start in (0, (1 << 35) - 40, (1 << 35) + 3 * H, n - 100):
            assert torch.equal(x.view(-1)[start:start + 100].cpu() != 0, keep(100, 0.5, (3, 4), start))


# ------------------------------------------------------------- the boundary
WIDTHS = [1, 2, 7, 8, 12, 31, 33, 64, 100, 250, 256, 264, 516, 768, 1000, 1001, 2050, 4096, 4097, 4104, 8192]
KINDS = [("layer", True, True), ("rms", False, False), (None, True, False), ("rms", True, True), ("layer", False, False),
         (None, False, False), ("layer", True, False), ("rms", False, True)]


@DTYPES
@pytest.mark.parametrize("i,H", list(enumerate(WIDTHS)))
def test_widths(dtype, i, H):
    for j, rows in enumerate((5, 1, 3, 2)):
        norm, bias, beta = KINDS[(i + j) % len(KINDS)]
        v = make((rows, H), dtype, norm, bias, beta, seed=100 * i + j)
        what, rng = f"{rows}x{H} {norm} bias {bias} beta {beta}", (1000 + i, (1 << 33) * j + i)
        check_fwd(v, 0.3, rng, norm, what=what, with_x=j != 1, as_tensor=j == 2)
        check_bwd(v, 0.3, rng, norm, what=what, dy=True, dh=j != 3 or norm is None, as_tensor=j == 0)


@pytest.mark.parametrize("dtype,H", [(F32, 8193), (F32, 16384), (F16, 16400), (BF16, 32767), (BF16, 32768)])
@pytest.mark.parametrize("norm,full", [("layer", True), ("rms", False)])
def test_longest_rows(dtype, H, norm, full):
    v = make((3, H), dtype, norm, full, full, seed=H)
    check_fwd(v, 0.1, (1, 2), norm, what=f"{H}")
    check_bwd(v, 0.1, (1, 2), norm, what=f"{H}")


@pytest.mark.parametrize("rows,H,dtype", [(1200, 64, F32), (1216, 96, BF16), (700, 40, F16), (1000, 1001, BF16),
                                          (640, 4104, F16), (1100, 768, F16)])
@pytest.mark.parametrize("norm,bias,beta", KINDS[:5])
def test_many_rows(rows, H, dtype, norm, bias, beta):
    v = make((rows, H), dtype, norm, bias, beta, seed=rows)
    check_fwd(v, 0.1, (11, 12), norm, what=f"{rows}x{H} {norm}")
    check_bwd(v, 0.1, (11, 12), norm, dh=norm is None, what=f"{rows}x{H} {norm}")


@DTYPES
@pytest.mark.parametrize("p", [0.0, 2.0 ** -16, 0.5, 0.999, 1.0])
def test_probabilities(dtype, p):
    for H in (768, 1001):
        v = make((6, H), dtype, "layer", True, True, seed=H)
        check_fwd(v, p, (21, 22), "layer", what=f"p {p}")
        check_bwd(v, p, (21, 22), "layer", what=f"p {p}")


@DTYPES
def test_mask_is_that_of_dropout(dtype):
    f = randn((7, 1001), dtype, 3)
    h, y, st = mba.dropout_add_norm(f.cuda(), p=0.2, rng=(5, 6), norm=None)
    assert y is None and st is None
    assert torch.equal(h, mba.dropout(f.cuda(), 0.2, (5, 6)))
    # the stream's shape does not matter, its indexes do
    h2, _, _ = mba.dropout_add_norm(f.cuda().view(7, 7, 143), p=0.2, rng=(5, 6), norm=None)
    assert torch.equal(h2.view(-1), h.view(-1))


@DTYPES
def test_dropped_values_do_not_reach_the_row(dtype):
    # infinities and NaN where the mask drops them change nothing
    v = make((4, 264), dtype, "layer", False, True, seed=8)
    k = keep(4 * 264, 0.5, (3, 3)).view(4, 264)
    f2 = v["f"].clone()
    f2[~k] = torch.tensor([float("nan"), float("inf"), torch.finfo(dtype).min] * 400, dtype=dtype)[:int((~k).sum())]
    a = mba.dropout_add_norm(v["f"].cuda(), v["x"].cuda(), p=0.5, rng=(3, 3), gamma=v["gamma"].cuda())
    b = mba.dropout_add_norm(f2.cuda(), v["x"].cuda(), p=0.5, rng=(3, 3), gamma=v["gamma"].cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@DTYPES
def test_lowest_values(dtype):
    # a mask's lowest values in the stream: where the sum of squares passes fp32,
    # 1 / rms is 0 and so is the row
    low = torch.finfo(dtype).min
    x = randn((3, 264), dtype, 1)
    x[1, 40:200] = low
    f, w = torch.zeros(3, 264, dtype=dtype), torch.ones(264)
    h, y, st = mba.dropout_add_norm(f.cuda(), x.cuda(), p=0.5, rng=(1, 2), norm="rms", gamma=w.cuda(), want_stats=True)
    assert torch.equal(h.cpu(), x)
    if dtype is F16:
        wh, wy, _, eh, ey = drop_forward(f, x, None, 0.5, (1, 2), "rms", w, None, 1e-5)
        assert_within(y, wy, ey, "y")
    else:
        assert st[1][1] == 0 and not y[1].any() and y[0].any()


@DTYPES
@pytest.mark.parametrize("H", [5, 520, 768, 4099])
def test_off_the_borders_and_given_outputs(dtype, H):
    v = make((6, H), dtype, "layer", True, True, seed=H)
    vec = lambda k, o: at_offset(v[k], o)[0]  # noqa: E731
    h, hw = at_offset(torch.zeros(6, H, dtype=dtype), 3)
    y, yw = at_offset(torch.zeros(6, H, dtype=dtype), 4)
    before = hw.clone(), yw.clone()
    kw = dict(p=0.3, rng=(8, 9), norm="layer")
    mba.dropout_add_norm_fwd(vec("f", 1), vec("x", 2), h, y, bias=vec("bias", 1), gamma=vec("gamma", 3), beta=vec("beta", 2), **kw)
    wh, wy, st, eh, ey = drop_forward(v["f"], v["x"], v["bias"], 0.3, (8, 9), "layer", v["gamma"], v["beta"], 1e-5)
    assert_within(h, wh, eh, "h")
    assert_within(y, wy, ey, "y")
    hs, st = wh.to(dtype), [t.reshape(-1).float() for t in st]
    dy = randn((6, H), dtype, 5)
    want, err = drop_backward(dy, None, hs, st, 0.3, (8, 9), "layer", v["gamma"])
    outs = {k: at_offset(torch.zeros(6, H, dtype=dtype), 5 + i) for i, k in enumerate(("df", "dx"))}
    outs |= {k: at_offset(torch.zeros(H), 1 + i) for i, k in enumerate(("dbias", "dgamma", "dbeta"))}
    olds = {k: w.clone() for k, (_, w) in outs.items()}
    mba.dropout_add_norm_bwd(at_offset(dy, 9)[0], None, at_offset(hs, 10)[0], tuple(t.cuda() for t in st), outs["df"][0],
                             outs["dx"][0], gamma=vec("gamma", 1), **{k: outs[k][0] for k in ("dbias", "dgamma", "dbeta")}, **kw)
    for k, (t, w) in outs.items():
        assert_within(t, want[k].reshape(t.shape), err[k].reshape(t.shape), k)
        t.zero_()
        assert torch.equal(w, olds[k]), f"beside {k}"
    h.zero_(), y.zero_()
    assert torch.equal(hw, before[0]) and torch.equal(yw, before[1])


@DTYPES
@pytest.mark.parametrize("H", [768, 1001])
def test_in_place(dtype, H):
    v = make((40, H), dtype, "rms", True, False, seed=4)
    d = cuda(v)
    kw = dict(p=0.3, rng=(8, 9), norm="rms", gamma=d["gamma"], bias=d["bias"])
    h, y, st = mba.dropout_add_norm(d["f"], d["x"], want_stats=True, **kw)
    f, x = d["f"].clone(), d["x"].clone()
    mba.dropout_add_norm_fwd(f, x, x, f, **kw)
    assert torch.equal(x, h) and torch.equal(f, y)
    y2 = torch.empty_like(y)
    mba.dropout_add_norm_fwd(d["f"], d["x"], None, y2, **kw)  # h is not wanted
    assert torch.equal(y2, y)
    dy, dh = randn((40, H), dtype, 6).cuda(), randn((40, H), dtype, 7).cuda()
    kw.pop("bias")
    g = mba.dropout_add_norm_backward(dy, dh, h, st, **kw)
    a, b = dy.clone(), h.clone()
    mba.dropout_add_norm_bwd(a, dh, b, st, b, a, **kw)
    assert torch.equal(b, g.df) and torch.equal(a, g.dx)
    a = dh.clone()
    mba.dropout_add_norm_bwd(dy, a, h, st, a, None, **kw)  # dx is not wanted
    assert torch.equal(a, g.df)


def test_without_dy_the_norm_has_zero_gradients():
    v = make((9, 300), F32, "layer", True, True, seed=1)
    d = cuda(v)
    dh = randn((9, 300), seed=2).cuda()
    g = mba.dropout_add_norm_backward(None, dh, None, None, p=0.1, rng=(1, 2), **{k: d[k] for k in ("bias", "gamma", "beta")})
    assert not g.dgamma.any() and not g.dbeta.any() and torch.equal(g.dx, dh)
    assert torch.equal(g.df, mba.dropout(dh, 0.1, (1, 2)))


def test_no_rows():
    e = torch.empty(0, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda")
    h, y, st = mba.dropout_add_norm(e, e, p=0.1, rng=(1, 2), gamma=w, want_stats=True)
    assert h.shape == y.shape == (0, 64) and st[1].shape == (0,)
    g = mba.dropout_add_norm_backward(e, None, h, st, p=0.1, rng=(1, 2), gamma=w, bias=w, beta=w)
    assert not (g.dbias.any() or g.dgamma.any() or g.dbeta.any())


@pytest.mark.slow
def test_rows_past_32_bits():
    # 66000 x 32768 is above 2^31 elements; rows on both sides of the border
    rows, H = 66000, 32768
    f = torch.zeros(rows, H, dtype=BF16, device="cuda")
    x = torch.zeros_like(f)
    at = [0, 65535, 65536, rows - 1]
    part = randn((4, H), BF16, 3)
    f[at] = part.cuda()
    gamma = randn((H,), seed=4, loc=1.0)
    h, y, st = mba.dropout_add_norm(f, x, p=0.5, rng=(6, 7), norm="rms", gamma=gamma.cuda(), want_stats=True)
    del f
    x[at] = part.cuda()
    df = torch.empty_like(x)
    mba.dropout_add_norm_bwd(None, x, None, None, df, None, p=0.5, rng=(6, 7), norm=None)
    for i, r in enumerate(at):
        wh, wy, _, eh, ey = drop_forward(part[i:i + 1], None, None, 0.5, (6, 7), "rms", gamma, None, 1e-5, start=r * H)
        assert_within(h[r:r + 1], wh, eh, f"h {r}")
        assert_within(y[r:r + 1], wy, ey, f"y {r}")
        assert torch.equal(df[r], h[r])


# ------------------------------------------------------------------- autograd
@pytest.mark.parametrize("norm", ["layer", "rms", None])
@pytest.mark.parametrize("shape", [(6, 5, 264), (8, 1001)])
def test_autograd_against_the_formula_and_differences(norm, shape):
    v = make(shape, F32, norm, True, norm is not None, seed=3)
    names = [k for k in ("f", "x", "bias", "gamma", "beta") if v[k] is not None]
    leaf = {k: v[k].cuda().requires_grad_(True) for k in names}
    wy, wh = randn(shape, seed=60), randn(shape, seed=61, sc=0.5)
    rng = torch.tensor([4, 5], device="cuda")
    kw = {k: leaf.get(k) for k in ("bias", "gamma", "beta")}
    h, y = mba.dropout_add_norm_train(leaf["f"], leaf["x"], p=0.2, rng=rng, norm=norm, **kw)
    rng += 1  # the backward keeps the call's own
    loss = (h * wh.cuda()).sum() + (0 if y is None else (y * wy.cuda()).sum())
    loss.backward()
    k = keep(wy.numel(), 0.2, (4, 5)).view(shape) * scale(0.2)

    def plain(t):
        h = t["x"] + k * (t["f"] + t["bias"])
        L = (h * wh.double()).sum()
        if norm is not None:
            c = h - h.mean(-1, keepdim=True) if norm == "layer" else h
            n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * t["gamma"] + t["beta"]
            L = L + (n * wy.double()).sum()
        return L

    ref = {n: v[n].double().requires_grad_(True) for n in names}
    plain(ref).backward()
    for n in names:
        got, want = leaf[n].grad.cpu().double(), ref[n].grad
        # sums of up to 1001 fp32 terms, rounded at 32 u of their magnitudes' mean
        assert (got - want).abs().max() < 1e-4 * (1 + want.abs().max()), n
        # along one direction, central differences in 64 bits: off by a third
        # derivative times 1e-10, of terms that are of the size of the sum below
        with torch.no_grad():
            d = randn(v[n].shape, seed=70).double()
            e = 1e-5
            two = [plain({**{m: ref[m] for m in names}, n: ref[n] + s * e * d}) for s in (1, -1)]
            slope = float(two[0] - two[1]) / (2 * e)
        assert abs(float((got * d).sum()) - slope) < 1e-4 * (1 + float((want * d).abs().sum())), n


def test_dropout_train():
    x = randn((50, 33), seed=1).cuda().requires_grad_(True)
    y = mba.dropout_train(x, 0.3, (1, 2))
    w = randn((50, 33), seed=2).cuda()
    (y * w).sum().backward()
    assert torch.equal(x.grad, mba.dropout(w, 0.3, (1, 2)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_module(dtype):
    m = mba.FusedDropoutAddNorm(264, p=0.25, input_bias=True, device="cuda")
    f, x = randn((12, 264), dtype, 1).cuda(), randn((12, 264), dtype, 2).cuda()
    seed = int(m.rng[0])
    first, second = m(f, x)[0], m(f, x)[0]
    assert int(m.rng[1]) == 2 and not torch.equal(first, second)
    again = m(f, x, rng=(seed, 0))[0]
    assert torch.equal(first, again) and int(m.rng[1]) == 2
    m.eval()
    h, y = m(f, x)
    assert int(m.rng[1]) == 2
    assert torch.equal(h, (f.float() + x.float()).to(dtype))
    m.train()
    fr = f.clone().requires_grad_(True)
    (m(fr, x)[1].float() ** 2).sum().backward()
    assert fr.grad is not None and all(p.grad is not None for p in m.parameters())


def test_captured_training_step():
    # each replay draws the next mask, and its backward uses the same one
    torch.manual_seed(0)
    m = mba.FusedDropoutAddNorm(768, p=0.5, norm="rms", bias=False, device="cuda")
    f = randn((64, 768), seed=1).cuda().requires_grad_(True)
    x = randn((64, 768), seed=2).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            f.grad = m.weight.grad = None
            h, y = m(f, x)
            (y * y).sum().backward()
        del h, y
    torch.cuda.current_stream().wait_stream(s)
    f.grad = m.weight.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, y = m(f, x)
        (y * y).sum().backward()
    seed, at, seen = int(m.rng[0]), int(m.rng[1]), []
    for i in range(3):
        f.grad.zero_(), m.weight.grad.zero_()
        g.replay()
        torch.cuda.synchronize()
        k = keep(64 * 768, 0.5, (seed, at + i)).view(64, 768)
        assert torch.equal(h.cpu() == x.cpu(), ~k)
        assert torch.equal(f.grad.cpu() == 0, ~k)
        seen.append(h.clone())
    assert not torch.equal(seen[0], seen[1]) and int(m.rng[1]) == at + 3


def test_other_streams_and_repeats():
    v = make((333, 1001), BF16, "layer", True, True, seed=5)
    d = cuda(v)
    kw = dict(p=0.3, rng=(8, 9), norm="layer", gamma=d["gamma"], beta=d["beta"], bias=d["bias"])
    h, y, st = mba.dropout_add_norm(d["f"], d["x"], want_stats=True, **kw)
    g = mba.dropout_add_norm_backward(y, h, h, st, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h2, y2, st2 = mba.dropout_add_norm(d["f"], d["x"], want_stats=True, stream=s, **kw)
    g2 = mba.dropout_add_norm_backward(y2, h2, h2, st2, stream=s.cuda_stream, **kw)
    d2 = mba.dropout(d["f"], 0.3, (8, 9), stream=s)
    torch.cuda.synchronize()
    for a, b in zip((h, y, *st, *g, mba.dropout(d["f"], 0.3, (8, 9))), (h2, y2, *st2, *g2, d2)):
        assert torch.equal(a, b)


def test_a_workspace_serves_fewer_rows():
    size = mba.dropout_add_norm_bwd_workspace_size(5000, 768, mba.BF16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    w = torch.ones(768, device="cuda")
    for rows in (1, 37, 300, 1234, 2500, 4999):
        assert mba.dropout_add_norm_bwd_workspace_size(rows, 768, mba.BF16) <= size
        dy, h, st = randn((rows, 768), BF16, 1).cuda(), randn((rows, 768), BF16, 2).cuda(), torch.ones(rows, device="cuda")
        for dbias in (None, torch.empty(768, device="cuda")):
            df, dg, dg2 = torch.empty_like(dy), torch.empty(768, device="cuda"), torch.empty(768, device="cuda")
            kw = dict(p=0.1, rng=(1, 1), norm="rms", gamma=w)
            mba.dropout_add_norm_bwd(dy, None, h, (None, st), df, None, dbias=dbias, dgamma=dg, workspace=ws, **kw)
            mba.dropout_add_norm_bwd(dy, None, h, (None, st), df, None, dbias=dbias, dgamma=dg2, **kw)
            assert torch.equal(dg, dg2)


def test_refusals():
    f = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    kw = dict(p=0.1, rng=(1, 2), gamma=w)
    for bad in (dict(kw, p=1.5), dict(kw, p=float("nan")), dict(kw, gamma=None), dict(kw, norm=None), dict(kw, eps=-1.0)):
        with pytest.raises(mba.AddLNError):
            mba.dropout_add_norm(f, f, **bad)
    for bad in (dict(kw, norm="batch"), dict(kw, gamma=w.half()), dict(kw, bias=torch.ones(7, device="cuda")),
                dict(kw, rng=torch.zeros(2, dtype=torch.int64)), dict(kw, rng=(1, 2, 3))):
        with pytest.raises(ValueError):
            mba.dropout_add_norm(f, f, **bad)
    with pytest.raises(ValueError):
        mba.dropout_add_norm(f, torch.zeros(8, 4, device="cuda"), **kw)
    with pytest.raises(ValueError):
        mba.dropout_add_norm(f.half(), f, **kw)
    with pytest.raises(ValueError):
        mba.dropout_add_norm(f.t(), f.t(), p=0.1, rng=(1, 2), gamma=w[:4])
    with pytest.raises(ValueError):
        mba.dropout(f.t(), 0.1, (1, 2))
    with pytest.raises(ValueError):
        mba.dropout(f.long(), 0.1, (1, 2))
    with pytest.raises(TypeError):
        mba.dropout(f, 0.1, 7)
    with pytest.raises(mba.AddLNError):
        mba.dropout_add_norm_bwd(f, None, f, (None, w[:4].clone()), f.clone(), f.clone(), norm="rms", gamma=w, p=0.1,
                                 rng=(1, 2), dgamma=torch.empty(8, device="cuda"), workspace=torch.empty(8, device="cuda"))
    with pytest.raises(ValueError):
        mba.FusedDropoutAddNorm(8, p=2.0)


def test_written_tensors_change_their_version():
    f = torch.zeros(4, 8, device="cuda")
    y = torch.empty_like(f)
    v = y._version
    mba.dropout_fwd(f, y, 0.1, (1, 2))
    assert y._version > v
    v = y._version
    mba.dropout_add_norm_fwd(f, f, y, p=0.1, rng=(1, 2), norm=None)
    assert y._version > v
