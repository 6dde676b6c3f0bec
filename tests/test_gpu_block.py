"""The block boundary (post norm, gate, scaled residual sum, pre norm),
forward and backward, against its plain 64-bit form; bounds are derived in
_block_ref."""
from __future__ import annotations

import pytest
import torch

from _block_ref import assert_within, backward, forward, stats_of

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")
from memory_bound_add_gb300 import block  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import build
    build()
    yield
    torch.cuda.synchronize()
    assert mba.addln_get_device_error() == 0


def make(shape, dtype, post, pre, gate=None, beta=False, seed=0, loc=0.1):
    """Host inputs: f, x, parameters."""
    g = torch.Generator().manual_seed(seed)
    H = shape[-1]
    r = lambda s, sc=1.0, lo=0.0: torch.randn(s, generator=g) * sc + lo  # noqa: E731
    f, x = r(shape, 0.7, loc).to(dtype), r(shape, 1.5, loc).to(dtype)
    p = {}
    for side, kind in (("post", post), ("pre", pre)):
        if kind is not None:
            p[side + "_gamma"] = r((H,), 0.1, 1.0)
            if beta:
                p[side + "_beta"] = r((H,), 0.1)
    if gate == "channel":
        p["gate"] = r((H,), 0.2, 0.5)
    elif gate is not None:
        p["gate"] = r(gate, 0.5, 0.2).to(dtype)
    return f, x, p


def cuda(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def check_fwd(f, x, p, post, pre, a=1.0, s=1.0, eps=1e-5, what="", **kw):
    h, y, st = mba.block_norm(f.cuda(), x.cuda(), post=post, pre=pre, residual_scale=a, block_scale=s, eps=eps,
                              want_stats=True, **cuda(p), **kw)
    torch.cuda.synchronize()
    wh, wy, wst, eh, ey = forward(f, x, p, post, pre, a, s, eps)
    assert_within(h, wh, eh, what + " h")
    if pre is None:
        assert y is None
    else:
        assert_within(y, wy, ey, what + " y")
    for i, (g, w) in enumerate(zip(st, wst)):
        assert (g is None) == (w is None)
        if w is None:
            continue
        v = f.double() if i < 2 else wh
        dev = (v - v.mean(-1, keepdim=True)).abs().amax(-1, keepdim=True)
        if i in (0, 2):
            err = 2.0 ** -24 * (v.abs().amax(-1, keepdim=True) + 8 * dev)
        else:
            err = 2.0 ** -24 * 24 * w
        if i >= 2:  # h itself is off by eh
            err = err + (eh.amax(-1, keepdim=True) * (1 if i == 2 else w * w) * 2)
        assert_within(g, w.reshape(-1), err.reshape(-1), what + f" stat {i}")
    return h, y, st


def check_bwd(f, x, p, post, pre, a=1.0, s=1.0, eps=1e-5, what="", dy=True, dh=True, seed=7):
    g = torch.Generator().manual_seed(seed)
    wh, _, wst, _, _ = forward(f, x, p, post, pre, a, s, eps)
    dt = f.dtype
    h = wh.to(dt)
    st = [None if t is None else t.reshape(-1).float() for t in wst]
    dyt = torch.randn(f.shape, generator=g).to(dt) if dy and pre is not None else None
    dht = (torch.randn(f.shape, generator=g) * 0.5).to(dt) if dh else None
    want, err = backward(dyt, dht, f, h, st, p, post, pre, a, s)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = mba.block_norm_backward(c(dyt), c(dht), f.cuda(), h.cuda(), tuple(map(c, st)), post=post, pre=pre,
                                  residual_scale=a, block_scale=s, **cuda(p))
    torch.cuda.synchronize()
    for k, v in got._asdict().items():
        if v is None:
            continue
        assert_within(v, want[k].reshape(v.shape), err[k].reshape(v.shape), f"{what} {k}")
    return got


KINDS = [("rms", "rms"), ("layer", "layer"), (None, "rms"), (None, "layer"), ("rms", None), ("layer", "rms"),
         ("rms", "layer"), (None, None)]
# widths around every access width, warp, CTA and cluster border
WIDTHS = [1, 2, 7, 8, 31, 33, 64, 100, 250, 256, 264, 768, 1000, 1001, 2050, 4096, 4097, 4104, 8192]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("i,H", list(enumerate(WIDTHS)))
def test_widths(dtype, i, H):
    post, pre = KINDS[i % len(KINDS)]
    post2, pre2 = KINDS[(i + 1) % len(KINDS)]
    for j, (a, b, rows) in enumerate([(post, pre, 5), (post2, pre2, 1), ("layer", "layer", 3), ("rms", "rms", 2)]):
        gate = [None, "channel", (rows, H), (1, H)][(i + j) % 4]
        f, x, p = make((rows, H), dtype, a, b, gate, beta=(i + j) % 2 == 1, seed=100 * i + j)
        what = f"{rows}x{H} {a}/{b} gate {gate}"
        check_fwd(f, x, p, a, b, a=0.9, s=0.5, what=what)
        check_bwd(f, x, p, a, b, a=0.9, s=0.5, what=what)


@pytest.mark.parametrize("dtype,H", [(F32, 8193), (F32, 16384), (F16, 16400), (BF16, 32767), (BF16, 32768)])
def test_longest_rows(dtype, H):
    f, x, p = make((3, H), dtype, "layer", "layer", (3, H), beta=True, seed=H)
    check_fwd(f, x, p, "layer", "layer", what=f"{H}")
    check_bwd(f, x, p, "layer", "layer", what=f"{H}")
    f, x, p = make((2, H), dtype, "rms", "rms", "channel", seed=H + 1)
    check_fwd(f, x, p, "rms", "rms", what=f"{H}")
    check_bwd(f, x, p, "rms", "rms", what=f"{H}")


# every kind of gate row: one a row, one a few rows, one for all; gate rows
# that meet none, one or many borders between walkers
@pytest.mark.parametrize("post,pre,beta", [("rms", "rms", False), ("layer", "layer", True), (None, "rms", False),
                                           ("rms", None, True)])
@pytest.mark.parametrize("B,S,H,dtype", [(600, 1, 64, F32), (300, 2, 96, BF16), (7, 100, 40, F16),
                                         (1, 700, 33, F32), (3, 333, 200, BF16), (2, 500, 1001, F16),
                                         (5, 9, 4104, BF16), (1, 5000, 16, F32), (40, 128, 24, F16)])
def test_gate_rows(post, pre, beta, B, S, H, dtype):
    f, x, p = make((B, S, H), dtype, post, pre, (B, 1, H), beta=beta, seed=B * S + H)
    what = f"{B}x{S}x{H}"
    check_fwd(f, x, p, post, pre, s=0.7, what=what)
    check_bwd(f, x, p, post, pre, s=0.7, what=what)


@pytest.mark.parametrize("rows,H,dtype", [(1, 64, F32), (1000, 128, F16), (2048, 768, BF16), (333, 1001, BF16)])
@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "channel"), ("layer", "layer", None), (None, "layer", "channel")])
def test_many_rows(rows, H, dtype, post, pre, gate):
    f, x, p = make((rows, H), dtype, post, pre, gate, beta=True, seed=rows + H)
    check_fwd(f, x, p, post, pre, what=f"{rows}x{H}")
    check_bwd(f, x, p, post, pre, what=f"{rows}x{H}")


@pytest.mark.parametrize("dy,dh", [(True, False), (False, True)])
@pytest.mark.parametrize("H", [48, 1001, 4200])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), (None, "rms")])
def test_one_of_the_gradients(dy, dh, H, post, pre):
    f, x, p = make((21, H), BF16, post, pre, "channel", beta=True, seed=H)
    check_bwd(f, x, p, post, pre, dy=dy, dh=dh, what=f"dy {dy} dh {dh}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("H", [512, 4096])
def test_addresses_off_the_vector_width(dtype, H):
    # every buffer in turn one element off a 16-byte boundary: same values
    f, x, p = make((4, H), dtype, "rms", "layer", (4, H), beta=True, seed=H)
    off = lambda t: torch.cat([t.reshape(-1)[:1], t.reshape(-1)]).cuda()[1:].view(t.shape)  # noqa: E731
    ref = check_fwd(f, x, p, "rms", "layer")
    for which in ("f", "x", "gate", "post_gamma", "pre_beta"):
        q = {k: (off(v) if k == which else v.cuda()) for k, v in p.items()}
        h, y, _ = mba.block_norm(off(f) if which == "f" else f.cuda(), off(x) if which == "x" else x.cuda(),
                                 post="rms", pre="layer", want_stats=True, **q)
        assert_within(h, ref[0].cpu().double(), 2.0 ** -20 * (1 + ref[0].cpu().double().abs()) +
                      torch.finfo(dtype).eps * ref[0].cpu().double().abs(), which)
        assert_within(y, ref[1].cpu().double(), 2.0 ** -19 * (1 + ref[1].cpu().double().abs()) +
                      torch.finfo(dtype).eps * ref[1].cpu().double().abs(), which)


def at_offset(t, k):
    """t's values k elements into a buffer of its own whose other elements
    are 7, and that buffer."""
    buf = torch.full((t.numel() + 32,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[k:k + t.numel()].view(t.shape)
    v.copy_(t)
    return v, buf


def untouched(buf, k, n):
    return bool((buf[:k] == 7).all()) and bool((buf[k + n:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("H,post,pre", [(520, "rms", "rms"), (520, "layer", "layer"), (4099, "rms", "rms"),
                                        (1003, "layer", "rms")])
def test_each_buffer_off_the_borders(dtype, H, post, pre):
    # one buffer in turn (and all of them, each by its own distance) off the
    # 16-byte borders: values as ever, nothing written beside the outputs
    rows = 7
    f, x, p = make((rows, H), dtype, post, pre, (rows, H), beta=post == "layer", seed=H)
    wh, wy, wst, eh, ey = forward(f, x, p, post, pre, 0.9, 0.5, 1e-5)
    h0 = wh.to(dtype)
    st = tuple(None if t is None else t.reshape(-1).float().cuda() for t in wst)
    g = torch.Generator().manual_seed(3)
    dy, dh = torch.randn(rows, H, generator=g).to(dtype), torch.randn(rows, H, generator=g).to(dtype)
    want, err = backward(dy, dh, f, h0, [None if t is None else t.cpu() for t in st], p, post, pre, 0.9, 0.5)
    names = ["f", "x", "h", "y", "dy", "dh", "df", "dx", "gate", "dgate", "post_gamma", "pre_gamma"]
    for which in names + ["all"]:
        bufs = {}

        def place(name, t):
            k = 1 + names.index(name) if which == "all" else int(which == name)
            v, buf = at_offset(t, k)
            bufs[name] = (buf, k, t.numel())
            return v

        q = {k: place(k, v) if k in names else v.cuda() for k, v in p.items()}
        fc, xc = place("f", f), place("x", x)
        h, y = place("h", torch.zeros_like(f)), place("y", torch.zeros_like(f))
        mba.block_norm_fwd(fc, xc, h, y, post=post, pre=pre, residual_scale=0.9, block_scale=0.5, **q)
        torch.cuda.synchronize()
        assert_within(h, wh, eh, which + " h")
        assert_within(y, wy, ey, which + " y")
        assert all(untouched(*bufs[k]) for k in ("h", "y")), which
        h.copy_(h0)
        got = {k: place(k, torch.zeros_like(f)) for k in ("df", "dx", "dgate")}
        q.pop("pre_beta", None)
        mba.block_norm_bwd(place("dy", dy), place("dh", dh), fc, h, st, got["df"], got["dx"], post=post, pre=pre,
                           residual_scale=0.9, block_scale=0.5, dgate=got["dgate"], **q)
        torch.cuda.synchronize()
        for k, v in got.items():
            assert_within(v, want[k].reshape(v.shape), err[k].reshape(v.shape), f"{which} {k}")
            assert untouched(*bufs[k]), f"{which}: beside {k}"


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,S,H,parts", [(3, 50, 333, 3), (40, 7, 1002, 2), (2, 300, 4099, 2), (5, 1, 71, 6)])
def test_gate_rows_that_lie_off_the_borders(dtype, B, S, H, parts):
    # the parts of a projection of an odd width, each row shifted by its own
    # distance
    f, x, p = make((B, S, H), dtype, "rms", "layer", None, seed=H)
    wide = torch.randn(B, parts * H, generator=torch.Generator().manual_seed(2)).to(dtype)
    dy = torch.randn(B, S, H, generator=torch.Generator().manual_seed(3)).to(dtype)
    dev = wide.cuda()
    for part in (0, parts - 1):
        q = dict(p, gate=wide.chunk(parts, -1)[part].unsqueeze(1))
        dq = dict(cuda(p), gate=dev.chunk(parts, -1)[part].unsqueeze(1))
        wh, wy, wst, eh, ey = forward(f, x, q, "rms", "layer", 1.0, 1.0, 1e-5)
        h, y, _ = mba.block_norm(f.cuda(), x.cuda(), post="rms", pre="layer", **dq)
        assert_within(h, wh, eh, "h")
        assert_within(y, wy, ey, "y")
        hs, sts = wh.to(dtype), [None if t is None else t.reshape(-1).float() for t in wst]
        want, err = backward(dy, None, f, hs, sts, q, "rms", "layer", 1.0, 1.0)
        got = mba.block_norm_backward(dy.cuda(), None, f.cuda(), hs.cuda(),
                                      tuple(None if t is None else t.cuda() for t in sts), post="rms", pre="layer", **dq)
        for k in ("df", "dx", "dgate", "dpost_gamma", "dpre_gamma"):
            v = getattr(got, k)
            assert_within(v, want[k].reshape(v.shape), err[k].reshape(v.shape), k)


def test_in_place_off_the_borders():
    # rows that share 16-byte granules with their neighbours', written over
    for H, dtype in ((1001, BF16), (37, F16), (4101, F32), (16389, BF16)):
        f, x, p = make((300 if H < 2000 else 9, H), dtype, "rms", "rms", "channel", seed=H)
        q = cuda(p)
        h, y, st = mba.block_norm(f.cuda(), x.cuda(), post="rms", pre="rms", want_stats=True, **q)
        (f1, b1), (x1, b2) = at_offset(f, 3), at_offset(x, 5)
        mba.block_norm_fwd(f1, x1, x1, f1, post="rms", pre="rms", **q)
        torch.cuda.synchronize()
        assert torch.equal(x1, h) and torch.equal(f1, y)
        assert untouched(b1, 3, f.numel()) and untouched(b2, 5, f.numel())
        dy = torch.randn_like(h)
        want = mba.block_norm_backward(dy, h, f.cuda(), h, st, post="rms", pre="rms", **q)
        (d1, b1), (h1, b2) = at_offset(dy, 1), at_offset(h, 2)
        mba.block_norm_bwd(d1, h.clone(), f.cuda(), h1, st, d1, h1, post="rms", pre="rms", **q)
        torch.cuda.synchronize()
        assert torch.equal(d1, want.df) and torch.equal(h1, want.dx)
        assert untouched(b1, 1, f.numel()) and untouched(b2, 2, f.numel())


def test_gate_with_a_stride():
    # one part of a wider projection, as a modulation layer gives it
    B, S, H = 3, 50, 256
    f, x, p = make((B, S, H), BF16, "rms", "rms", None, seed=1)
    wide = torch.randn(B, 6 * H, generator=torch.Generator().manual_seed(2)).to(BF16)
    for part in (0, 2, 5):
        q = dict(p, gate=wide.chunk(6, -1)[part].unsqueeze(1))
        wh, wy, wst, eh, ey = forward(f, x, q, "rms", "rms", 1.0, 1.0, 1e-5)
        dev = wide.cuda().chunk(6, -1)[part].unsqueeze(1)
        assert not dev.is_contiguous()
        h, y, st = mba.block_norm(f.cuda(), x.cuda(), post="rms", pre="rms", want_stats=True, **dict(cuda(p), gate=dev))
        assert_within(h, wh, eh, "h")
        assert_within(y, wy, ey, "y")
        dy = torch.randn(B, S, H, generator=torch.Generator().manual_seed(3)).to(BF16)
        hs = wh.to(BF16)
        sts = [None if t is None else t.reshape(-1).float() for t in wst]
        want, err = backward(dy, None, f, hs, sts, q, "rms", "rms", 1.0, 1.0)
        got = mba.block_norm_backward(dy.cuda(), None, f.cuda(), hs.cuda(),
                                      tuple(None if t is None else t.cuda() for t in sts), post="rms", pre="rms",
                                      **dict(cuda(p), gate=dev))
        assert got.dgate.shape == (B, 1, H) and got.dgate.is_contiguous()
        for k in ("df", "dx", "dgate", "dpost_gamma", "dpre_gamma"):
            assert_within(getattr(got, k), want[k].reshape(getattr(got, k).shape), err[k].reshape(getattr(got, k).shape), k)


def test_in_place():
    for H in (96, 1001, 4104):
        f, x, p = make((9, H), F16, "layer", "rms", "channel", beta=True, seed=H)
        q = cuda(p)
        kw = dict(post="layer", pre="rms", **q)
        h, y, st = mba.block_norm(f.cuda(), x.cuda(), want_stats=True, **kw)
        f2, x2 = f.cuda(), x.cuda()
        mba.block_norm_fwd(f2, x2, x2, f2, **kw)       # h over x, y over f
        assert torch.equal(x2, h) and torch.equal(f2, y)
        f3, x3 = f.cuda(), x.cuda()
        mba.block_norm_fwd(f3, x3, f3, x3, **kw)
        assert torch.equal(f3, h) and torch.equal(x3, y)
        dy, dh = torch.randn_like(h), torch.randn_like(h)
        kb = dict(kw)
        kb.pop("pre_beta")
        ref = mba.block_norm_backward(dy, dh, f.cuda(), h, st, **kw)
        for df_at, dx_at in ((0, 1), (2, 3), (3, 0), (1, 2)):
            t = [dy.clone(), dh.clone(), f.cuda(), h.clone()]
            mba.block_norm_bwd(t[0], t[1], t[2], t[3], st, t[df_at], t[dx_at], **kb)
            assert torch.equal(t[df_at], ref.df) and torch.equal(t[dx_at], ref.dx)


def test_large_mean_and_constant_rows():
    # layer norms of rows whose mean is large against their spread, of rows
    # that are constant (variance 0, eps above 0: y = beta), and rms of zeros
    rows, H = 6, 1000
    f, x, p = make((rows, H), F32, "layer", "layer", None, beta=True, seed=3)
    f = f * 0.01 + 100.0
    x = x * 0.01 - 300.0
    f[1] = 7.0
    x[1] = 5.0
    h, y, st = check_fwd(f, x, p, "layer", "layer", what="large mean")
    f, x, p = make((rows, H), BF16, "rms", "rms", None, seed=4)
    f[2] = 0
    x[2] = 0
    h, y, _ = check_fwd(f, x, p, "rms", "rms", what="zeros")
    assert not h[2].any() and not y[2].any()


@pytest.mark.parametrize("H", [64, 1001, 4096, 8192])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer")])
def test_nan_and_infinity_stay_in_their_row(H, post, pre):
    f, x, p = make((8, H), BF16, post, pre, None, seed=H)
    clean = mba.block_norm(f.cuda(), x.cuda(), post=post, pre=pre, want_stats=True, **cuda(p))
    f2, x2 = f.clone(), x.clone()
    f2[2, H // 2] = float("nan")
    x2[5, H - 1] = float("inf")
    h, y, _ = mba.block_norm(f2.cuda(), x2.cuda(), post=post, pre=pre, want_stats=True, **cuda(p))
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(h[keep], clean[0][keep]) and torch.equal(y[keep], clean[1][keep])
    assert torch.isnan(h[2]).all() and torch.isnan(y[2]).all() and torch.isinf(h[5, H - 1])
    dy, dh = torch.randn_like(h), torch.randn_like(h)
    st = clean[2]
    want = mba.block_norm_backward(dy, dh, f.cuda(), clean[0], st, post=post, pre=pre, **cuda(p))
    dy2 = dy.clone()
    dy2[3, 0] = float("nan")
    got = mba.block_norm_backward(dy2, dh, f.cuda(), clean[0], st, post=post, pre=pre, **cuda(p))
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got.df[keep], want.df[keep]) and torch.equal(got.dx[keep], want.dx[keep])
    assert torch.isnan(got.dx[3]).all()


def test_no_rows():
    p = cuda(make((1, 64), F32, "rms", "rms", "channel", seed=0)[2])
    f = torch.empty(0, 64, device="cuda")
    h, y, st = mba.block_norm(f, f, post="rms", pre="rms", want_stats=True, **p)
    assert h.shape == y.shape == (0, 64) and st[1].shape == (0,)
    g = mba.block_norm_backward(f, f, f, f, st, post="rms", pre="rms", **p)
    torch.cuda.synchronize()
    for t in (g.dpost_gamma, g.dgate, g.dpre_gamma):
        assert t.shape == (64,) and not t.any()


def test_gate_rows_of_empty_sequences():
    # four sequences of no rows: their gate rows served nothing
    p = cuda(make((1, 64), F16, "rms", "rms", seed=0)[2])
    f, gate = torch.empty(4, 0, 64, dtype=F16, device="cuda"), torch.ones(4, 1, 64, dtype=F16, device="cuda")
    h, y, st = mba.block_norm(f, f, post="rms", pre="rms", gate=gate, want_stats=True, **p)
    assert h.shape == f.shape and st[1].shape == (0,)
    dgate = torch.full_like(gate, 5.0)
    mba.block_norm_bwd(f, f, f, f, st, torch.empty_like(f), torch.empty_like(f), post="rms", pre="rms", gate=gate,
                       dgate=dgate, **p)
    torch.cuda.synchronize()
    assert not dgate.any()
    g = gate.requires_grad_(True)
    h, y = mba.block_norm_train(f.requires_grad_(True), f.detach(), post="rms", pre="rms", gate=g, **p)
    (h.sum() + y.sum()).backward()
    assert g.grad.shape == gate.shape and not g.grad.any()


def test_same_bits_again_and_on_another_stream():
    f, x, p = make((3, 400, 520), F16, "layer", "rms", (3, 1, 520), beta=True, seed=11)
    q = cuda(p)
    fc, xc = f.cuda(), x.cuda()
    h, y, st = mba.block_norm(fc, xc, post="layer", pre="rms", want_stats=True, **q)
    dy = torch.randn_like(h)
    g = mba.block_norm_backward(dy, h, fc, h, st, post="layer", pre="rms", **q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for stream in (None, side, side.cuda_stream):
        h2, y2, st2 = mba.block_norm(fc, xc, post="layer", pre="rms", want_stats=True, stream=stream, **q)
        g2 = mba.block_norm_backward(dy, h, fc, h, st, post="layer", pre="rms", stream=stream, **q)
        outs.append((h2, y2, g2))
    torch.cuda.synchronize()
    for h2, y2, g2 in outs:
        assert torch.equal(h, h2) and torch.equal(y, y2)
        for u, v in zip(g, g2):
            assert u is None or torch.equal(u, v)


def test_two_streams_at_once():
    # each call has its own workspace, so calls may overlap
    cases, streams = [], [torch.cuda.Stream() for _ in range(4)]
    for i in range(4):
        f, x, p = make((500, 640 + 8 * i), BF16, "rms", "rms", "channel", seed=20 + i)
        q = cuda(p)
        h, _, st = mba.block_norm(f.cuda(), x.cuda(), post="rms", pre="rms", want_stats=True, **q)
        cases.append((f.cuda(), h, st, q, torch.randn_like(h)))
    want = [mba.block_norm_backward(dy, dy, f, h, st, post="rms", pre="rms", **q) for f, h, st, q, dy in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for i, (f, h, st, q, dy) in enumerate(cases):
            got[i].append(mba.block_norm_backward(dy, dy, f, h, st, post="rms", pre="rms", stream=streams[i], **q))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert all(u is None or torch.equal(u, v) for u, v in zip(w, g))


def test_captured_and_replayed():
    f, x, p = make((64, 1024), BF16, "rms", "rms", (64, 1024), seed=5)
    q, fc, xc = cuda(p), f.cuda(), x.cuda()
    dy = torch.randn_like(fc)

    def step():
        h, y, st = mba.block_norm(fc, xc, post="rms", pre="rms", want_stats=True, **q)
        return h, y, mba.block_norm_backward(dy, None, fc, h, st, post="rms", pre="rms", **q)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, y, gr = step()
    for k in range(3):
        fc.copy_(torch.randn_like(fc))
        g.replay()
        h2, y2, gr2 = step()
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2)
        assert all(u is None or torch.equal(u, v) for u, v in zip(gr, gr2))


def test_captured_training_step():
    # forward and backward through autograd in one graph, on leaves without an
    # eager graph of their own
    f, x, p = make((64, 1000), F16, "layer", "rms", "channel", beta=True, seed=15)
    fc, xc = f.cuda().requires_grad_(True), x.cuda().requires_grad_(True)
    q = {k: v.cuda().requires_grad_(True) for k, v in p.items()}
    leaves_ = [fc, xc, *q.values()]

    def step():
        h, y = mba.block_norm_train(fc, xc, post="layer", pre="rms", **q)
        return torch.autograd.grad((h.float() * 0.5 + y.float() ** 2).sum(), leaves_)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(2):
        with torch.no_grad():
            fc.copy_(torch.randn_like(fc))
        g.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(mine, want))


def test_two_graphs_with_one_workspace():
    # replayed one after the other on one stream, they may share it
    f, x, p = make((300, 768), F16, "rms", "rms", "channel", seed=6)
    q, fc = cuda(p), f.cuda()
    h, _, st = mba.block_norm(fc, x.cuda(), post="rms", pre="rms", want_stats=True, **q)
    ws = torch.empty(mba.block_norm_bwd_workspace_size(300, 768, mba.FP16, 1), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for i in range(2):
        dy = torch.randn_like(h)
        t = [torch.empty_like(h), torch.empty_like(h)] + [torch.empty(768, device="cuda") for _ in range(3)]

        def call(dy=dy, t=t):
            mba.block_norm_bwd(dy, None, fc, h, st, t[0], t[1], post="rms", pre="rms", dpost_gamma=t[2], dgate=t[3],
                               dpre_gamma=t[4], workspace=ws, **q)
        call()
        torch.cuda.synchronize()
        want = [v.clone() for v in t]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        outs.append((t, want, dy))  # a graph does not keep its inputs alive
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for t, want, _ in outs:
        assert all(torch.equal(u, v) for u, v in zip(t, want))


@pytest.mark.parametrize("dtype,H", [(F32, 768), (F16, 264), (BF16, 1024), (BF16, 4096), (F16, 5001), (BF16, 32768)])
def test_a_workspace_serves_shorter_calls(dtype, H):
    code = block.DTYPE_CODE[dtype]
    for kind, rpg in ((block.GATE_NONE, 1), (block.GATE_ROWS, 1), (block.GATE_ROWS, 7)):
        sizes = [mba.block_norm_bwd_workspace_size(r, H, code, kind, rpg)
                 for r in (1, 2, 100, 151, 152, 153, 200, 304, 305, 700, 1216, 1217, 5000, 9729, 40000, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[0] > 0
    most = 700 if H < 30000 else 40
    f, x, p = make((most, H), dtype, "rms", "rms", None, seed=H)
    q = dict(cuda(p), gate=torch.randn(most // 7 + 1, H, device="cuda").to(dtype))
    ws = torch.empty(mba.block_norm_bwd_workspace_size(most, H, code, block.GATE_ROWS, 7), dtype=torch.uint8,
                     device="cuda")
    for r in (most, most // 2, 153, 152, 35, 1):
        r = max(1, min(r, most) // 7 * 7)
        if r < 7:
            continue
        fc, xc = f[:r].cuda().view(-1, 7, H), x[:r].cuda().view(-1, 7, H)
        gate = q["gate"][:r // 7].unsqueeze(1)
        kw = dict(post="rms", pre="rms", **dict(q, gate=gate))
        h, _, st = mba.block_norm(fc, xc, want_stats=True, **kw)
        want = mba.block_norm_backward(h, None, fc, h, st, **kw)
        got = {k: torch.empty_like(getattr(want, k)) for k in ("df", "dx", "dgate", "dpost_gamma", "dpre_gamma")}
        mba.block_norm_bwd(h, None, fc, h, st, got["df"], got["dx"], workspace=ws, dgate=got["dgate"],
                           dpost_gamma=got["dpost_gamma"], dpre_gamma=got["dpre_gamma"], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(v, getattr(want, k)) for k, v in got.items())


def test_rows_behind_the_last_are_left():
    f, x, p = make((5, 1001), BF16, "rms", "rms", "channel", seed=8)
    big = [torch.full((8, 1001), 3.0, dtype=BF16, device="cuda") for _ in range(2)]
    mba.block_norm_fwd(f.cuda(), x.cuda(), big[0][:5], big[1][:5], post="rms", pre="rms", **cuda(p))
    torch.cuda.synchronize()
    for t in big:
        assert bool((t[5:] == 3.0).all()) and not bool((t[:5] == 3.0).all())


def test_offsets_past_32_bits():
    rows, H = 280000, 8192          # 2.3e9 elements a tensor
    g = torch.Generator(device="cuda").manual_seed(1)
    f = torch.empty(rows, H, dtype=BF16, device="cuda")
    x = torch.empty_like(f)
    for t in (f, x):
        t.zero_()
        t[-3:] = torch.randn(3, H, generator=g, device="cuda").to(BF16)
    p = {"post_gamma": torch.ones(H), "pre_gamma": torch.ones(H)}
    h, y, st = mba.block_norm(f, x, post="rms", pre="rms", want_stats=True, **cuda(p))
    fs, xs = f[-3:].cpu(), x[-3:].cpu()
    wh, wy, wst, eh, ey = forward(fs, xs, p, "rms", "rms", 1.0, 1.0, 1e-5)
    assert_within(h[-3:], wh, eh, "h")
    assert_within(y[-3:], wy, ey, "y")
    assert not h[:-3].any() and not y[:-3].any()
    del y
    hs = wh.to(BF16)
    h[-3:] = hs.cuda()
    for i in (1, 3):
        st[i][-3:] = wst[i].reshape(-1).float().cuda()
    got = mba.block_norm_backward(x, None, f, h, st, post="rms", pre="rms", **cuda(p))
    sts = [None, wst[1].reshape(-1).float(), None, wst[3].reshape(-1).float()]
    want, err = backward(xs, None, fs, hs, sts, p, "rms", "rms", 1.0, 1.0)
    for k in ("df", "dx"):
        assert_within(getattr(got, k)[-3:], want[k], err[k], k)
        assert not getattr(got, k)[:-3].any()
    for k in ("dpost_gamma", "dpre_gamma"):
        assert_within(getattr(got, k), want[k], err[k], k)


# ------------------------------------------------------------------ training
def leaves(f, x, p):
    return [t.cuda().requires_grad_(True) for t in (f, x)], {k: v.cuda().requires_grad_(True) for k, v in p.items()}


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "channel"), ("layer", "layer", (2, 1, 96)), (None, "rms", None),
                                           ("layer", None, (2, 7, 96)), (None, "layer", "channel")])
def test_autograd_against_differences(post, pre, gate):
    # along a random direction of all inputs at once, the derivative of the
    # plain 64-bit loss by central differences (step t: an error of t^2 beside
    # rounding of 2^-52 / t) against the kernels' gradients
    shape = (2, 7, 96)
    f, x, p = make(shape, F32, post, pre, gate, beta=True, seed=9)
    (fc, xc), q = leaves(f, x, p)
    h, y = mba.block_norm_train(fc, xc, post=post, pre=pre, residual_scale=0.9, block_scale=0.6, **q)
    gen = torch.Generator().manual_seed(10)
    wy, wh = torch.randn(shape, generator=gen), torch.randn(shape, generator=gen)
    loss = (h * wh.cuda()).sum()
    if pre is not None:
        loss = loss + (y * wy.cuda()).sum()
    loss.backward()
    names = ["f", "x"] + list(p)
    vals = [f.double(), x.double()] + [p[k].double() for k in p]
    grads = [fc.grad, xc.grad] + [q[k].grad for k in p]
    dirs = [torch.randn(v.shape, generator=gen, dtype=torch.float64) for v in vals]

    def value(t):
        w = [v + t * d for v, d in zip(vals, dirs)]
        hh, yy, _, _, _ = forward(w[0], w[1], dict(zip(names[2:], w[2:])), post, pre, 0.9, 0.6, 1e-5)
        out = (hh * wh.double()).sum()
        return out + (yy * wy.double()).sum() if pre is not None else out

    t = 1e-5
    want = float((value(t) - value(-t)) / (2 * t))
    terms = [(g.cpu().double() * d) for g, d in zip(grads, dirs)]
    got = float(sum(v.sum() for v in terms))
    scale = float(sum(v.abs().sum() for v in terms))
    # fp32 gradients: 64 u of the magnitudes; differences: t^2 of third
    # derivatives (of the magnitudes' size times about 100 for these rows)
    assert abs(got - want) <= scale * (64 * 2.0 ** -24 + 100 * t * t) + 1e-9, (got, want, scale)


def test_only_the_gradients_asked_for():
    f, x, p = make((20, 256), BF16, "layer", "layer", "channel", beta=True, seed=12)
    (fc, xc), q = leaves(f, x, p)
    h, y = mba.block_norm_train(fc, xc, post="layer", pre="layer", **q)
    (h.float().sum() + (y.float() ** 2).sum()).backward()
    q2 = {k: v.detach() for k, v in q.items()}
    q2["gate"] = q["gate"].detach().clone().requires_grad_(True)
    x2 = xc.detach().clone().requires_grad_(True)
    h, y = mba.block_norm_train(fc.detach(), x2, post="layer", pre="layer", **q2)
    (h.float().sum() + (y.float() ** 2).sum()).backward()
    torch.cuda.synchronize()
    assert torch.equal(x2.grad, xc.grad) and torch.equal(q2["gate"].grad, q["gate"].grad)


def test_expanded_and_shared_inputs():
    # a gate that is expanded over the batch, a gradient that is expanded (a
    # plain sum), and f also being the residual stream
    B, S, H = 3, 5, 64
    f, _, p = make((B, S, H), F32, "rms", "rms", None, seed=13)
    gate = torch.randn(1, 1, H, generator=torch.Generator().manual_seed(1))
    fc = f.cuda().requires_grad_(True)
    q = {k: v.cuda().requires_grad_(True) for k, v in p.items()}
    gc = gate.cuda().requires_grad_(True)
    h, y = mba.block_norm_train(fc, fc, post="rms", pre="rms", gate=gc.expand(B, 1, H), **q)
    (h.sum() + y.sum()).backward()
    f2 = f.double().requires_grad_(True)
    q2 = {k: v.double().requires_grad_(True) for k, v in p.items()}
    g2 = gate.double().requires_grad_(True)
    hh, yy, _, _, _ = forward(f2, f2, dict(q2, gate=g2), "rms", "rms", 1.0, 1.0, 1e-5)
    (hh.sum() + yy.sum()).backward()
    for u, v in [(fc.grad, f2.grad), (gc.grad, g2.grad)] + [(q[k].grad, q2[k].grad) for k in q]:
        v = v.reshape(u.shape)
        # 15 rows: fp32 sums of terms of the size of the row's gradients
        assert_within(u, v, 2.0 ** -24 * 64 * (v.abs() + v.abs().amax() + 15), "gradient")


def test_module():
    m = mba.FusedBlockNorm(256, post="layer", pre="layer", bias=True, layer_scale=0.1, block_scale=0.5, device="cuda")
    assert sorted(n for n, _ in m.named_parameters()) == ["layer_scale", "post_bias", "post_weight", "pre_bias",
                                                          "pre_weight"]
    f, x = torch.randn(4, 9, 256, device="cuda"), torch.randn(4, 9, 256, device="cuda")
    h, y = m(f, x)
    want, wy, _, eh, ey = forward(f.cpu(), x.cpu(), {"post_gamma": torch.ones(256), "pre_gamma": torch.ones(256),
                                                     "post_beta": torch.zeros(256), "pre_beta": torch.zeros(256),
                                                     "gate": torch.full((256,), 0.1)}, "layer", "layer", 1.0, 0.5, 1e-5)
    assert_within(h, want, eh, "h")
    assert_within(y, wy, ey, "y")
    (y ** 2).mean().backward()
    assert all(v.grad is not None and bool(torch.isfinite(v.grad).all()) for v in m.parameters())
    with pytest.raises(ValueError):
        m(f, x, gate=torch.ones_like(f))
    plain = mba.FusedBlockNorm(256, post=None, pre=None, device="cuda")
    h, y = plain(f, x)
    assert y is None and torch.equal(h, x + f)
    g = torch.randn(4, 1, 256, device="cuda")
    h, _ = plain(f, x, gate=g)
    # x + f g: at most one rounding of the product (2^-24 of it) beside the
    # sum's own, which assert_within counts; whether the product is rounded
    # at all is not part of the definition, so no equality with another order
    fg = f.cpu().double() * g.cpu().double()
    assert_within(h, x.cpu().double() + fg, 2.0 ** -24 * fg.abs(), "h")


def test_refusals_of_the_wrapper():
    f, x, p = make((4, 64), F16, "rms", "rms", None, seed=14)
    fc, xc, q = f.cuda(), x.cuda(), cuda(p)
    kw = dict(post="rms", pre="rms", **q)
    bad = [dict(f=fc, x=xc.float()), dict(f=fc, x=xc[:2]), dict(f=fc.t(), x=xc.t()), dict(f=f, x=x),
           dict(f=fc, x=xc, gate=torch.ones(64, dtype=F16, device="cuda")),
           dict(f=fc, x=xc, gate=torch.ones(4, 64, device="cuda")),
           dict(f=fc, x=xc, gate=torch.ones(2, 64, dtype=F16, device="cuda")),
           dict(f=fc, x=xc, gate=torch.ones(1, 64, dtype=F16, device="cuda").expand(4, 64)),
           dict(f=fc, x=xc, post_gamma=torch.ones(63, device="cuda")),
           dict(f=fc, x=xc, post_gamma=torch.ones(64, device="cuda", dtype=F16)),
           dict(f=fc, x=xc, post="batch"), dict(f=fc.double(), x=xc.double())]
    for b in bad:
        with pytest.raises((ValueError, TypeError)):
            mba.block_norm(b.pop("f"), b.pop("x"), **{**kw, **b})
    for b, code in ((dict(eps=-1.0), -4), (dict(residual_scale=float("nan")), block.ERR_SCALE),
                    (dict(block_scale=float("inf")), block.ERR_SCALE), (dict(pre_gamma=None), -1),
                    (dict(post=None), block.ERR_KIND), (dict(pre=None), block.ERR_KIND)):
        with pytest.raises(mba.AddLNError) as e:
            mba.block_norm(fc, xc, **{**kw, **b})
        assert e.value.code == code, b
    with pytest.raises(mba.AddLNError) as e:
        mba.block_norm_fwd(fc, xc, xc, xc, **kw)
    assert e.value.code == -5
    h, y, st = mba.block_norm(fc, xc, want_stats=True, **kw)
    with pytest.raises(mba.AddLNError) as e:
        mba.block_norm_bwd(y, None, fc, h, st, torch.empty_like(h), torch.empty_like(h), post="rms", pre="rms",
                           dpre_gamma=torch.empty(64, device="cuda"),
                           workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **q)
    assert e.value.code == -10
    with pytest.raises(ValueError):
        mba.block_norm_backward(y[:, :32].contiguous(), None, fc, h, st, **kw)
    with pytest.raises(TypeError):
        mba.block_norm_backward(None, None, fc, h, st, **kw)
    with pytest.raises(ValueError):  # as many elements, but another shape
        mba.block_norm_train(fc, xc.view(8, 32), **kw)


@pytest.mark.parametrize("H", [64, 1000, 1001, 4096, 8200])
@pytest.mark.parametrize("c", [7.0, 0.1, -3.3e4, 1e-20])
def test_rows_of_equal_values(H, c):
    # variance exactly 0: y is beta, and without eps the 0 * inf of the formula
    x = torch.full((3, H), c, device="cuda")
    f = torch.zeros_like(x)
    g, b = torch.rand(H, device="cuda") + 0.5, torch.randn(H, device="cuda")
    for kw in (dict(eps=1e-5), dict(eps=1e-12)):
        _, y, st = mba.block_norm(f, x, pre="layer", pre_gamma=g, pre_beta=b, want_stats=True, **kw)
        assert torch.equal(y, b.expand_as(y))
        assert bool(((st[2] - c).abs() <= 2.0 ** -23 * abs(c)).all())
    _, y, _ = mba.block_norm(f, x, pre="layer", pre_gamma=g, pre_beta=b, eps=0.0)
    assert bool(torch.isnan(y).all())
    # one value a single step off is a variance, where the square of a step is
    # an fp32 value at all: (2^-23 * 1e-20)^2 is about 1e-54, below the least
    # subnormal 1.4e-45, and the fp32 variance is then 0
    if abs(c) < 1e-10:
        return
    x[1, H // 2] = torch.nextafter(x[1, 0], torch.tensor(float("inf"), device="cuda"))
    _, y, _ = mba.block_norm(f, x, pre="layer", pre_gamma=torch.ones_like(g), eps=0.0)
    assert bool(torch.isfinite(y[1]).all()) and bool(torch.isnan(y[0]).all())


@pytest.mark.parametrize("post,pre", [("layer", None), (None, "layer")])
def test_means_near_zero_keep_their_digits(post, pre):
    # A mean that is small against the values.  Around the first estimate K of
    # the mean, the roundings of d = v - K (u |d| / sqrt 3 each, independent)
    # and of the sums of d (12 in a thread, 10 levels beyond, each of a partial
    # sum of about sqrt(its length) spreads) give the mean of 768 values an rms
    # error of about sqrt(1/3 + 22/3) u spread / sqrt(768) = 0.1 u spread, and
    # the result's own rounding u |mean| / sqrt 3 with |mean| about 0.05; h adds
    # u spread / sqrt(3 * 768).  Shifting by one value of the row instead costs
    # roundings of that value's size, some u spread each.
    f, x, p = make((200, 768), F16, post, pre, None, seed=77, loc=0.05)
    _, _, st = mba.block_norm(f.cuda(), x.cuda(), post=post, pre=pre, eps=1e-12, want_stats=True, **cuda(p))
    h, _, want, _, _ = forward(f, x, p, post, pre, 1.0, 1.0, 1e-12)
    got, w, v = (st[0], want[0], f.double()) if post else (st[2], want[2], h)
    rms = ((got.cpu().double() - w.reshape(-1)) ** 2).mean().sqrt()
    assert float(rms) <= 2.0 ** -24 * float(v.std()) * 0.5


def fill_shared_memory_with_nan():
    """A backward over rows of NaN, whose staged rows stay behind in the
    shared memory of every SM."""
    bad = torch.full((2048, 4096), float("nan"), dtype=BF16, device="cuda")
    one, r = torch.ones(4096, device="cuda"), torch.ones(2048, device="cuda")
    mba.block_norm_backward(bad, bad, bad, bad, (None, r, None, r), post="rms", post_gamma=one, pre="rms",
                            pre_gamma=one)


@pytest.mark.parametrize("dtype,H", [(F32, 1), (F32, 2), (F32, 3)] + [(t, h) for t in (F16, BF16) for h in range(1, 8)])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), (None, "rms")])
def test_shortest_rows_off_the_borders(dtype, H, post, pre):
    # the first row of a buffer ends within its first 16 bytes: what the rest of
    # them held in shared memory before must not matter
    rows = 3
    for k in range(1, 16 // torch.empty((), dtype=dtype).element_size()):
        for gate in (None, "channel", (rows, H), (1, H)):
            f, x, p = make((rows, H), dtype, post, pre, gate, beta=True, seed=100 * H + k)
            wh, wy, wst, eh, ey = forward(f, x, p, post, pre, 1.0, 1.0, 1e-5)
            q = {n: at_offset(v, k)[0] if n == "gate" and v.dim() > 1 else v.cuda() for n, v in p.items()}
            fc, xc = at_offset(f, k)[0], at_offset(x, k)[0]
            what = f"offset {k} gate {gate}"
            fill_shared_memory_with_nan()
            h, y, _ = mba.block_norm(fc, xc, post=post, pre=pre, **q)
            assert_within(h, wh, eh, what + " h")
            assert_within(y, wy, ey, what + " y")
            g = torch.Generator().manual_seed(k)
            dy, dh = torch.randn(rows, H, generator=g).to(dtype), torch.randn(rows, H, generator=g).to(dtype)
            h0, st = wh.to(dtype), [None if t is None else t.reshape(-1).float() for t in wst]
            want, err = backward(dy, dh, f, h0, st, p, post, pre, 1.0, 1.0)
            args = [at_offset(t, k)[0] for t in (dy, dh)] + [fc, at_offset(h0, k)[0]]
            fill_shared_memory_with_nan()
            got = mba.block_norm_backward(*args, tuple(None if t is None else t.cuda() for t in st), post=post,
                                          pre=pre, **q)
            for n, v in got._asdict().items():
                if v is not None:
                    assert_within(v, want[n].reshape(v.shape), err[n].reshape(v.shape), f"{what} {n}")


@pytest.mark.parametrize("dtype,H", [(F32, 16384), (F16, 32760), (BF16, 32768), (BF16, 20001)])
def test_rows_of_a_cluster_call_after_call(dtype, H):
    # rows that several CTAs share, in short calls one close upon another and on
    # two streams at once: the CTAs of a cluster write into each other's shared
    # memory from the first row on
    f, x, p = make((3, H), dtype, "layer", "layer", "channel", beta=True, seed=H)
    q, fc, xc = cuda(p), f.cuda(), x.cuda()
    kw = dict(post="layer", pre="layer", **q)
    h, y, st = check_fwd(f, x, p, "layer", "layer", what=f"{H}")
    check_bwd(f, x, p, "layer", "layer", what=f"{H}")
    want = mba.block_norm_backward(y, h, fc, h, st, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        s = streams[i % 2]
        got.append((mba.block_norm(fc, xc, want_stats=True, stream=s, **kw)[:2],
                    mba.block_norm_backward(y, h, fc, h, st, stream=s, **kw)))
    torch.cuda.synchronize()
    for (h2, y2), g in got:
        assert torch.equal(h, h2) and torch.equal(y, y2)
        assert all(u is None or torch.equal(u, v) for u, v in zip(want, g))


@pytest.mark.parametrize("rpg", [9, 1 << 31, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, 1 << 40, (1 << 63) - 1])
@pytest.mark.parametrize("rows,H,dtype", [(8, 64, F32), (8, 1001, BF16), (1, 96, F16)])
def test_a_gate_row_for_more_rows_than_there_are(rpg, rows, H, dtype):
    # the library's own entry points: one gate row for all rows, whatever the
    # number of rows that it could serve
    lib, code = block.lib(), block.DTYPE_CODE[dtype]
    f, x, p = make((rows, H), dtype, "rms", "rms", (1, H), seed=H)
    q, fc, xc = cuda(p), f.cuda(), x.cuda()
    kw = dict(post="rms", pre="rms", **q)
    h, y, st = mba.block_norm(fc, xc, want_stats=True, **kw)
    want = mba.block_norm_backward(y, h, fc, h, st, **kw)
    h2, y2 = torch.empty_like(h), torch.empty_like(y)
    stream = torch.cuda.current_stream().cuda_stream
    pg, ng, gate = (q[k].data_ptr() for k in ("post_gamma", "pre_gamma", "gate"))
    assert lib.block_norm_fwd(fc.data_ptr(), xc.data_ptr(), block.NORM_RMS, pg, None, gate, block.GATE_ROWS, H, rpg, 1.0,
                              1.0, block.NORM_RMS, ng, None, h2.data_ptr(), y2.data_ptr(), None, None, None, None, rows,
                              H, 1e-5, code, stream) == 0
    assert torch.equal(h, h2) and torch.equal(y, y2)
    size = mba.block_norm_bwd_workspace_size(rows, H, code, block.GATE_ROWS, rpg)
    assert size == mba.block_norm_bwd_workspace_size(rows, H, code, block.GATE_ROWS, rows)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    got = {k: torch.empty_like(getattr(want, k)) for k in ("df", "dx", "dgate", "dpost_gamma", "dpre_gamma")}
    at = {k: v.data_ptr() for k, v in got.items()}
    assert lib.block_norm_bwd(y.data_ptr(), h.data_ptr(), fc.data_ptr(), h.data_ptr(), block.NORM_RMS, pg, None, None,
                              st[1].data_ptr(), gate, block.GATE_ROWS, H, rpg, 1.0, 1.0, block.NORM_RMS, ng, None,
                              st[3].data_ptr(), at["df"], at["dx"], at["dpost_gamma"], None, at["dgate"],
                              at["dpre_gamma"], None, rows, H, code, ws.data_ptr(), size, stream) == 0
    torch.cuda.synchronize()
    for k, v in got.items():
        assert torch.equal(v, getattr(want, k)), k


def test_refusals_of_other_shapes():
    # as many elements, but rows that are not each other's
    kw = dict(post="rms", pre="rms", post_gamma=torch.ones(32, device="cuda"), pre_gamma=torch.ones(32, device="cuda"))
    f = torch.randn(4, 6, 32, device="cuda")
    other = [f.transpose(0, 1).contiguous(), f.view(2, 12, 32), f.view(3, 8, 32), f.view(12, 64), f.view(4, 3, 64)]
    h, y, st = mba.block_norm(f, f, want_stats=True, **kw)
    new = lambda: torch.empty_like(f)  # noqa: E731
    for t in other:
        for call in (lambda: mba.block_norm(f, t, **kw), lambda: mba.block_norm_fwd(f, t, new(), new(), **kw),
                     lambda: mba.block_norm_fwd(f, f, torch.empty_like(t), new(), **kw),
                     lambda: mba.block_norm_fwd(f, f, new(), torch.empty_like(t), **kw),
                     lambda: mba.block_norm_backward(y, t, f, h, st, **kw),
                     lambda: mba.block_norm_backward(y, None, t, h, st, **kw),
                     lambda: mba.block_norm_backward(y, None, f, t, st, **kw),
                     lambda: mba.block_norm_bwd(y, h, f, h, st, torch.empty_like(t), new(), **kw),
                     lambda: mba.block_norm_bwd(y, h, f, h, st, new(), torch.empty_like(t), **kw)):
            with pytest.raises(ValueError):
                call()
    gate = torch.randn(4, 1, 32, device="cuda")
    for bad in (torch.empty(8, 16, device="cuda"), torch.empty(2, 64, device="cuda"), torch.empty(128, device="cuda")):
        with pytest.raises(ValueError):
            mba.block_norm_bwd(y, h, f, h, st, new(), new(), gate=gate, dgate=bad, **kw)
    # the same rows with leading sizes joined or split are no other rows
    for shape in ((24, 1, 32), (4, 2, 3, 32), (1, 4, 6, 32)):
        h2, y2, _ = mba.block_norm(f, f.view(shape), **kw)
        assert torch.equal(h2, h) and torch.equal(y2, y)
    flat = lambda t: t.view(24, 32)  # noqa: E731
    h2, y2, _ = mba.block_norm(f, flat(f), **kw)
    h3, y3, _ = mba.block_norm(flat(f), f, **kw)
    assert torch.equal(h2, h) and torch.equal(h3, flat(h)) and torch.equal(y2, y) and torch.equal(y3, flat(y))
    want = mba.block_norm_backward(y, h, f, h, st, gate=gate, **kw)
    df, dx, dg = torch.empty(24, 32, device="cuda"), new(), torch.empty(4, 32, device="cuda")
    mba.block_norm_bwd(y, flat(h), flat(f), h, st, df, dx, gate=gate, dgate=dg, **kw)
    assert torch.equal(df, flat(want.df)) and torch.equal(dx, want.dx) and torch.equal(dg, want.dgate.view(4, 32))


def test_autograd_sees_what_is_written():
    # every tensor that a call is given to write into has changed for autograd,
    # so that a graph that saved it refuses to go on
    f, x, p = make((4, 64), F32, "rms", "rms", "channel", seed=21)
    q = cuda(p)
    kw = dict(post="rms", pre="rms", **q)
    new = lambda *s: torch.zeros(*(s or (4, 64)), device="cuda")  # noqa: E731
    fc, xc = f.cuda(), x.cuda()
    h, y, st = new(), new(), (None, new(4), None, new(4))
    outs = [h, y, st[1], st[3]]
    before = [t._version for t in outs]
    mba.block_norm_fwd(fc, xc, h, y, st, **kw)
    assert all(t._version > v for t, v in zip(outs, before))
    g = dict(dpost_gamma=new(64), dgate=new(64), dpre_gamma=new(64))
    outs = [new(), new(), *g.values()]
    before = [t._version for t in outs]
    mba.block_norm_bwd(y, h, fc, h, st, outs[0], outs[1], **g, **kw)
    assert all(t._version > v for t, v in zip(outs, before))
    # in place over a tensor that a graph has saved
    a = x.cuda().requires_grad_(True)
    b = a * 1.0
    loss = (b * b).sum()
    with torch.no_grad():
        mba.block_norm_fwd(fc, b.detach(), b.detach(), y, **kw)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # tensors without versions are written all the same
    with torch.inference_mode():
        h2, y2 = new(), new()
    mba.block_norm_fwd(fc, xc, h2, y2, **kw)
    want = mba.block_norm(fc, xc, **kw)
    assert torch.equal(h2, want[0]) and torch.equal(y2, want[1])


def test_two_graphs_with_one_workspace_write_their_outputs():
    # each replay by itself fills outputs that were NaN before
    f, x, p = make((300, 768), F16, "rms", "rms", "channel", seed=6)
    q, fc = cuda(p), f.cuda()
    h, _, st = mba.block_norm(fc, x.cuda(), post="rms", pre="rms", want_stats=True, **q)
    ws = torch.empty(mba.block_norm_bwd_workspace_size(300, 768, mba.FP16, 1), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for i in range(2):
        dy = torch.randn_like(h)
        t = [torch.empty_like(h), torch.empty_like(h)] + [torch.empty(768, device="cuda") for _ in range(3)]

        def call(dy=dy, t=t):
            mba.block_norm_bwd(dy, None, fc, h, st, t[0], t[1], post="rms", pre="rms", dpost_gamma=t[2], dgate=t[3],
                               dpre_gamma=t[4], workspace=ws, **q)
        call()
        torch.cuda.synchronize()
        want = [v.clone() for v in t]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        outs.append((t, want, dy))  # a graph does not keep its inputs alive
        graphs.append(g)

    def clear():
        for t, _, _ in outs:
            for v in t:
                v.fill_(float("nan"))
        ws.fill_(255)  # NaN patterns

    for g, (t, want, _) in list(zip(graphs, outs)) * 2:
        clear()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(t, want))
    clear()
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for t, want, _ in outs:
        assert all(torch.equal(u, v) for u, v in zip(t, want))


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
def test_a_single_row_of_one_dimension(dtype):
    # f, x and a gate of f's dtype, all [H]
    f, x, p = make((200,), dtype, "rms", "layer", None, seed=3)
    p["gate"] = torch.randn(200, generator=torch.Generator().manual_seed(4)).to(dtype)
    wh, wy, wst, eh, ey = forward(f, x, p, "rms", "layer", 1.0, 1.0, 1e-5)
    h, y, st = mba.block_norm(f.cuda(), x.cuda(), post="rms", pre="layer", want_stats=True, **cuda(p))
    assert_within(h, wh, eh, "h")
    assert_within(y, wy, ey, "y")
    row = lambda t: t.cuda().view(1, 200)  # noqa: E731
    q = dict(cuda(p), gate=row(p["gate"]))
    dy = torch.randn(200, generator=torch.Generator().manual_seed(5)).to(dtype)
    got = mba.block_norm_backward(dy.cuda(), None, f.cuda(), h, st, post="rms", pre="layer", **cuda(p))
    want = mba.block_norm_backward(row(dy), None, row(f), h.view(1, 200), st, post="rms", pre="layer", **q)
    assert got.dgate.dtype == dtype and got.dgate.shape == (200,)
    for u, v in zip(got, want):
        # the same sums of one row: a channel gate's go through fp32 columns
        assert u is None or u.dtype is F32 and dtype is F32 or torch.equal(u.reshape(-1), v.reshape(-1))
    leaf = p["gate"].cuda().requires_grad_(True)
    _, y2 = mba.block_norm_train(f.cuda(), x.cuda(), post="rms", pre="layer", **dict(cuda(p), gate=leaf))
    (y2.float() * dy.cuda().float()).sum().backward()
    assert torch.equal(leaf.grad, got.dgate)


@pytest.mark.parametrize("shape", [(5, 0, 64), (0, 5, 64), (2, 0, 3, 64)])
def test_gates_of_no_rows(shape):
    # a gate of its own for every row, where there are none
    p = cuda(make((1, 64), F16, "rms", "rms", seed=0)[2])
    f = torch.empty(shape, dtype=F16, device="cuda", requires_grad=True)
    gate = torch.empty(shape, dtype=F16, device="cuda", requires_grad=True)
    q = {k: v.requires_grad_(True) for k, v in p.items()}
    h, y = mba.block_norm_train(f, f.detach(), post="rms", pre="rms", gate=gate, **q)
    (h.sum() + y.sum()).backward()
    torch.cuda.synchronize()
    assert h.shape == y.shape == f.grad.shape == gate.grad.shape == shape
    assert all(not v.grad.any() for v in q.values())


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "layer"), ("layer", "rms"), ("rms", "rms")])
@pytest.mark.parametrize("offset", [10.0, 100.0])
def test_gradients_with_an_offset(dtype, post, pre, offset):
    # a dy, and a dh, whose mean is large against its spread: the bounds go by
    # the magnitudes, which the offset raises
    rows, H = 6, 4096
    f, x, p = make((rows, H), dtype, post, pre, "channel", beta=True, seed=31)
    wh, _, wst, _, _ = forward(f, x, p, post, pre, 1.0, 1.0, 1e-5)
    h, st = wh.to(dtype), [None if t is None else t.reshape(-1).float() for t in wst]
    g = torch.Generator().manual_seed(32)
    dy, dh = ((torch.randn(rows, H, generator=g) + offset).to(dtype) for _ in range(2))
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    for one, other in ((dy, None), (None, dh), (dy, dh)):
        want, err = backward(one, other, f, h, st, p, post, pre, 1.0, 1.0)
        got = mba.block_norm_backward(c(one), c(other), f.cuda(), h.cuda(), tuple(map(c, st)), post=post, pre=pre,
                                      **cuda(p))
        torch.cuda.synchronize()
        for k, v in got._asdict().items():
            if v is not None:
                assert_within(v, want[k].reshape(v.shape), err[k].reshape(v.shape), k)
