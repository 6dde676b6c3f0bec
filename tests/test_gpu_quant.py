"""The norm with an 8-bit output, and reading it back, against the plain 64-bit
forms of _quant_ref, which derives the bounds."""
from __future__ import annotations

import pytest
import torch

from _block_ref import TINY, U, assert_within
from _quant_ref import LEAST, TOP, TORCH, check, norm_quant, to_grid
from test_gpu_block import at_offset, cuda
from test_gpu_drop import randn

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
FORMATS = pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "int8"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import build
    build()
    yield
    torch.cuda.synchronize()
    assert mba.addln_get_device_error() == 0


def make(shape, dtype, norm, beta=False, residual=True, seed=0):
    H = shape[-1]
    v = {"x": randn(shape, dtype, seed, 0.7, 0.1), "residual": randn(shape, dtype, seed + 1, 1.5, 0.1) if residual else None}
    v["gamma"] = randn((H,), seed=seed + 2, sc=0.1, loc=1.0) if norm else None
    v["beta"] = randn((H,), seed=seed + 3, sc=0.1) if norm and beta else None
    return v


def values(q, scale, scaling, group):
    """q * scale in 64 bits, [rows, H], on the host."""
    H = q.shape[-1]
    q = q.cpu().double().reshape(-1, H)
    if scaling == "tensor":
        return q * float(scale)
    s = scale.cpu().float().double().reshape(q.shape[0], -1)
    return q * s.repeat_interleave(group or H, 1)[:, :H]


def check_read(q, scale, scaling, group, what=""):
    """dequantise: one product and the output's rounding."""
    want = values(q, scale, scaling, group)
    for dt in (F32, F16, BF16):
        got = mba.dequantise(q, scale, dtype=dt)
        assert got.shape == q.shape
        fits = want.abs() < torch.finfo(dt).max  # fp16 and a wide scale
        bound = U * want.abs()
        assert_within(got.reshape(want.shape).cpu()[fits], want[fits], bound[fits], f"{what} read back to {dt}")


def check_fwd(v, norm, fmt, scaling, group=None, eps=1e-5, what="", major=False, given=None, read=True):
    d = cuda(v)
    s = None if given is None else torch.tensor(given, device="cuda")
    r = mba.norm_quant(d["x"], d["residual"], norm=norm, gamma=d["gamma"], beta=d["beta"], eps=eps, format=fmt,
                       scaling=scaling, group=group, scale=s, group_major=major, want_stats=True)
    torch.cuda.synchronize()
    h, y, st, eh, ey = norm_quant(v["x"], v["residual"], norm, v["gamma"], v["beta"], eps)
    assert r.q.dtype is TORCH[fmt] and r.q.shape == v["x"].shape
    if v["residual"] is None:
        assert r.h is None
    else:
        assert_within(r.h, h.view(r.h.shape), eh.view(r.h.shape), what + " h")
    g = group or (128 if scaling == "group" else 32 if scaling == "pow2" else 0)
    sc = r.scale.cpu().float().reshape(y.shape[0], -1) if scaling != "tensor" else None
    check(r.q.cpu().float().reshape(y.shape), sc, y, ey, fmt, scaling, g, what, given)
    assert (r.mean is not None) == (norm == "layer") and (r.rstd is not None) == (norm is not None)
    if r.rstd is not None:
        e = U * 24 * st[1] + eh.amax(-1, keepdim=True) * st[1] * st[1] * 2
        assert_within(r.rstd, st[1].reshape(-1), e.reshape(-1), what + " rstd")
    if r.mean is not None:
        dev = (h - h.mean(-1, keepdim=True)).abs().amax(-1, keepdim=True)
        e = U * (h.abs().amax(-1, keepdim=True) + 8 * dev) + 2 * eh.amax(-1, keepdim=True)
        assert_within(r.mean, st[0].reshape(-1), e.reshape(-1), what + " mean")
    if read:
        check_read(r.q, r.scale, scaling, g, what)
    return r


SCALINGS = [("row", None), ("group", 32), ("group", 64), ("group", 128), ("pow2", 32), ("pow2", 64), ("pow2", 128)]
WIDTHS = [1, 2, 4, 7, 8, 12, 31, 33, 64, 100, 250, 256, 264, 516, 768, 1000, 1001, 2050, 4096, 4097, 4104, 8192]
KINDS = [("rms", False), ("layer", True), (None, False), ("rms", True), ("layer", False)]


@DTYPES
@pytest.mark.parametrize("i,H", list(enumerate(WIDTHS)))
def test_widths(dtype, i, H):
    for j, (scaling, group) in enumerate(SCALINGS):
        norm, beta = KINDS[(i + j) % len(KINDS)]
        fmt = ["e4m3", "e5m2", "int8"][(i + j) % 3]
        rows = [5, 1, 3, 2][(i + j) % 4]
        v = make((rows, H), dtype, norm, beta, residual=j % 3 != 2, seed=100 * i + j)
        check_fwd(v, norm, fmt, scaling, group, major=j % 2 == 1, what=f"{rows}x{H} {norm} {fmt} {scaling} {group}")


@DTYPES
@FORMATS
@pytest.mark.parametrize("scaling,group", [("row", None), ("group", 128), ("pow2", 32)])
def test_shapes(dtype, fmt, scaling, group):
    for shape in ((300, 768), (2, 40, 264), (161, 1001), (7, 3, 5, 64)):
        v = make(shape, dtype, "rms", seed=shape[-1])
        r = check_fwd(v, "rms", fmt, scaling, group, what=f"{shape}")
        G = -(-shape[-1] // group) if group else 1
        assert r.scale.shape == (*shape[:-1], G)


@pytest.mark.parametrize("dtype,H", [(F32, 8193), (F32, 16384), (F16, 16400), (BF16, 32767), (BF16, 32768)])
@pytest.mark.parametrize("scaling,group", [("row", None), ("group", 128), ("pow2", 64)])
def test_longest_rows(dtype, H, scaling, group):
    for norm, beta in (("rms", False), ("layer", True)):
        v = make((3, H), dtype, norm, beta, seed=H)
        check_fwd(v, norm, "e4m3", scaling, group, what=f"{H}")


@DTYPES
@FORMATS
def test_given_scale(dtype, fmt):
    for H in (768, 1001):
        v = make((6, H), dtype, "rms", seed=H)
        for given in (0.01, 1.0 / 448, 5.0 / TOP[fmt], 1e-30):
            check_fwd(v, "rms", fmt, "tensor", given=given, what=f"given {given}", read=given > 1e-20)


@DTYPES
@pytest.mark.parametrize("H", [5, 520, 768, 4099])
@pytest.mark.parametrize("scaling,group", [("row", None), ("group", 64), ("pow2", 32)])
def test_off_the_borders(dtype, H, scaling, group):
    # every tensor at a distance of its own; nothing beside the outputs is written
    rows = 6
    v = make((rows, H), dtype, "layer", True, seed=H)
    h, y, _, eh, ey = norm_quant(v["x"], v["residual"], "layer", v["gamma"], v["beta"], 1e-5)
    G = -(-H // group) if group else 1
    for k, fmt in ((0, "e4m3"), (1, "int8"), (5, "e5m2")):
        qb = torch.full((rows * H + 32,), 0x55, dtype=torch.uint8, device="cuda")
        q = qb[k:k + rows * H].view(TORCH[fmt]).view(rows, H)
        hb = torch.full((rows * H + 32,), 7.0, dtype=dtype, device="cuda")
        ho = hb[k + 1:k + 1 + rows * H].view(rows, H)
        if scaling == "pow2":
            sb = torch.full((rows * G + 32,), 0x55, dtype=torch.uint8, device="cuda")
            sc = sb[k:k + rows * G].view(torch.float8_e8m0fnu).view(rows, G)
        else:
            sb = torch.full((rows * G + 32,), 7.0, device="cuda")
            sc = sb[k:k + rows * G].view(rows, G)
        mba.norm_quant_fwd(at_offset(v["x"], k)[0], at_offset(v["residual"], 2)[0], q, sc, ho, norm="layer",
                           gamma=at_offset(v["gamma"], 1)[0], beta=at_offset(v["beta"], 3)[0])
        assert_within(ho, h, eh, "h")
        check(q.cpu().float(), sc.cpu().float(), y, ey, fmt, scaling, group, f"{H} {fmt}")
        if scaling != "row" or H > 1:
            out, whole = at_offset(torch.zeros(rows, H, dtype=dtype), k + 2)
            old = whole.clone()
            mba.dequant_rows(q, sc, out)
            assert torch.equal(out, mba.dequantise(q.clone(), sc.clone(), dtype=dtype))
            out.zero_()
            assert torch.equal(whole, old)
        for b, t, fill in ((qb, q, 0x55), (hb, ho, 7.0), (sb, sc, 7.0 if sb.dtype is F32 else 0x55)):
            n = t.numel()
            first = (t.data_ptr() - b.data_ptr()) // b.element_size()
            assert (b[:first] == fill).all() and (b[first + n:] == fill).all()


@DTYPES
def test_in_place(dtype):
    for H in (768, 1001):
        v = make((40, H), dtype, "rms", seed=4)
        d = cuda(v)
        r = mba.norm_quant(d["x"], d["residual"], gamma=d["gamma"])
        for which in ("x", "residual"):
            x, res = d["x"].clone(), d["residual"].clone()
            q, s = torch.empty_like(r.q), torch.empty_like(r.scale)
            mba.norm_quant_fwd(x, res, q, s, x if which == "x" else res, gamma=d["gamma"])
            assert torch.equal(x if which == "x" else res, r.h)
            assert torch.equal(q.view(torch.uint8), r.q.view(torch.uint8)) and torch.equal(s, r.scale)


@DTYPES
@FORMATS
def test_rows_and_groups_of_zeros(dtype, fmt):
    x = torch.zeros(3, 264, dtype=dtype)
    x[1, 200:] = 1.5
    for scaling in ("row", "group", "pow2"):
        r = mba.norm_quant(x.cuda(), norm=None, format=fmt, scaling=scaling)
        assert not r.q[0].cpu().float().any()
        s = r.scale.cpu().float()
        assert (s[0] == LEAST).all() and (s[2] == LEAST).all()
        assert torch.equal(mba.dequantise(r.q, r.scale, dtype=dtype).cpu()[1] != 0, x[1] != 0)


@DTYPES
@FORMATS
@pytest.mark.parametrize("scaling,group", [("group", 64), ("pow2", 32), ("row", None)])
def test_groups_of_zeros_in_small_rows(dtype, fmt, scaling, group):
    # 1 / scale of the zeros times the row's 1 / rms is beyond fp32
    x = torch.zeros(3, 264, dtype=dtype)
    x[0, 128:] = randn((136,), dtype, 1, 1e-3)
    x[1, :7] = randn((7,), dtype, 2, 1e-3)
    v = {"x": x, "residual": None, "gamma": randn((264,), seed=3, sc=0.1, loc=1.0), "beta": None}
    check_fwd(v, "rms", fmt, scaling, group, eps=1e-8)


@DTYPES
@FORMATS
def test_infinities_and_nan(dtype, fmt):
    H = 264
    x = randn((4, H), dtype, 1)
    x[1, 40], x[2, 200], x[3, 263] = float("nan"), float("inf"), float("-inf")
    whole = {"row": H, "group": 128, "pow2": 32}
    for scaling, g in whole.items():
        r = mba.norm_quant(x.cuda(), norm=None, format=fmt, scaling=scaling)
        s, q = r.scale.cpu().float(), r.q.cpu().float()
        bad = torch.zeros(4, H, dtype=torch.bool)
        for row, c in ((1, 40), (2, 200), (3, 263)):
            bad[row, c // g * g:(c // g + 1) * g] = True
        sbad = s.isnan().repeat_interleave(g, 1)[:, :H]
        assert torch.equal(sbad, bad)
        if fmt == "int8":
            assert not q[bad].any()
        else:
            assert q[bad].isnan().all()
        assert q[~bad].isfinite().all()
        back = mba.dequantise(r.q, r.scale, dtype=F32).cpu()
        assert back[bad].isnan().all() and back[~bad].isfinite().all()
        # a norm carries them through the row
        n = mba.norm_quant(x.cuda(), norm="rms", gamma=torch.ones(H, device="cuda"), format=fmt, scaling="row")
        assert n.scale.cpu().isnan().view(-1).tolist() == [False, True, True, True]
    # a given scale cuts infinities and keeps NaN
    r = mba.norm_quant(x.cuda(), norm=None, format=fmt, scaling="tensor", scale=torch.tensor(0.5, device="cuda"))
    q = r.q.cpu().float()
    assert q[2, 200] == TOP[fmt] and q[3, 263] == -TOP[fmt]
    assert q[1, 40] == 0 if fmt == "int8" else q[1, 40].isnan()


@DTYPES
@FORMATS
@pytest.mark.parametrize("scaling,group", [("row", None), ("group", 32), ("pow2", 64)])
def test_lowest_values(dtype, fmt, scaling, group):
    # a mask's lowest values: where the sum of squares passes fp32, 1 / rms is 0 and
    # so is the row; fp16's lowest is an ordinary number
    low = torch.finfo(dtype).min
    x = randn((3, 264), dtype, 1)
    x[1, 40:200], x[2, 7] = low, -low
    gamma = randn((264,), seed=2, sc=0.1, loc=1.5)
    v = {"x": x, "residual": None, "gamma": gamma, "beta": None}
    r = mba.norm_quant(x.cuda(), gamma=gamma.cuda(), format=fmt, scaling=scaling, group=group, want_stats=True)
    if dtype is F16:
        check_fwd(v, "rms", fmt, scaling, group)
    else:
        assert not r.q[1:].cpu().float().any() and (r.scale[1:].cpu().float() == LEAST).all()
        assert r.rstd[1:].tolist() == [0.0, 0.0] and r.q[0].cpu().float().any()


@DTYPES
def test_wide_gammas(dtype):
    x = randn((5, 264), dtype, 1)
    for g in (1e-6, 1e-3, 1e3, 1e6):
        v = {"x": x, "residual": None, "gamma": randn((264,), seed=2, sc=g), "beta": None}
        for scaling, group in (("row", None), ("group", 32), ("pow2", 32)):
            check_fwd(v, "rms", "e4m3", scaling, group, read=False)


@FORMATS
def test_powers_of_two_at_their_borders(fmt):
    # a row's largest value at the format's largest times a power of two, and
    # one step of fp32 above and below it
    top = torch.tensor(TOP[fmt])
    at = []
    for e in (-100, -20, -1, 0, 1, 40, 100):
        b = top * 2.0 ** e
        at += [torch.nextafter(b, torch.tensor(0.0)), b, torch.nextafter(b, torch.tensor(float("inf")))]
    x = torch.zeros(len(at), 32)
    x[:, 3] = torch.stack(at)
    r = mba.norm_quant(x.cuda(), norm=None, format=fmt, scaling="pow2")
    want = [2.0 ** e for e in (-100, -20, -1, 0, 1, 40, 100) for e in (e, e, e + 1)]
    assert r.scale.cpu().float().view(-1).tolist() == want
    assert (r.q.cpu().float()[:, 3] <= TOP[fmt]).all()


@FORMATS
def test_every_value_of_16_bits(fmt):
    # all finite fp16 numbers under a scale of 1: torch's own conversion
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(F16)
    v = v[v.isfinite()]
    r = mba.norm_quant(v.view(1, -1)[:, :32000].cuda(), norm=None, format=fmt, scaling="tensor", scale=torch.ones(1, device="cuda"))
    x = v[:32000].double()
    assert torch.equal(r.q.cpu().float().double().view(-1), to_grid(x, fmt))
    # and all 8-bit values come back
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(TORCH[fmt]).view(1, 256)
    want = q.float()
    for dt in (F32, F16, BF16):
        got = mba.dequantise(q.cuda(), torch.ones(1, device="cuda"), dtype=dt).cpu().float()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])


def test_read_back_of_the_least_scales():
    q = torch.ones(4, 32).to(torch.float8_e4m3fn).cuda()
    s = torch.tensor([[0], [1], [127], [255]], dtype=torch.uint8).view(torch.float8_e8m0fnu).cuda()
    got = mba.dequantise(q, s, dtype=F32).cpu()[:, 0]
    assert got[:3].tolist() == [2.0 ** -127, 2.0 ** -126, 1.0] and got[3].isnan()


@DTYPES
def test_one_dimension(dtype):
    # a single row without leading sizes
    for H in (20, 264):
        x = randn((H,), dtype, 1)
        for scaling, group in SCALINGS:
            r = mba.norm_quant(x.cuda(), norm=None, scaling=scaling, group=group)
            two = mba.norm_quant(x.cuda().view(1, H), norm=None, scaling=scaling, group=group)
            assert r.q.shape == (H,) and r.scale.shape == two.scale.shape[1:]
            a, b = mba.dequantise(r.q, r.scale), mba.dequantise(two.q, two.scale)
            assert torch.equal(a, b[0])


def test_no_rows_and_one_column():
    e = torch.empty(0, 64, device="cuda", dtype=BF16)
    r = mba.norm_quant(e, e, gamma=torch.ones(64, device="cuda"), scaling="group")
    assert r.q.shape == (0, 64) and r.scale.shape == (0, 1) and r.h.shape == (0, 64)
    assert mba.dequantise(r.q, r.scale).shape == (0, 64)


@pytest.mark.slow
def test_rows_past_32_bits():
    rows, H = 66000, 32768  # above 2^31 elements
    x = torch.zeros(rows, H, dtype=BF16, device="cuda")
    at = [0, 65535, 65536, rows - 1]
    part = randn((4, H), BF16, 3)
    x[at] = part.cuda()
    gamma = randn((H,), seed=4, loc=1.0)
    r = mba.norm_quant(x, norm="rms", gamma=gamma.cuda(), scaling="group", group_major=True)
    _, y, _, _, ey = norm_quant(part, None, "rms", gamma, None, 1e-5)
    check(r.q[at].cpu().float(), r.scale[at].cpu(), y, ey, "e4m3", "group", 128, "rows")
    back = mba.dequantise(r.q, r.scale)
    want = values(r.q[at], r.scale[at], "group", 128)
    assert_within(back[at], want, U * want.abs(), "read back")


def test_training_with_what_q_stands_for():
    # straight through: block_norm's backward at the same h and statistics
    v = make((40, 264), F32, "layer", True, seed=9)
    d = cuda(v)
    r = mba.norm_quant(d["x"], d["residual"], norm="layer", gamma=d["gamma"], beta=d["beta"], want_stats=True)
    dy = randn((40, 264), seed=3).cuda()
    g = mba.block_norm_backward(dy, None, None, r.h, (None, None, r.mean, r.rstd), pre="layer", pre_gamma=d["gamma"],
                                pre_beta=d["beta"])
    t = {k: v[k].double().requires_grad_(True) for k in ("x", "gamma", "beta")}
    h = t["x"] + v["residual"].double()
    c = h - h.mean(-1, keepdim=True)
    (c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * t["gamma"] + t["beta"]).backward(dy.cpu().double())
    # fp32 sums of up to 264 terms, at 32 u of their magnitudes
    for got, want in ((g.dx, t["x"].grad), (g.dpre_gamma, t["gamma"].grad), (g.dpre_beta, t["beta"].grad)):
        assert (got.cpu().double() - want).abs().max() < 1e-4 * (1 + want.abs().max())


def test_a_step_of_a_model():
    """Dropout boundary in training, the same boundary served with 8 bits, and
    the values read back: at p = 0 the 8-bit output is y's rounding."""
    f, x = randn((64, 768), BF16, 1).cuda(), randn((64, 768), BF16, 2).cuda()
    gamma = randn((768,), seed=3, sc=0.1, loc=1.0).cuda()
    h, y, _ = mba.dropout_add_norm(f, x, p=0.0, rng=(0, 0), norm="rms", gamma=gamma)
    h2, y2, _ = mba.block_norm(f, x, pre="rms", pre_gamma=gamma)
    r = mba.norm_quant(f, x, norm="rms", gamma=gamma, scaling="group")
    assert torch.equal(h, r.h) and torch.equal(h, h2)
    back = mba.dequantise(r.q, r.scale).cpu().double()
    yd = y.cpu().double()
    amax = yd.abs().view(64, 6, 128).amax(-1).repeat_interleave(128, 1)
    # e4m3: half a step of 2^-4 of the value, or of the least normal number's
    # 2^-10 of 448 at the group's scale; bf16 twice, 2^-8 each
    assert ((back - yd).abs() <= yd.abs() * (2.0 ** -4 + 2.0 ** -7) + amax / 448 * 2.0 ** -10).all()
    # dropped: what is read back is the dropped rows' norm
    hd, yd, _ = mba.dropout_add_norm(f, x, p=0.3, rng=(1, 2), norm="rms", gamma=gamma)
    d = mba.dropout(f, 0.3, (1, 2))
    # x + d with d rounded to bf16: one more rounding of d
    assert ((hd - (x + d)).abs().float() <= d.abs().float() * 2.0 ** -8 + hd.abs().float() * 2.0 ** -7).all()


def test_captured_and_other_streams():
    v = make((333, 1001), BF16, "layer", True, seed=5)
    d = cuda(v)
    kw = dict(norm="layer", gamma=d["gamma"], beta=d["beta"], scaling="group", format="int8")
    a = mba.norm_quant(d["x"], d["residual"], **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = mba.norm_quant(d["x"], d["residual"], stream=s, **kw)
    back = mba.dequantise(b.q, b.scale, stream=s.cuda_stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = mba.norm_quant(d["x"], d["residual"], **kw)
        back2 = mba.dequantise(c.q, c.scale)
    c.q.zero_(), c.h.zero_(), back2.zero_()
    g.replay()
    torch.cuda.synchronize()
    for o in (b, c):
        assert torch.equal(a.q, o.q) and torch.equal(a.scale, o.scale) and torch.equal(a.h, o.h)
    assert torch.equal(back, back2)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(mba.AddLNError):
        mba.norm_quant(x)  # no gamma
    with pytest.raises(mba.AddLNError):
        mba.norm_quant(x, norm=None, gamma=w)
    for bad in (dict(format="e3m4"), dict(scaling="column"), dict(scaling="group", group=16), dict(group=32), dict(norm="l2"),
                dict(scale=torch.ones(1, device="cuda")), dict(gamma=w[:8].clone()), dict(gamma=w.half())):
        with pytest.raises(ValueError):
            mba.norm_quant(x, **{"gamma": w, **bad})
    with pytest.raises(TypeError):
        mba.norm_quant(x, gamma=w, scaling="tensor")
    with pytest.raises(ValueError):
        mba.norm_quant(x, x.half(), gamma=w)
    with pytest.raises(ValueError):
        mba.norm_quant(x.t(), gamma=w[:4].clone())
    r = mba.norm_quant(x, gamma=w)
    for q, s in ((x, r.scale), (r.q, r.scale[:2]), (r.q, r.scale.cpu()), (r.q.t(), r.scale), (r.q, r.scale.half())):
        with pytest.raises(ValueError):
            mba.dequantise(q, s)
    with pytest.raises(ValueError):
        mba.dequantise(r.q, r.scale, dtype=torch.float64)
    with pytest.raises(ValueError):
        mba.dequant_rows(r.q, r.scale, torch.empty(64, 4, device="cuda"))
    with pytest.raises(ValueError):
        mba.norm_quant_fwd(x, None, torch.empty(4, 64, device="cuda"), r.scale, gamma=w)


def test_written_tensors_change_their_version():
    x = torch.zeros(4, 64, device="cuda")
    r = mba.norm_quant(x, norm=None)
    v = r.q._version, r.scale._version
    mba.norm_quant_fwd(x, None, r.q, r.scale, norm=None)
    assert r.q._version > v[0] and r.scale._version > v[1]
    out = torch.empty_like(x)
    v = out._version
    mba.dequant_rows(r.q, r.scale, out)
    assert out._version > v
