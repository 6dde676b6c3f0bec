"""Global gradient norm and clipping against 64 bits.

With u = 2^-24: a thread sums at most 33 squares in fp32 over four
accumulators (9 roundings, 2 more to join them, one of the square each: 12 u
relative, all terms being positive); the shares are added as hi + lo, whose
roundings are of order u^2 each, and rounded to fp32 once (1 u).  The root
halves that, and its own rounding and scale's product add 2 u: below 12 u.  The
factor adds the roundings of
norm + 1e-6, the quotient and scale's product (3 u), out one more beside its
own rounding: below 17 u."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24
TINY = {F32: 2.0 ** -150, F16: 2.0 ** -25, BF16: 2.0 ** -134}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import build
    build()
    yield
    torch.cuda.synchronize()
    assert mba.addln_get_device_error() == 0


def exact_norm(gs, scale=1.0):
    return scale * math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))


def check(gs, outs, norm, max_norm, scale=1.0):
    """outs against the gradients gs as they were."""
    want = exact_norm(gs, scale)
    assert abs(float(norm) - want) <= 12 * U * want + 2.0 ** -150, (float(norm), want)
    c = scale * min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(gs, outs):
        w = g.double() * c
        err = (o.double() - w).abs()
        bound = w.abs() * (17 * U + torch.finfo(o.dtype).eps / 2 * (1 + 17 * U)) + TINY[o.dtype]
        assert bool((err <= bound).all()), float((err - bound).max())


def draw(sizes, dtype, seed=0, scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dts = [F32, F16, BF16]
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dts[i % 3] if dtype == "mixed" else dtype)
            for i, n in enumerate(sizes)]


SIZES = [[1], [7], [8], [9], [255, 0, 1], [4096], [2047, 2048, 2049], [100000, 3, 65537, 0, 12], [0, 0, 5, 0],
         [5000000, 31]]


@pytest.mark.parametrize("dtype", [F32, F16, BF16, "mixed"], ids=["fp32", "fp16", "bf16", "mixed"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_sizes(dtype, i):
    gs = draw(SIZES[i], dtype, seed=i)
    assert float(mba.grad_norm(gs)) == pytest.approx(exact_norm(gs), rel=12 * U)
    for max_norm, scale in ((1e-3, 1.0), (1e9, 0.25), (1e-3, 1 / 64)):
        for out_dtype in (None, F32):
            outs = [torch.empty_like(g, dtype=out_dtype or g.dtype) for g in gs]
            norm = mba.clip_grads(gs, max_norm, out=outs, scale=scale)
            check(gs, outs, norm, max_norm, scale)
    mine = [g.clone() for g in gs]
    norm = mba.clip_grads(mine, 1e-3)
    check(gs, mine, norm, 1e-3)
    mine = [g.clone() for g in gs]
    norm = mba.clip_grads(mine, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(gs, mine))


@pytest.mark.parametrize("count", [1, 119, 120, 121, 999, 1000, 1001, 2300])
def test_numbers_of_tensors(count):
    # one, two and more launches; empty ones among them and behind the last
    sizes = [(i * 37) % 200 for i in range(count)] + [0, 0, 0]
    gs = draw(sizes, "mixed", seed=count)
    mine = [g.clone() for g in gs]
    norm = mba.clip_grads(mine, 0.01)
    check(gs, mine, norm, 0.01)
    assert float(mba.grad_norm(gs)) == float(norm)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_addresses(dtype):
    # gradients at every element offset of one buffer; outs at the same
    # offsets, and at others (no common place for 16-byte accesses)
    flat = draw([40000], dtype, seed=3)[0]
    at, gs = 0, []
    for i in range(17):
        gs.append(flat[at:at + 2000 + i])
        at += 2000 + i + 1
    for out_dtype in {dtype, F32}:
        for shift in (0, 1, 3):
            buf = torch.full((40100,), 5.0, dtype=out_dtype, device="cuda")
            at, outs = shift, []
            for g in gs:
                outs.append(buf[at:at + g.numel()])
                at += g.numel() + 1
            norm = mba.clip_grads(gs, 0.01, out=outs)
            check(gs, outs, norm, 0.01)
            # the elements between the outs are left as they were
            for o in outs:
                o.fill_(5.0)
            assert bool((buf == 5.0).all())


def test_orders_of_dimensions():
    g = torch.randn(48, 40, device="cuda")
    gs = [g.t(), torch.randn(4, 6, 5, 3, device="cuda").to(memory_format=torch.channels_last)]
    before = [t.clone() for t in gs]
    norm = mba.clip_grads(gs, 0.5)
    check(before, gs, norm, 0.5)
    for bad in (g[:, :20], torch.ones(4, 1, device="cuda").expand(4, 8), torch.ones(8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            mba.clip_grads([bad], 1.0)
        with pytest.raises(ValueError):
            mba.grad_norm([bad])
    with pytest.raises(ValueError):
        mba.clip_grads([g.t()], 1.0, out=[torch.empty(40, 48, device="cuda")])


@pytest.mark.parametrize("mag", [1e-40, 1e-30, 1e-22, 1e-15, 1e15, 1e20, 3e37])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_whose_squares_leave_fp32(mag, dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    big = (torch.rand(5001, generator=g, device="cuda") + 0.5).mul(mag).to(dtype)
    rest = torch.zeros(9000, dtype=dtype, device="cuda")
    want = exact_norm([big, rest])
    got = float(mba.grad_norm([big, rest]))
    if want > torch.finfo(F32).max:
        assert got == math.inf
    else:
        assert abs(got - want) <= 12 * U * want + 2.0 ** -150, (got, want)
    # beside ordinary values: a few huge among many, many tiny beside few
    mixed = torch.randn(5001, generator=g, device="cuda").to(dtype)
    mixed[17] = mag
    want = exact_norm([mixed])
    assert abs(float(mba.grad_norm([mixed])) - want) <= 12 * U * want


@pytest.mark.parametrize("n", [1, 3, 8, 13, 4099])
@pytest.mark.parametrize("off", [0, 1, 5])
def test_bf16_of_the_largest_exponents(n, off):
    # bit patterns that would be NaN in the other 16-bit type, also in the
    # vectors that hold a tensor's first and last elements
    big = torch.full((n + off,), 2.0 ** 125, dtype=BF16, device="cuda")[off:]
    norm = mba.grad_norm([big], scale=2.0 ** -10)
    want = 2.0 ** 115 * math.sqrt(n)
    assert abs(float(norm) - want) <= 12 * U * want
    out = [torch.empty(n, device="cuda")]
    mba.clip_grads([big], math.inf, out=out, scale=2.0 ** -10)
    assert bool((out[0] == 2.0 ** 115).all())


def test_nan_and_infinity():
    gs = draw([1000, 70], F32, seed=5)
    gs[0][3] = float("nan")
    mine = [g.clone() for g in gs]
    norm = mba.clip_grads(mine, 1.0)
    assert math.isnan(float(norm)) and all(bool(torch.isnan(g).all()) for g in mine)
    gs[0][3] = float("inf")
    mine = [g.clone() for g in gs]
    norm = mba.clip_grads(mine, 1.0)
    assert float(norm) == math.inf
    assert math.isnan(float(mine[0][3])) and not mine[1].any() and int((mine[0] != 0).sum()) == 1
    zero = [torch.zeros(100, device="cuda")]
    assert float(mba.clip_grads(zero, 1.0)) == 0.0 and not zero[0].any()
    g = draw([100], F32, seed=6)
    mine = [g[0].clone()]
    mba.clip_grads(mine, 0.0)
    assert not mine[0].any()
    mine = [g[0].clone()]
    mba.clip_grads(mine, math.inf)
    assert torch.equal(mine[0], g[0])


def test_a_norm_that_is_there_already():
    gs = draw([1000, 33], "mixed", seed=7)
    norm = torch.tensor(8.0, device="cuda")
    mine = [g.clone() for g in gs]
    got = mba.clip_grads(mine, 2.0, norm=norm, scale=0.5)
    assert got is norm
    c = 0.5 * 2.0 / (8.0 + 1e-6)
    for g, o in zip(gs, mine):
        assert bool(((o.double() - g.double() * c).abs() <= (g.double() * c).abs() *
                     (17 * U + torch.finfo(o.dtype).eps / 2) + TINY[o.dtype]).all())
    for bad in (torch.tensor(8.0), torch.tensor(8.0, device="cuda", dtype=F16), torch.ones(2, device="cuda"), 8.0):
        with pytest.raises(ValueError):
            mba.clip_grads(mine, 2.0, norm=bad)


def test_empty_lists_and_refusals():
    assert float(mba.grad_norm([])) == 0.0 and float(mba.clip_grads([], 1.0)) == 0.0
    assert float(mba.clip_grad_norm_([torch.nn.Parameter(torch.ones(3, device="cuda"))], 1.0)) == 0.0
    assert float(mba.grad_norm([torch.empty(0, device="cuda")])) == 0.0
    g = torch.ones(64, device="cuda")
    for bad in ([torch.ones(3)], [g, torch.ones(3)], [g.double()], [g.int()]):
        with pytest.raises(ValueError):
            mba.grad_norm(bad)
        with pytest.raises(ValueError):
            mba.clip_grads(bad, 1.0)
    with pytest.raises(TypeError):
        mba.grad_norm([3.0])
    with pytest.raises(ValueError):
        mba.clip_grads([g], 1.0, out=[])
    with pytest.raises(ValueError):
        mba.clip_grads([g], 1.0, out=[torch.ones(63, device="cuda")])
    for grads, out in (([g, g], None), ([g, g[10:]], None), ([g, g.clone()], [g.clone(), g])):
        with pytest.raises(mba.AddLNError) as e:
            mba.clip_grads(grads, 1.0, out=out)
        assert e.value.code == -5
    with pytest.raises(mba.AddLNError):
        mba.clip_grads([g.half()], 1.0, out=[torch.empty(64, device="cuda", dtype=BF16)])
    with pytest.raises(mba.AddLNError):
        mba.clip_grads([g], -1.0)
    with pytest.raises(mba.AddLNError):
        mba.grad_norm([g], scale=0.0)
    assert bool((g == 1).all())
    # the norm of a tensor that is listed twice counts it twice
    assert float(mba.grad_norm([g, g])) == pytest.approx(math.sqrt(128.0), rel=12 * U)


def test_streams_and_bits():
    gs = draw([1 << 20, 12345, 7], "mixed", seed=8)
    want = [g.clone() for g in gs]
    norm = mba.clip_grads(want, 0.1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        mine = [g.clone() for g in gs]
        torch.cuda.synchronize()
        n2 = mba.clip_grads(mine, 0.1, stream=stream)
        torch.cuda.synchronize()
        assert float(n2) == float(norm) and all(torch.equal(a, b) for a, b in zip(want, mine))
        assert float(mba.grad_norm(gs, stream=stream)) == float(norm)


def test_captured_and_replayed():
    gs = draw([300000, 17, 999], BF16, seed=9)
    outs = [torch.empty_like(g, dtype=F32) for g in gs]
    mba.clip_grads(gs, 0.1, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mba.clip_grads(gs, 0.1, out=outs)
    for k in range(3):
        for g in gs:
            g.normal_(std=0.01 * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        check(gs, outs, norm, 0.1)


def test_a_tensor_past_32_bits():
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[0], g[1 << 31], g[-1] = 3.0, 4.0, 12.0
    norm = mba.clip_grads([g], 6.5)
    assert float(norm) == 13.0
    for i, v in ((0, 1.5), (1 << 31, 2.0), (n - 1, 6.0)):
        assert float(g[i]) == pytest.approx(v, rel=2.0 ** -8)
    assert float(g.count_nonzero()) == 3


def test_autograd_sees_the_change():
    p = torch.nn.Parameter(torch.randn(64, device="cuda"))
    (p * p).sum().backward()
    v = p.grad._version
    mba.clip_grad_norm_([p], 0.1)
    assert p.grad._version > v


# --------------------------------------------------- a training step together
class Layer(torch.nn.Module):
    def __init__(self, H, post, pre, scale):
        super().__init__()
        self.w = torch.nn.Parameter(torch.randn(H, H) / math.sqrt(H))
        self.norm = mba.FusedBlockNorm(H, post=post, pre=pre, bias=True, layer_scale=scale, residual_scale=0.9)


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer")])
def test_training_step(post, pre):
    """Three blocks (a product, then the boundary), their gradients, and the
    clipped gradients, against the same step in 64 bits."""
    torch.manual_seed(0)
    H, shape = 128, (4, 16, 128)
    layers = torch.nn.ModuleList([Layer(H, post, pre, 0.5) for _ in range(3)]).cuda()
    x0 = torch.randn(shape, device="cuda")
    tgt = torch.randn(shape, device="cuda")

    def plain_norm(v, kind, g, b):
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * g + b

    x, y = x0, x0
    torch.backends.cuda.matmul.allow_tf32 = False
    for m in layers:
        x, y = m.norm(y @ m.w, x)
    ((y - tgt) ** 2).mean().backward()
    params = list(layers.parameters())
    before = [p.grad.clone() for p in params]
    norm = mba.clip_grad_norm_(params, 0.05)

    ref = {n: p.detach().double().requires_grad_(True) for n, p in layers.named_parameters()}
    x = y = x0.double()
    for i in range(3):
        q = lambda k: ref[f"{i}.{k}"]  # noqa: E731
        n = plain_norm(y @ q("w"), post, q("norm.post_weight"), q("norm.post_bias"))
        x = 0.9 * x + q("norm.layer_scale") * n
        y = plain_norm(x, pre, q("norm.pre_weight"), q("norm.pre_bias"))
    ((y - tgt.double()) ** 2).mean().backward()
    want = {n: t.grad for n, t in ref.items()}
    for (n, _), g in zip(layers.named_parameters(), before):
        # three layers of products of 128 terms in fp32: each carries errors
        # of below 128 u of its inputs' norm on (measured against the norm)
        assert float((g.double() - want[n]).norm()) <= 3 * 3 * 128 * U * float(want[n].norm()), n
    total = math.sqrt(sum(float((g ** 2).sum()) for g in want.values()))
    assert abs(float(norm) - total) <= 3 * 3 * 128 * U * total
    check(before, [p.grad for p in params], norm, 0.05)
    assert float(norm) > 0.05


def test_an_infinite_norm_without_a_limit():
    # max_norm infinite: no limit, so what is finite is unscaled and infinities stay
    gs = draw([1000, 70], F32, seed=11)
    gs[0][3], gs[0][5] = math.inf, -math.inf
    for scale in (1.0, 0.25):
        want = [g * scale for g in gs]
        mine = [g.clone() for g in gs]
        norm = mba.clip_grads(mine, math.inf, scale=scale)
        assert float(norm) == math.inf and all(torch.equal(a, b) for a, b in zip(mine, want))
        outs = [torch.empty_like(g) for g in gs]
        mba.clip_grads(gs, math.inf, out=outs, scale=scale, norm=norm)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a norm that leaves fp32 without an infinity among the gradients
    big = [torch.full((5000,), 2.0 ** 127, dtype=BF16, device="cuda")]
    mine = [big[0].clone()]
    assert float(mba.clip_grads(mine, math.inf)) == math.inf and torch.equal(mine[0], big[0])
    # a NaN stays one
    gs[1][0] = math.nan
    mba.clip_grads(gs, math.inf)
    assert all(bool(torch.isnan(g).all()) for g in gs)


def test_many_large_squares():
    # the squares' sum leaves fp32 although no thread's share of them does: 32
    # squares of 1.7e14 are 9e29, and 1.25e10 of them 3.6e38
    n = 12_500_000_000
    if torch.cuda.mem_get_info()[0] < 2 * n + (4 << 30):
        pytest.skip("needs 30 GB of device memory")
    g = torch.full((n,), 1.7e14, dtype=BF16, device="cuda")
    want = float(g[0]) * math.sqrt(n)
    assert 32 * float(g[0]) ** 2 < 1e30 and want ** 2 > torch.finfo(F32).max
    assert abs(float(mba.grad_norm([g])) - want) <= 12 * U * want
