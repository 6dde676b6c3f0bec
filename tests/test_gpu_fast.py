"""The extension's calls against the Python path's: the same bits, the same
refusals, and calls that it has to leave to the Python path."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_drop import randn

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")
from memory_bound_add_gb300 import drop, fast, quant  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import build
    build()
    drop.lib(), quant.lib()
    yield
    torch.cuda.synchronize()
    assert mba.addln_get_device_error() == 0


class Counted:
    """The extension, counting the calls that it took."""

    def __init__(self, module):
        self.module, self.taken = module, 0

    def __getattr__(self, name):
        f = getattr(self.module, name)

        def call(*a):
            r = f(*a)
            self.taken += r is not None
            return r

        return call


@pytest.fixture
def counted(monkeypatch):
    assert fast.module() is not None
    c = Counted(fast.module())
    monkeypatch.setattr(drop, "_fast", c)
    monkeypatch.setattr(quant, "_fast", c)
    return c


def flat(r):
    if r is None or isinstance(r, torch.Tensor):
        return [r]
    return [t for x in r for t in flat(x)]


def both(counted, monkeypatch, f, taken=True):
    before = counted.taken
    a = flat(f())
    assert (counted.taken > before) == taken
    with monkeypatch.context() as m:
        m.setattr(drop, "_fast", None)
        m.setattr(quant, "_fast", None)
        b = flat(f())
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype is y.dtype and x.shape == y.shape and x.stride() == y.stride() and not x.requires_grad
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
def test_the_same_bits(counted, monkeypatch, dtype):
    w, v, b = (randn((264,), seed=i, sc=0.1, loc=1.0).cuda() for i in range(3))
    f, x = randn((3, 5, 264), dtype, 1).cuda(), randn((3, 5, 264), dtype, 2).cuda()
    dev = torch.tensor([3, 4], device="cuda")
    for rng in ((3, 4), ((1 << 64) - 1, 1 << 63), dev):
        both(counted, monkeypatch, lambda: mba.dropout(f, 0.3, rng))
        for norm, g, be, bi in (("rms", w, None, None), ("layer", w, v, b), (None, None, None, b), ("layer", w, None, None)):
            kw = dict(p=0.3, rng=rng, norm=norm, gamma=g, bias=bi)
            for stats in (False, True):
                both(counted, monkeypatch, lambda: mba.dropout_add_norm(f, x, beta=be, want_stats=stats, **kw))
            both(counted, monkeypatch, lambda: mba.dropout_add_norm(f, beta=be, **kw))
            h, y, st = mba.dropout_add_norm(f, x, beta=be, want_stats=True, **kw)
            for dy, dh in ((f, x), (f, None), (None, x)):
                if norm is None and dy is not None:
                    continue
                both(counted, monkeypatch, lambda: mba.dropout_add_norm_backward(dy, dh, h if norm else None, st, beta=be, **kw))
    for norm, g, be in (("rms", w, None), ("layer", w, v), (None, None, None)):
        for fmt in ("e4m3", "e5m2", "int8"):
            for scaling, group in (("row", None), ("group", None), ("group", 32), ("pow2", None), ("pow2", 128)):
                for r in (None, x):
                    for stats in (False, True):
                        both(counted, monkeypatch, lambda: mba.norm_quant(f, r, norm=norm, gamma=g, beta=be, format=fmt,
                                                                          scaling=scaling, group=group, want_stats=stats))
                q = mba.norm_quant(f, x, norm=norm, gamma=g, beta=be, format=fmt, scaling=scaling, group=group)
                for dt in (torch.float32, torch.float16, torch.bfloat16):
                    both(counted, monkeypatch, lambda: mba.dequantise(q.q, q.scale, dtype=dt))


def test_what_it_leaves_alone(counted, monkeypatch):
    f = randn((4, 64), seed=1).cuda()
    w = torch.ones(64, device="cuda")
    s = torch.cuda.Stream()
    leave = lambda g: both(counted, monkeypatch, g, taken=False)  # noqa: E731
    leave(lambda: mba.dropout(f, 0.1, (1, 2), stream=torch.cuda.current_stream()))
    leave(lambda: mba.dropout(f, 0.1, (-1, 2)))
    leave(lambda: mba.dropout(f, 0, (1, 2)))
    leave(lambda: mba.dropout(f[:0], 0.1, (1, 2)))
    leave(lambda: mba.dropout_add_norm(f, f.view(2, 2, 64), p=0.1, rng=(1, 2), norm="rms", gamma=w))
    leave(lambda: mba.norm_quant(f, gamma=w, scaling="group", group=32, group_major=True))
    leave(lambda: mba.norm_quant(f, gamma=w, scaling="tensor", scale=w[:1].clone()))
    q = mba.norm_quant(f, gamma=w, scaling="group", group=32, group_major=True)
    leave(lambda: mba.dequantise(q.q, q.scale))
    leave(lambda: mba.norm_quant(torch.nn.Parameter(f).detach().as_subclass(Sub), gamma=w)[:1])
    # a current stream other than the default one is its own
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        both(counted, monkeypatch, lambda: mba.dropout(f, 0.1, (1, 2)))
    torch.cuda.synchronize()
    # a parameter is a tensor like any other, and no graph is made
    both(counted, monkeypatch, lambda: mba.norm_quant(torch.nn.Parameter(f), gamma=torch.nn.Parameter(w)))
    with torch.inference_mode():
        both(counted, monkeypatch, lambda: mba.norm_quant(f, gamma=w))


class Sub(torch.Tensor):
    pass


def test_refusals_stay(counted):
    f = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for call, error in [
            (lambda: mba.dropout(f, 1.5, (1, 2)), mba.AddLNError), (lambda: mba.dropout(f, "p", (1, 2)), Exception),
            (lambda: mba.dropout(f, 0.1, (1, 1 << 64)), ValueError), (lambda: mba.dropout(f.t(), 0.1, (1, 2)), ValueError),
            (lambda: mba.dropout(f.cpu(), 0.1, (1, 2)), ValueError), (lambda: mba.dropout(f.long(), 0.1, (1, 2)), ValueError),
            (lambda: mba.dropout(None, 0.1, (1, 2)), TypeError),
            (lambda: mba.dropout_add_norm(f, f, p=0.1, rng=(1, 2), norm="rms"), mba.AddLNError),
            (lambda: mba.dropout_add_norm(f, f, p=0.1, rng=(1, 2), norm="l2", gamma=w), ValueError),
            (lambda: mba.dropout_add_norm(f, f[:2], p=0.1, rng=(1, 2), norm="rms", gamma=w), ValueError),
            (lambda: mba.dropout_add_norm(f, f.half(), p=0.1, rng=(1, 2), norm="rms", gamma=w), ValueError),
            (lambda: mba.dropout_add_norm_backward(f, None, None, None, p=0.1, rng=(1, 2), norm="rms", gamma=w), mba.AddLNError),
            (lambda: mba.dropout_add_norm_backward(None, None, None, None, p=0.1, rng=(1, 2), gamma=w), TypeError),
            (lambda: mba.norm_quant(f, gamma=w.half()), ValueError), (lambda: mba.norm_quant(f, gamma=w, eps=-1.0), mba.AddLNError),
            (lambda: mba.norm_quant(f, norm=None, gamma=w), mba.AddLNError),
            (lambda: mba.dequantise(f, w[:4].view(4, 1)), ValueError),
            (lambda: mba.dequantise(f.to(torch.int8), torch.ones(4, 3, device="cuda")), ValueError)]:
        with pytest.raises(error):
            call()
    assert counted.taken == 0


@pytest.mark.parametrize("yes,no", [(1, 0), (np.bool_(True), np.bool_(False)), ("yes", "")])
def test_truth_values_that_are_no_bools(counted, monkeypatch, yes, no):
    f, w = randn((4, 64), seed=1).cuda(), torch.ones(64, device="cuda")
    for v in (yes, no):
        for call in (lambda: mba.dropout_add_norm(f, f, p=0.1, rng=(1, 2), gamma=w, want_stats=v),
                     lambda: mba.norm_quant(f, norm="layer", gamma=w, want_stats=v)):
            both(counted, monkeypatch, call, taken=False)
    assert all(t is not None for t in mba.dropout_add_norm(f, f, p=0.1, rng=(1, 2), gamma=w, want_stats=yes)[2])
    assert mba.norm_quant(f, norm="layer", gamma=w, want_stats=yes).rstd is not None


def test_gradients_have_their_vectors_shapes(counted, monkeypatch):
    # a vector of H elements may have other sizes of 1; its gradient is like it
    f, st = randn((4, 64), seed=1).cuda(), (torch.zeros(4, device="cuda"), torch.ones(4, device="cuda"))
    for name in ("bias", "gamma", "beta"):
        kw = dict({k: torch.ones(64, device="cuda") for k in ("bias", "gamma", "beta")}, p=0.1, rng=(1, 2))
        kw[name] = kw[name].view(1, 64)
        both(counted, monkeypatch, lambda: mba.dropout_add_norm_backward(f, f, f, st, **kw), taken=False)
        assert getattr(mba.dropout_add_norm_backward(f, f, f, st, **kw), "d" + name).shape == (1, 64)
