"""Which masks the autograd forms and the module draw."""
from __future__ import annotations

import copy

import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from test_gpu_drop import F32, _built, mba, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make", [list, np.array], ids=["list", "array"])
def test_an_rng_that_is_changed_before_the_backward(make):
    x, w = randn((50, 33), seed=1).cuda().requires_grad_(True), randn((50, 33), seed=2).cuda()
    rng = make([1, 2])
    y = mba.dropout_train(x, 0.3, rng)
    rng[1] += 1
    (y * w).sum().backward()
    assert torch.equal(x.grad, mba.dropout(w, 0.3, (1, 2)))
    rng = make([1, 2])
    x.grad = None
    h, y = mba.dropout_add_norm_train(x, p=0.3, rng=rng, norm=None)
    rng[0] = 9
    (h * w).sum().backward()
    assert torch.equal(x.grad, mba.dropout(w, 0.3, (1, 2)))


def step(f, x, call):
    leaf = f.clone().requires_grad_(True)
    h, y = call(leaf, x)
    (h.square() + y).sum().backward()
    return h.detach(), leaf.grad


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_step_that_is_computed_again(reentrant):
    m = mba.FusedDropoutAddNorm(264, p=0.25, input_bias=True, device="cuda")
    f, x = randn((12, 264), F32, 1).cuda(), randn((12, 264), F32, 2).cuda()
    again = lambda *rng: lambda a, b: checkpoint(m, a, b, *rng, use_reentrant=reentrant)  # noqa: E731
    # the module's own offset has moved on by then: another mask, so it is refused
    with pytest.raises(RuntimeError, match="rng"):
        step(f, x, again())
    for rng in ((int(m.rng[0]), 7), m.rng.clone()):
        want = step(f, x, lambda a, b: m(a, b, rng))
        got = step(f, x, again(rng))
        assert all(map(torch.equal, got, want))
    # without dropout there is nothing to draw
    m.eval()
    assert all(map(torch.equal, step(f, x, again()), step(f, x, m)))


def test_copies_draw_their_own_masks():
    m = mba.FusedDropoutAddNorm(264, p=0.5, device="cuda")
    f, x = randn((12, 264), F32, 1).cuda(), randn((12, 264), F32, 2).cuda()
    m(f, x)
    c = copy.deepcopy(m)
    seen = [(int(v.rng[0]), int(v.rng[1])) for v in (m, c)]
    assert seen[0][0] != seen[1][0]
    assert not torch.equal(m(f, x)[0], c(f, x)[0])
    # a state is continued by loading it
    c.load_state_dict(m.state_dict())
    assert torch.equal(c.rng, m.rng) and c.rng.data_ptr() != m.rng.data_ptr()
    assert torch.equal(m(f, x)[0], c(f, x)[0])


def test_a_captured_step_that_is_computed_again():
    # as the module's docstring has it: every replay draws the next mask, for its backward too
    m = mba.FusedDropoutAddNorm(768, p=0.5, norm="rms", bias=False, device="cuda")
    f, x = randn((64, 768), seed=1).cuda().requires_grad_(True), randn((64, 768), seed=2).cuda()

    def train():
        rng = m.rng.clone()
        m.rng[1] += 1
        h, y = checkpoint(m, f, x, rng, use_reentrant=False, preserve_rng_state=False)
        (h.square() + y).sum().backward()
        return h

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            train()
    torch.cuda.current_stream().wait_stream(s)
    f.grad = m.weight.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = train()
    seed, at = m.rng.tolist()
    for i in range(3):
        f.grad.zero_(), m.weight.grad.zero_()
        g.replay()
        want = step(f.detach(), x, lambda a, b: m(a, b, (seed, at + i)))
        assert torch.equal(h, want[0]) and torch.equal(f.grad, want[1])
    assert m.rng.tolist() == [seed, at + 3]
