"""What the dropout operators' autograd forms keep for their backward, without a GPU."""
from __future__ import annotations

import copy

import numpy as np
import pytest
import torch

from memory_bound_add_gb300.drop import FusedDropoutAddNorm, _frozen, _rng_args


def test_a_kept_rng_does_not_follow_what_it_was_made_of():
    for rng in ([3, 4], np.array([3, 4]), torch.tensor([3, 4]), (torch.tensor(3), torch.tensor(4))):
        kept = _frozen(rng)
        v = rng[1]
        v += 1  # a tensor's in place
        if not isinstance(rng, tuple):
            rng[1] = v
        assert [int(v) for v in kept] == [3, 4]
    assert _rng_args(_frozen([3, 4]), 0) == (None, 3, 4)
    assert _frozen((3, 4)) == (3, 4) and _frozen(7) == 7


def test_no_mask_is_drawn_during_a_backward():
    m, x = FusedDropoutAddNorm(8, p=0.5), torch.zeros(2, 8)
    calls = [lambda: m(x, x), lambda: m(x, x, (1, 2)), lambda: m.eval()(x, x)]
    wants = [RuntimeError, ValueError, ValueError]  # the others are refused for not being on a GPU

    class Again(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            return a * 1

        @staticmethod
        def backward(ctx, g):
            for call, want in zip(calls, wants):
                with pytest.raises(want, match="rng" if want is RuntimeError else "CUDA"):
                    call()
            return g

    with pytest.raises(ValueError, match="CUDA"):
        m(x, x)
    Again.apply(torch.zeros(3, requires_grad=True)).sum().backward()
    assert m.rng[1] == 0


def test_copies_have_seeds_of_their_own():
    m = FusedDropoutAddNorm(8, p=0.5, input_bias=True)
    m.rng[1] = 5
    m.weight.data.fill_(3.0)
    layers = torch.nn.ModuleList([copy.deepcopy(m) for _ in range(3)])
    assert len({int(v.rng[0]) for v in (m, *layers)}) == 4 and all(int(v.rng[1]) == 0 for v in layers)
    c = copy.deepcopy(layers)[0]
    assert c.rng[0] != layers[0].rng[0] and c.weight[0] == 3.0 and c.weight is not m.weight and c.training
    assert {n for n, _ in c.named_parameters()} == {"weight", "bias", "input_bias"}
    # one module twice stays one module
    assert len({id(v) for v in copy.deepcopy([m, m])}) == 1
    # a state is continued by loading it
    c.load_state_dict(m.state_dict())
    assert torch.equal(c.rng, m.rng) and c.rng.data_ptr() != m.rng.data_ptr()
