"""What the dropout operators' autograd forms keep for their backward, without a GPU."""
from __future__ import annotations

import numpy as np
import torch

from memory_bound_add_gb300.drop import _frozen, _rng_args


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
