"""Which masks the autograd forms and the module draw."""
from __future__ import annotations

import numpy as np
import pytest
import torch

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
