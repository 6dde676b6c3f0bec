"""The extension without a GPU: it builds against the installed PyTorch, binds
to the library, and leaves what is not on a GPU to the Python path."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture(scope="module")
def ext():
    from memory_bound_add_gb300.build import build
    build()
    from memory_bound_add_gb300 import fast
    assert fast.module() is not None
    return fast.module()


def test_it_takes_nothing_without_a_gpu(ext):
    x, w = torch.zeros(4, 64), torch.ones(64)
    q, s = x.to(torch.int8), torch.ones(4, 1)
    for call in (lambda a: ext.dropout(a, 0.1, (1, 2)), lambda a: ext.dropout(a),
                 lambda a: ext.dropout_add_norm(a, None, 0.1, (1, 2), None, 1, w, None, 1e-5, False),
                 lambda a: ext.dropout_add_norm_backward(a, None, a, None, w, 0.1, (1, 2), None, 1, w, None),
                 lambda a: ext.norm_quant(a, None, w, None, 1e-5, 1, 0, 0, 0, False), lambda a: ext.dequantise(a, s, 0)):
        for a in (x, q, None, 3, "x", [x]):
            assert call(a) is None


def test_init_wants_six_addresses(ext):
    with pytest.raises(TypeError):
        ext.init(1, 2, 3)
    with pytest.raises(TypeError):
        ext.init(*"abcdef")


def test_the_python_path_refuses_what_it_leaves():
    import memory_bound_add_gb300 as mba
    x = torch.zeros(4, 64)
    for call in (lambda: mba.dropout(x, 0.1, (1, 2)), lambda: mba.dropout_add_norm(x, p=0.1, rng=(1, 2), norm=None),
                 lambda: mba.norm_quant(x, norm=None), lambda: mba.dequantise(x.to(torch.int8), torch.ones(4, 1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
