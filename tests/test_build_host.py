"""Building without a GPU: what the extension's file is named after, and a build
where there is no PyTorch."""
from __future__ import annotations

import os
import sys
import sysconfig

import pytest
import torch

from memory_bound_add_gb300 import build as b


def test_the_extension_is_for_one_pytorch_and_one_python(monkeypatch):
    name = os.path.basename(b.fast_lib())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda k: "cpython-399-other" if k == "SOABI" else get(k))
    assert os.path.basename(b.fast_lib()) != name


def test_without_a_pytorch_the_library_is_built_alone(monkeypatch):
    b.build()
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="Python path"):
        assert b.build_fast() is None
    with pytest.warns(UserWarning, match="Python path"):
        assert b.build() == b.LIB
