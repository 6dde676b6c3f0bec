"""The extension that makes the commonest calls of ``drop`` and ``quant``.

``csrc/fast.cpp`` checks the same things as their Python and calls the same
entry points of the library; what it does not take (another device or stream,
tensors that have to be refused) it leaves to them.  Without it every call takes
the Python path.
"""
from __future__ import annotations

import ctypes
import importlib.util

from . import binding
from .build import fast_lib

_ENTRIES = ("dropout_fwd", "dropout_add_norm_fwd", "dropout_add_norm_bwd", "dropout_add_norm_bwd_workspace_size",
            "norm_quant_fwd", "dequant_rows")
_module = False  # not looked for yet


def module():
    """The extension, which calls binding.lib(), or None where there is none."""
    global _module
    if _module is False:
        handle = binding.lib()
        try:
            spec = importlib.util.spec_from_file_location("addln_fast", fast_lib())
            found = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(found)
            found.init(*(ctypes.cast(getattr(handle, n), ctypes.c_void_p).value for n in _ENTRIES))
        except (ImportError, OSError):  # not built, or for another PyTorch
            found = None
        _module = found
    return _module
