"""Host-side checks of include/addln_grad.h (no GPU, no kernel launched):
symbols, signatures, and the refusal of bad lists before the first CUDA call.
Device pointers are fake addresses; every call is refused."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "addln_grad.h")
BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from memory_bound_add_gb300.build import build
    build()
    from memory_bound_add_gb300 import grads
    return grads.lib()


def test_symbols_and_signatures(lib):
    from memory_bound_add_gb300 import grads
    from memory_bound_add_gb300.build import LIB
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(grads.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def at(i):
    return BASE + i * 0x1000000


def arr(ctype, v):
    return None if v is None else (ctype * len(v))(*v)


P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


def call(lib, which="both", g=(at(0), at(1)), o=None, n=(100, 7), d=(0, 1), od=(0, 1), count=2, scale=1.0, limit=1.0,
         norm=at(8), ws=at(9), wb=1 << 20):
    g, o, n, d, od = arr(P, g), arr(P, o), arr(I64, n), arr(I, d), arr(I, od)
    if which == "norm":
        return lib.grad_norm(g, n, d, count, scale, norm, ws, wb, None)
    if which == "clip":
        return lib.grad_clip(g, o, n, d, od, count, scale, limit, norm, None)
    return lib.grad_norm_clip(g, o, n, d, od, count, scale, limit, norm, ws, wb, None)


def test_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    nan, inf = float("nan"), float("inf")
    for which in ("both", "norm", "clip"):
        for kw, code in [
                (dict(count=-1), b.ERR_SHAPE), (dict(scale=0.0), k.ERR_SCALE), (dict(scale=-1.0), k.ERR_SCALE),
                (dict(scale=nan), k.ERR_SCALE), (dict(scale=inf), k.ERR_SCALE), (dict(g=None), b.ERR_NULL),
                (dict(n=None), b.ERR_NULL), (dict(d=None), b.ERR_NULL), (dict(d=(0, 3)), b.ERR_DTYPE),
                (dict(n=(4, -1)), b.ERR_SHAPE), (dict(n=(1 << 46, 1)), b.ERR_SHAPE),
                (dict(n=(1 << 43, 1)), b.ERR_SHAPE), (dict(g=(at(0), None)), b.ERR_NULL),
                (dict(g=(at(0) + 2, at(1))), k.ERR_ALIGN), (dict(g=(at(0), at(1) + 1)), k.ERR_ALIGN),
                (dict(norm=None), b.ERR_NULL), (dict(norm=at(8) + 2), k.ERR_ALIGN)]:
            assert call(lib, which, **kw) == code, (which, kw)
    for which in ("both", "norm"):
        for kw, code in [(dict(ws=None), b.ERR_WORKSPACE), (dict(ws=at(9) + 8), b.ERR_WORKSPACE),
                         (dict(wb=16), b.ERR_WORKSPACE), (dict(norm=at(0) + 8), b.ERR_ALIAS),
                         (dict(norm=at(9) + 64), b.ERR_ALIAS), (dict(ws=at(1)), b.ERR_ALIAS)]:
            assert call(lib, which, **kw) == code, (which, kw)
    for which in ("both", "clip"):
        for kw, code in [
                (dict(limit=-1.0), k.ERR_SCALE), (dict(limit=nan), k.ERR_SCALE),
                (dict(o=(at(3), at(4)), od=None), b.ERR_NULL), (dict(o=(at(3), None)), b.ERR_NULL),
                (dict(o=(at(3), at(4)), od=(0, 2)), b.ERR_DTYPE), (dict(o=(at(3), at(4)), od=(1, 1)), b.ERR_DTYPE),
                (dict(o=(at(3) + 2, at(4))), k.ERR_ALIGN), (dict(g=(at(0), at(0))), b.ERR_ALIAS),
                (dict(g=(at(0), at(0) + 396)), b.ERR_ALIAS), (dict(o=(at(3), at(3))), b.ERR_ALIAS),
                (dict(o=(at(0) + 4, at(4))), b.ERR_ALIAS), (dict(o=(at(1), at(4))), b.ERR_ALIAS),
                (dict(o=(at(3), at(1)), od=(0, 0)), b.ERR_ALIAS), (dict(norm=at(0) + 4), b.ERR_ALIAS)]:
            assert call(lib, which, **kw) == code, (which, kw)


def test_workspace_size(lib):
    from memory_bound_add_gb300 import binding as b
    assert lib.grad_norm_workspace_size(-1) == b.ERR_SHAPE
    sizes = [lib.grad_norm_workspace_size(n) for n in (0, 1, 119, 120, 1000, 5000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_dense():
    from memory_bound_add_gb300.grads import _dense
    e = torch.empty
    for t in (e(3, 4), e(3, 4).t(), e(2, 3, 4).permute(2, 0, 1), e(5, 1, 3), e(()), e(1, 1),
              e(2, 3, 4, 5).to(memory_format=torch.channels_last)):
        assert _dense(t)
    for t in (e(3, 4)[:, :2], e(4, 1).expand(4, 3), e(6)[::2], e(3, 8)[:, ::2]):
        assert not _dense(t)


def test_workspace_size_of_absurd_counts(lib):
    # 32 KB for each 120 tensors or part of them, or refused: never a size that
    # does not fit 64 bits
    from memory_bound_add_gb300 import binding as b
    for e in range(10, 63):
        for n in ((1 << e) - 1, 1 << e, 3 << (e - 1)):
            size = lib.grad_norm_workspace_size(n)
            assert size == (n // 120 + 1) * (1 << 15) or size == b.ERR_SHAPE and n >= 1 << 48, n
