"""Host-side checks of include/addln_block.h (no GPU, no kernel launched):
exported symbols, binding signatures, and the refusal of bad arguments before
the first CUDA call.  Pointers are fake addresses; every call is refused."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "addln_block.h")
BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from memory_bound_add_gb300.build import build
    build()
    from memory_bound_add_gb300 import block
    return block.lib()


def header_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))


def test_symbols_signatures_and_codes(lib):
    from memory_bound_add_gb300 import block, binding
    from memory_bound_add_gb300.build import LIB
    assert header_functions() == sorted(block.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(header_functions()) <= exported
    d = {m.group(1): int(m.group(2))
         for m in re.finditer(r"#define\s+(ADDLN_\w+)\s+\(?(-?\d+)\)?", open(HEADER).read())}
    for k in ("NORM_NONE", "NORM_RMS", "NORM_LAYER", "GATE_NONE", "GATE_CHANNEL", "GATE_ROWS", "ERR_ALIGN",
              "ERR_KIND", "ERR_SCALE"):
        assert getattr(block, k) == d["ADDLN_" + k]
    for code in (block.ERR_ALIGN, block.ERR_KIND, block.ERR_SCALE, block.ERR_HOST_MEMORY):
        assert "unknown error" not in binding.strerror(code)


def at(i):
    return BASE + i * 0x1000000


def fwd(lib, **kw):
    a = dict(f=at(0), x=at(1), post=1, pg=at(2), pb=None, gate=None, gk=0, gs=0, rpg=0, a=1.0, s=1.0, pre=2,
             ng=at(3), nb=at(4), h=at(5), y=at(6), pm=None, pr=None, nm=None, nr=None, rows=4, H=8, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.block_norm_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(dy=at(0), dh=at(1), f=at(2), h=at(3), post=1, pg=at(4), pb=None, pm=None, pr=at(5), gate=None, gk=0, gs=0,
             rpg=0, a=1.0, s=1.0, pre=1, ng=at(6), nm=None, nr=at(7), df=at(8), dx=at(9), dpg=at(10), dpb=None,
             dg=None, dng=at(11), dnb=None, rows=4, H=8, dtype=0, ws=at(12), wb=1 << 20)
    a.update(kw)
    return lib.block_norm_bwd(*a.values(), None)


def test_forward_refusals(lib):
    from memory_bound_add_gb300 import block as k, binding as b
    nan, inf = float("nan"), float("inf")
    for kw, code in [
            (dict(dtype=3), b.ERR_DTYPE), (dict(rows=-1), b.ERR_SHAPE), (dict(H=0), b.ERR_SHAPE),
            (dict(H=16385), b.ERR_SHAPE), (dict(H=32769, dtype=2), b.ERR_SHAPE), (dict(rows=1 << 61), b.ERR_SHAPE),
            (dict(post=3), k.ERR_KIND), (dict(pre=-1), k.ERR_KIND), (dict(gk=3), k.ERR_KIND),
            (dict(post=0), k.ERR_KIND), (dict(pre=0), k.ERR_KIND), (dict(gate=at(9)), k.ERR_KIND),
            (dict(a=nan), k.ERR_SCALE), (dict(s=inf), k.ERR_SCALE), (dict(eps=-1.0), b.ERR_EPS),
            (dict(eps=nan), b.ERR_EPS), (dict(f=None), b.ERR_NULL), (dict(x=None), b.ERR_NULL),
            (dict(h=None), b.ERR_NULL), (dict(y=None), b.ERR_NULL), (dict(pg=None), b.ERR_NULL),
            (dict(ng=None), b.ERR_NULL), (dict(gk=1), b.ERR_NULL), (dict(gk=2, gs=8, rpg=1), b.ERR_NULL),
            (dict(gk=2, gate=at(9), gs=7, rpg=1), b.ERR_SHAPE), (dict(gk=2, gate=at(9), gs=8, rpg=0), b.ERR_SHAPE),
            (dict(gk=2, gate=at(9), gs=1 << 62, rpg=1), b.ERR_SHAPE),
            (dict(f=at(0) + 2), k.ERR_ALIGN), (dict(ng=at(3) + 1), k.ERR_ALIGN), (dict(pr=at(7) + 2), k.ERR_ALIGN),
            (dict(dtype=1, h=at(5) + 1), k.ERR_ALIGN), (dict(gk=2, gate=at(9) + 1, gs=8, rpg=2), k.ERR_ALIGN),
            (dict(h=at(0) + 16), b.ERR_ALIAS), (dict(y=at(5)), b.ERR_ALIAS), (dict(y=at(1) + 32), b.ERR_ALIAS),
            (dict(h=at(2)), b.ERR_ALIAS), (dict(pr=at(5)), b.ERR_ALIAS), (dict(pr=at(7), nr=at(7)), b.ERR_ALIAS),
            (dict(gk=2, gate=at(5) + 64, gs=8, rpg=1), b.ERR_ALIAS),
            (dict(rows=0, f=None, x=None, h=None, y=None), b.OK), (dict(rows=0, dtype=7), b.ERR_DTYPE)]:
        assert fwd(lib, **kw) == code, kw


def test_backward_refusals(lib):
    from memory_bound_add_gb300 import block as k, binding as b
    for kw, code in [
            (dict(dtype=-1), b.ERR_DTYPE), (dict(rows=-2), b.ERR_SHAPE), (dict(H=-8), b.ERR_SHAPE),
            (dict(post=9), k.ERR_KIND), (dict(post=0), k.ERR_KIND), (dict(pre=0), k.ERR_KIND),
            (dict(pre=0, dy=None, ng=None, nr=None, dng=None, dg=at(13)), k.ERR_KIND),
            (dict(a=float("inf")), k.ERR_SCALE), (dict(wb=-1), b.ERR_WORKSPACE),
            (dict(dy=None, dh=None), b.ERR_NULL), (dict(f=None), b.ERR_NULL), (dict(h=None), b.ERR_NULL),
            (dict(nr=None), b.ERR_NULL), (dict(pr=None), b.ERR_NULL), (dict(pre=2), b.ERR_NULL),
            (dict(post=2), b.ERR_NULL), (dict(df=None), b.ERR_NULL), (dict(dx=None), b.ERR_NULL),
            (dict(gk=1, dg=at(13)), b.ERR_NULL), (dict(dpg=at(10) + 2), k.ERR_ALIGN),
            (dict(dtype=1, dy=at(0) + 1), k.ERR_ALIGN), (dict(nr=at(7) + 1), k.ERR_ALIGN),
            (dict(df=at(9)), b.ERR_ALIAS), (dict(df=at(0) + 16), b.ERR_ALIAS), (dict(dpg=at(4)), b.ERR_ALIAS),
            (dict(dng=at(10)), b.ERR_ALIAS), (dict(ws=at(9)), b.ERR_ALIAS), (dict(ws=at(2)), b.ERR_ALIAS),
            (dict(gk=2, gate=at(13), gs=8, rpg=2, dg=at(13)), b.ERR_ALIAS)]:
        assert bwd(lib, **kw) == code, kw


def test_workspace_size_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    size = lib.block_norm_bwd_workspace_size
    assert size(0, 64, 0, 0, 1) == 0
    assert size(-1, 64, 0, 0, 1) == b.ERR_SHAPE
    assert size(4, 64, 5, 0, 1) == b.ERR_DTYPE
    assert size(4, 64, 0, 7, 1) == k.ERR_KIND
    assert size(4, 64, 0, 2, 0) == b.ERR_SHAPE


def test_gate_layouts():
    from memory_bound_add_gb300.block import gate_layout
    e = torch.empty
    assert gate_layout(e(6, 32), (6, 32)) == (6, 32, 1)
    assert gate_layout(e(1, 32), (6, 32)) == (1, 32, 6)
    assert gate_layout(e(3, 1, 32), (3, 5, 32)) == (3, 32, 5)
    assert gate_layout(e(3, 5, 32), (3, 5, 32)) == (15, 32, 1)
    assert gate_layout(e(3, 96)[:, 32:64].unsqueeze(1), (3, 5, 32)) == (3, 96, 5)
    assert gate_layout(e(1, 1, 32), (1, 5, 32)) == (1, 32, 5)
    assert gate_layout(e(2, 3, 1, 32), (2, 3, 4, 32)) == (6, 32, 4)
    for bad, shape in [(e(2, 32), (6, 32)), (e(1, 5, 32), (3, 5, 32)), (e(3, 1, 31), (3, 5, 32)),
                       (e(1, 32).expand(6, 32), (6, 32)), (e(32, 6).t(), (6, 32)), (e(3, 32), (3, 5, 32)),
                       (e(4, 3, 32).transpose(0, 1), (3, 4, 32))]:
        with pytest.raises(ValueError):
            gate_layout(bad, shape)


def test_the_same_rows():
    from memory_bound_add_gb300.block import _same_rows
    for a, b in [((4, 6, 32), (24, 32)), ((4, 6, 32), (24, 1, 32)), ((1, 4, 6, 32), (4, 2, 3, 32)), ((32,), (1, 32)),
                 ((5, 1, 32), (5, 32)), ((2, 3, 4, 8), (6, 4, 8)), ((7, 32), (7, 32)), ((0, 32), (0, 32))]:
        assert _same_rows(a, b) and _same_rows(b, a)
    for a, b in [((4, 6, 32), (6, 4, 32)), ((4, 6, 32), (2, 12, 32)), ((4, 64), (8, 32)), ((2, 3, 4, 8), (3, 2, 4, 8)),
                 ((), (1, 1)), ((2, 16), (32,))]:
        assert not _same_rows(a, b) and not _same_rows(b, a)


def test_gate_layouts_of_no_rows():
    # a gate of its own for every row, where there are none
    from memory_bound_add_gb300.block import gate_layout
    for shape in ((5, 0, 32), (0, 5, 32), (2, 0, 3, 32), (0, 32)):
        assert gate_layout(torch.empty(shape), shape) == (0, 32, 1)
    assert gate_layout(torch.empty(5, 0, 1, 32), (5, 0, 4, 32)) == (0, 32, 4)
    with pytest.raises(ValueError):
        gate_layout(torch.empty(5, 0, 31), (5, 0, 32))
