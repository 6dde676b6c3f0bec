"""Host-side checks of include/addln_quant.h (no GPU, no kernel launched):
exported symbols, binding signatures, codes, layouts of scales, and the refusal
of bad arguments before the first CUDA call (pointers are fake addresses)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

from _quant_ref import TORCH, pow2_of, to_grid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "addln_quant.h")
BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from memory_bound_add_gb300.build import build
    build()
    from memory_bound_add_gb300 import quant
    return quant.lib()


def at(i):
    return BASE + i * 0x1000000


def test_symbols_signatures_and_codes(lib):
    from memory_bound_add_gb300 import quant
    from memory_bound_add_gb300.build import LIB
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(quant.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}
    for k, v in re.findall(r"#define\s+ADDLN_(\w+)\s+(\d+)", text):
        assert getattr(quant, k) == int(v)


def fwd(lib, **kw):
    a = dict(x=at(0), r=at(1), norm=2, gamma=at(2), beta=at(3), q=at(4), format=0, scaling=1, group=32, major=0,
             scale=at(5), h=at(6), mean=at(7), rstd=at(8), rows=4, H=64, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.norm_quant_fwd(*a.values(), None)


def deq(lib, **kw):
    a = dict(q=at(0), format=0, scaling=1, group=32, major=0, scale=at(1), out=at(2), rows=4, H=64, dtype=0)
    a.update(kw)
    return lib.dequant_rows(*a.values(), None)


def test_forward_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    for kw, code in [
            (dict(dtype=3), b.ERR_DTYPE), (dict(rows=-1), b.ERR_SHAPE), (dict(H=0), b.ERR_SHAPE),
            (dict(H=16385), b.ERR_SHAPE), (dict(H=32769, dtype=2), b.ERR_SHAPE), (dict(rows=1 << 61), b.ERR_SHAPE),
            (dict(norm=3), k.ERR_KIND), (dict(norm=0), k.ERR_KIND), (dict(format=3), k.ERR_KIND),
            (dict(scaling=4), k.ERR_KIND), (dict(group=0), k.ERR_KIND), (dict(group=96), k.ERR_KIND),
            (dict(scaling=2, group=256), k.ERR_KIND), (dict(eps=-1.0), b.ERR_EPS), (dict(eps=float("nan")), b.ERR_EPS),
            (dict(x=None), b.ERR_NULL), (dict(q=None), b.ERR_NULL), (dict(scale=None), b.ERR_NULL),
            (dict(gamma=None), b.ERR_NULL), (dict(x=at(0) + 2), k.ERR_ALIGN), (dict(scale=at(5) + 1), k.ERR_ALIGN),
            (dict(gamma=at(2) + 1), k.ERR_ALIGN), (dict(h=at(0) + 16), b.ERR_ALIAS), (dict(q=at(0)), b.ERR_ALIAS),
            (dict(q=at(6) + 64), b.ERR_ALIAS), (dict(scale=at(4)), b.ERR_ALIAS), (dict(scaling=3, scale=at(4)), b.ERR_ALIAS),
            (dict(rstd=at(7)), b.ERR_ALIAS), (dict(scaling=2, scale=at(4) + 255), b.ERR_ALIAS),
            (dict(rows=0, x=None, q=None, scale=None), b.OK), (dict(rows=0, group=7), k.ERR_KIND)]:
        assert fwd(lib, **kw) == code, kw


def test_read_back_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    for kw, code in [
            (dict(dtype=3), b.ERR_DTYPE), (dict(rows=-1), b.ERR_SHAPE), (dict(H=0), b.ERR_SHAPE),
            (dict(H=32769), b.ERR_SHAPE), (dict(format=-1), k.ERR_KIND), (dict(scaling=9), k.ERR_KIND),
            (dict(group=1), k.ERR_KIND), (dict(q=None), b.ERR_NULL), (dict(scale=None), b.ERR_NULL),
            (dict(out=None), b.ERR_NULL), (dict(out=at(2) + 2), k.ERR_ALIGN), (dict(scale=at(1) + 2), k.ERR_ALIGN),
            (dict(out=at(0)), b.ERR_ALIAS), (dict(out=at(1)), b.ERR_ALIAS), (dict(rows=0, q=None), b.OK)]:
        assert deq(lib, **kw) == code, kw


def test_scale_layouts():
    from memory_bound_add_gb300.quant import SCALE_GROUP as GROUP, SCALE_POW2 as POW2, SCALE_ROW as ROW, SCALE_TENSOR as ONE
    from memory_bound_add_gb300.quant import scale_layout
    e = torch.empty
    e8 = lambda *s: torch.empty(s, dtype=torch.uint8).view(torch.float8_e8m0fnu)  # noqa: E731
    assert scale_layout(e(()), (4, 64)) == (ONE, 0, 0) and scale_layout(e(1), (1, 64)) == (ONE, 0, 0)
    assert scale_layout(e(4, 1), (4, 64)) == (ROW, 0, 0) and scale_layout(e(2, 3, 1), (6, 64)) == (ROW, 0, 0)
    assert scale_layout(e(1, 1), (1, 64)) == (ROW, 0, 0)
    for H in (1, 31, 33, 64, 65, 100, 127, 129, 4096, 5001):
        for g in (32, 64, 128):
            G = -(-H // g)
            if G > 1:
                assert scale_layout(e(4, G), (4, H)) == (GROUP, g, 0)
                assert scale_layout(e(G, 4).t(), (4, H)) == (GROUP, g, 1)
                assert scale_layout(e(G, 2, 2).movedim(0, -1), (2, 2, H)) == (GROUP, g, 1)
                assert scale_layout(e8(4, G), (4, H)) == (POW2, g, 0)
            else:
                assert scale_layout(e8(4, 1), (4, H))[0] == POW2
    for bad, shape in [(e(4, 3), (4, 64)), (e(3, 1), (4, 64)), (e(4), (4, 64)), (e(4, 4)[:, ::2], (4, 64)),
                       (e(2, 4, 2)[:, :, :1], (8, 64)), (e8(1), (1, 64)), (e(4, 1).half(), (4, 64)),
                       (e(4, 2).t(), (4, 64))]:
        with pytest.raises(ValueError):
            scale_layout(bad, shape)


def test_group_arguments():
    from memory_bound_add_gb300.quant import _format, _group_of
    assert _group_of("group", None)[1] == 128 and _group_of("pow2", None)[1] == 32 and _group_of("row", None)[1] == 0
    for bad in (("row", 32), ("group", 16), ("pow2", 0), ("tile", None), ("tensor", 128)):
        with pytest.raises(ValueError):
            _group_of(*bad)
    with pytest.raises(ValueError):
        _format("fp8")


def test_plain_grids():
    # the plain rounding is torch's own conversion, for every 16-bit float
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16).double()
    v = v[v.isfinite()]
    for fmt, top in (("e4m3", 448), ("e5m2", 57344)):
        c = v.clamp(-top, top)
        assert torch.equal(to_grid(c, fmt), c.float().to(TORCH[fmt]).double())
    assert to_grid(torch.tensor([0.5, 1.5, -2.5, 200.0], dtype=torch.float64), "int8").tolist() == [0, 2, -2, 127]
    t = torch.tensor([0.0, 1.0, 1.1, 2.0, 0.25, 0.3], dtype=torch.float64)
    assert pow2_of(t).tolist() == [0.0, 1.0, 2.0, 2.0, 0.25, 0.5]
