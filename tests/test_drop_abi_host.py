"""Host-side checks of include/addln_dropout.h (no GPU, no kernel launched):
exported symbols, binding signatures, the refusal of bad arguments before the
first CUDA call (pointers are fake addresses), and the plain generator."""
from __future__ import annotations

import os
import re
import subprocess

import numpy as np
import pytest
import torch

from _drop_ref import keep, philox, scale, threshold

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "addln_dropout.h")
BASE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from memory_bound_add_gb300.build import build
    build()
    from memory_bound_add_gb300 import drop
    return drop.lib()


def at(i):
    return BASE + i * 0x1000000


def test_symbols_and_signatures(lib):
    from memory_bound_add_gb300 import drop
    from memory_bound_add_gb300.build import LIB
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(drop.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def drop_(lib, **kw):
    a = dict(x=at(0), y=at(1), n=100, p=0.1, rng=None, seed=1, offset=2, dtype=0)
    a.update(kw)
    return lib.dropout_fwd(*a.values(), None)


def fwd(lib, **kw):
    a = dict(f=at(0), x=at(1), bias=at(2), p=0.1, rng=None, seed=1, offset=2, norm=2, gamma=at(3), beta=at(4), h=at(5),
             y=at(6), mean=at(7), rstd=at(8), rows=4, H=8, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.dropout_add_norm_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(dy=at(0), dh=at(1), h=at(2), p=0.1, rng=None, seed=1, offset=2, norm=2, gamma=at(3), mean=at(4), rstd=at(5),
             df=at(6), dx=at(7), dbias=at(8), dgamma=at(9), dbeta=at(10), rows=4, H=8, dtype=0, ws=at(12), wb=1 << 20)
    a.update(kw)
    return lib.dropout_add_norm_bwd(*a.values(), None)


def test_dropout_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    for kw, code in [
            (dict(dtype=3), b.ERR_DTYPE), (dict(n=-1), b.ERR_SHAPE), (dict(n=1 << 62), b.ERR_SHAPE),
            (dict(p=-0.1), k.ERR_SCALE), (dict(p=1.5), k.ERR_SCALE), (dict(p=float("nan")), k.ERR_SCALE),
            (dict(rng=at(3) + 4), k.ERR_ALIGN), (dict(x=None), b.ERR_NULL), (dict(y=None), b.ERR_NULL),
            (dict(x=at(0) + 2), k.ERR_ALIGN), (dict(dtype=1, y=at(1) + 1), k.ERR_ALIGN), (dict(y=at(0) + 4), b.ERR_ALIAS),
            (dict(rng=at(1) + 16), b.ERR_ALIAS), (dict(n=0, x=None, y=None), b.OK), (dict(n=0, p=2.0), k.ERR_SCALE)]:
        assert drop_(lib, **kw) == code, kw


def test_forward_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    for kw, code in [
            (dict(dtype=3), b.ERR_DTYPE), (dict(rows=-1), b.ERR_SHAPE), (dict(H=0), b.ERR_SHAPE),
            (dict(H=16385), b.ERR_SHAPE), (dict(H=32769, dtype=2), b.ERR_SHAPE), (dict(rows=1 << 61), b.ERR_SHAPE),
            (dict(norm=3), k.ERR_KIND), (dict(norm=0), k.ERR_KIND), (dict(p=1.01), k.ERR_SCALE),
            (dict(eps=-1.0), b.ERR_EPS), (dict(eps=float("inf")), b.ERR_EPS), (dict(f=None), b.ERR_NULL),
            (dict(y=None), b.ERR_NULL), (dict(gamma=None), b.ERR_NULL),
            (dict(norm=0, y=None, gamma=None, beta=None, mean=None, rstd=None, h=None), b.ERR_NULL),
            (dict(rng=at(9) + 1), k.ERR_ALIGN), (dict(f=at(0) + 1), k.ERR_ALIGN), (dict(bias=at(2) + 2), k.ERR_ALIGN),
            (dict(mean=at(7) + 2), k.ERR_ALIGN), (dict(h=at(0) + 16), b.ERR_ALIAS), (dict(y=at(5)), b.ERR_ALIAS),
            (dict(h=at(2)), b.ERR_ALIAS), (dict(rstd=at(7)), b.ERR_ALIAS), (dict(y=at(1) + 32), b.ERR_ALIAS),
            (dict(rng=at(5)), b.ERR_ALIAS), (dict(rows=0, f=None, y=None), b.OK), (dict(rows=0, dtype=9), b.ERR_DTYPE)]:
        assert fwd(lib, **kw) == code, kw


def test_backward_refusals(lib):
    from memory_bound_add_gb300 import binding as b, block as k
    none = dict(norm=0, dy=None, gamma=None, mean=None, rstd=None, dgamma=None, dbeta=None)
    for kw, code in [
            (dict(dtype=-1), b.ERR_DTYPE), (dict(rows=-2), b.ERR_SHAPE), (dict(H=0), b.ERR_SHAPE),
            (dict(norm=7), k.ERR_KIND), (dict(norm=0), k.ERR_KIND), (dict(none, dgamma=at(9)), k.ERR_KIND),
            (dict(p=-1e-9), k.ERR_SCALE), (dict(wb=-1), b.ERR_WORKSPACE), (dict(dy=None, dh=None), b.ERR_NULL),
            (dict(none, dh=None), b.ERR_NULL), (dict(df=None), b.ERR_NULL), (dict(h=None), b.ERR_NULL),
            (dict(gamma=None), b.ERR_NULL), (dict(rstd=None), b.ERR_NULL), (dict(mean=None), b.ERR_NULL),
            (dict(dbias=at(8) + 1), k.ERR_ALIGN), (dict(dtype=2, dy=at(0) + 1), k.ERR_ALIGN), (dict(df=at(7)), b.ERR_ALIAS),
            (dict(df=at(0) + 16), b.ERR_ALIAS), (dict(dgamma=at(3)), b.ERR_ALIAS), (dict(dbias=at(9)), b.ERR_ALIAS),
            (dict(ws=at(6)), b.ERR_ALIAS), (dict(ws=at(2)), b.ERR_ALIAS), (dict(rng=at(6)), b.ERR_ALIAS)]:
        assert bwd(lib, **kw) == code, kw


def test_workspace_size_refusals(lib):
    from memory_bound_add_gb300 import binding as b
    size = lib.dropout_add_norm_bwd_workspace_size
    assert size(0, 64, 0) == 0
    assert size(-1, 64, 0) == b.ERR_SHAPE
    assert size(4, 0, 0) == b.ERR_SHAPE
    assert size(4, 64, 5) == b.ERR_DTYPE


def test_rng_arguments():
    from memory_bound_add_gb300.drop import _rng_args
    assert _rng_args((3, 4), 0) == (None, 3, 4)
    assert _rng_args((np.int64(-1), (1 << 64) - 1), 0) == (None, -1, (1 << 64) - 1)
    for bad in (5, (1.0, 2), None, "ab"):
        with pytest.raises(TypeError):
            _rng_args(bad, 0)
    for bad in ((1, 1 << 64), (-(1 << 63) - 1, 0), (1,), (1, 2, 3), torch.zeros(2), torch.zeros(3, dtype=torch.int64),
                torch.zeros(2, dtype=torch.int64)):
        with pytest.raises(ValueError):
            _rng_args(bad, 0)


def test_generator_known_answers():
    # the generator's published known answers
    z, f = [[0]] * 4, [[0xFFFFFFFF]] * 4
    pi = [[0x243F6A88], [0x85A308D3], [0x13198A2E], [0x03707344]]
    for counter, key, want in [
            (z, (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            (f, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            (pi, (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(v[0]) for v in philox(counter, key)) == want


def test_plain_mask():
    # a part of a mask is that part of the whole; the share kept is that of p
    whole = keep(1000, 0.3, (7, 8))
    for a, n in ((0, 5), (3, 700), (997, 3), (8, 16)):
        assert torch.equal(keep(n, 0.3, (7, 8), a), whole[a:a + n])
    k = keep(1 << 20, 0.3, (1, 2)).double().mean()
    # five standard deviations of a binomial share
    assert abs(float(k) - (1 - threshold(0.3) / 65536)) < 5 * (0.21 / (1 << 20)) ** 0.5
    assert threshold(0.0) == 0 and threshold(1.0) == 65536 and scale(1.0) == 0.0 and scale(0.5) == 2.0
