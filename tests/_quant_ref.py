"""Plain 64-bit forms of the 8-bit operators, and how far a kernel may be off.

y and its error ey before any rounding are _block_ref's.  With u = 2^-24 a scale
is off by ey of the largest value over the format's largest, and by the
quotient's roundings, 3 u.  So y / scale is off by (ey / scale) and by 8 u of
itself; q may be the rounding of any number that near, and what it stands for is
then off from y by half a step of the format at that number (of the step above
it, where it lies at a power of two), or, cut, by what the cut takes away.
Scales that are powers of two may be the next one where the largest value is
within its error of a border.
"""
from __future__ import annotations

import torch

from _block_ref import U, forward

TOP = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
_BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}
LEAST = 2.0 ** -126


def step(v, fmt):
    """The format's step at |v| (64 bits)."""
    if fmt == "int8":
        return torch.ones_like(v)
    bits, least = _BITS[fmt]
    e = torch.frexp(v.abs())[1].double() - 1
    return torch.exp2(e.clamp(min=least) - bits)


def to_grid(v, fmt):
    """v rounded to the format, ties to even, and cut."""
    if fmt == "int8":
        return v.round().clamp(-127, 127)
    s = step(v, fmt)
    return (torch.round(v / s) * s).clamp(-TOP[fmt], TOP[fmt])


def groups(v, group):
    """[rows, G, group] of [rows, H], zeros behind the end."""
    rows, H = v.shape
    G = -(-H // group)
    out = torch.zeros(rows, G * group, dtype=v.dtype)
    out[:, :H] = v
    return out.view(rows, G, group)


def pow2_of(t):
    """The least power of two that is at least t."""
    m, e = torch.frexp(t)
    return torch.where(t > 0, torch.exp2((e - (m == 0.5).int()).double()), 0.0)


def norm_quant(x, residual, norm, gamma, beta, eps):
    """h, y, (mean, rstd) and the errors of h and y before a rounding."""
    x = x.reshape(-1, x.shape[-1])
    zero = torch.zeros_like(x, dtype=torch.float64)
    r = zero if residual is None else residual.reshape(x.shape)
    h, y, st, eh, ey = forward(r, x, {"pre_gamma": gamma, "pre_beta": beta}, None, norm, 1.0, 1.0, eps)
    if norm is None:
        return h, h, (None, None), eh, eh
    return h, y, st[2:], eh, ey


def check(q, scale, y, ey, fmt, scaling, group, what, given=None):
    """q and scale ([rows, H] and [rows, G], on the host) against y."""
    rows, H = y.shape
    top = TOP[fmt]
    g = group or H
    sc = scale.double() if scaling != "tensor" else torch.full((rows, 1), float(given), dtype=torch.float64)
    if scaling != "tensor":
        amax = groups(y.abs(), g).amax(-1)
        # the largest value's own error, or that of one that passes it
        off = (groups(y.abs() + ey, g).amax(-1) - amax).clamp(min=0) + groups(ey, g).amax(-1)
        want = (amax / top).clamp(min=LEAST)
        if scaling == "pow2":
            lo, hi = pow2_of((amax - off).clamp(min=0) / top).clamp(min=LEAST), pow2_of((amax + off) / top).clamp(min=LEAST)
            assert ((sc >= lo) & (sc <= hi)).all(), f"{what}: scales beyond the next power of two"
            assert (torch.frexp(sc)[0] == 0.5).all(), f"{what}: scales that are no powers of two"
        else:
            bad = (sc - want).abs() > off / top + 3 * U * want
            assert not bad.any(), f"{what}: {int(bad.sum())} scales off, by up to {float(((sc - want) / want).abs().max()):.3g}"
    s = sc.repeat_interleave(g, 1)[:, :H]
    v = y / s
    slack = ey / s + 8 * U * v.abs()
    got = q.double()
    assert (got.abs() <= top).all()
    assert torch.equal(to_grid(got, fmt), got)
    cut = (v.abs() - top).clamp(min=0)  # a given scale may cut
    bound = step((v.abs() + slack).clamp(max=top), fmt) / 2 + slack + cut
    bad = (got - v).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off by more than half a step"
    # all but the ones near a border are the rounding itself
    sure = to_grid(v - slack, fmt) == to_grid(v + slack, fmt)
    assert torch.equal(got[sure], to_grid(v, fmt)[sure]), what
    return s
