"""Plain 64-bit forms of the block boundary and their error bounds.

u is half a step of fp32, 2^-24.  A kernel computes each row in fp32 from
exact inputs, so its error before the last rounding is some u times the
magnitudes of what is added up:

  statistics   a row's sum runs over at most 8 values in a thread, 5 levels
               in a warp and 8 levels over the warps of a cluster (128 of
               them): with the products' own roundings below 24 u of the sum
               of magnitudes; rstd takes half of that, and rsqrtf 2 units in
               the last place (4 u) more: 16 u
  fhat         the shift, the mean and rstd: 20 u |fhat|, and, the mean being
               off by at most 4 u of the row's largest deviation, 4 u R with
               R = max |fhat|
  n, gate, h   one rounding each, of the terms' magnitudes

All of it together is below 32 u of the magnitudes below, C = 32 u.  The
output's own rounding adds half a step of its type, or half the least
subnormal.  Column sums: at most 8 rows a walker are added in these tests, then
at most 64 partials in a thread's chain and butterfly: below 96 u of the sum
of magnitudes, beside the terms' own errors.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
C = 32 * U
CSUM = 96 * U
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rounding(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def stats_of(v, kind, eps):
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + eps)
    return mean, rstd


def expand_gate(gate, like):
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    return gate.double()


def forward(f, x, p, post, pre, a, s, eps):
    """h, y, stats and the errors of h and y before the last rounding."""
    f, x = f.double(), x.double()
    one, zero = torch.ones((), dtype=torch.float64), torch.zeros((), dtype=torch.float64)
    get = lambda k, d: p[k].double() if p.get(k) is not None else d  # noqa: E731
    pg, pb, ng, nb = get("post_gamma", one), get("post_beta", zero), get("pre_gamma", one), get("pre_beta", zero)
    gate = expand_gate(p.get("gate"), f)
    st = [None] * 4
    n, mag = f, f.abs()
    if post is not None:
        mean, rstd = stats_of(f, post, eps)
        hat = (f - mean) * rstd
        R = hat.abs().amax(-1, keepdim=True)
        n = hat * pg + pb
        mag = (hat.abs() + R) * pg.abs() + pb.abs()
        st[0], st[1] = (mean if post == "layer" else None), rstd
    h = a * x + s * gate * n
    eh = C * ((a * x).abs() + (s * gate).abs() * mag)
    y = ey = None
    if pre is not None:
        mean, rstd = stats_of(h, pre, eps)
        hat = (h - mean) * rstd
        R = hat.abs().amax(-1, keepdim=True)
        y = hat * ng + nb
        # eh moves h, its mean and its scale
        moved = rstd * (eh + (1 + hat.abs()) * eh.pow(2).mean(-1, keepdim=True).sqrt())
        ey = ng.abs() * moved + C * ((hat.abs() + R) * ng.abs() + nb.abs())
        st[2], st[3] = (mean if pre == "layer" else None), rstd
    return h, y, st, eh, ey


def backward(dy, dh, f, h, st, p, post, pre, a, s, rpg_shape=None):
    """Gradients and, for each, the error before the last rounding."""
    one, zero = torch.ones((), dtype=torch.float64), torch.zeros((), dtype=torch.float64)
    get = lambda k, d: p[k].double() if p.get(k) is not None else d  # noqa: E731
    pg, pb, ng = get("post_gamma", one), get("post_beta", zero), get("pre_gamma", one)
    gate = expand_gate(p.get("gate"), f)
    some = dy if dy is not None else dh
    lead = tuple(range(some.dim() - 1))
    full = torch.zeros(some.shape, dtype=torch.float64)
    col = [None if t is None else t.double().view(*some.shape[:-1], 1) for t in st]
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    D = full if dh is None else dh.double()
    eD = U * D.abs()
    g, e = {}, {}
    if dy is not None:
        dy = dy.double()
        hhat = (h.double() - (col[2] if pre == "layer" else 0)) * col[3]
        w = dy * ng
        t = w - hhat * mean(w * hhat)
        mag = w.abs() + hhat.abs() * mean((w * hhat).abs())
        if pre == "layer":
            t = t - mean(w)
            mag = mag + mean(w.abs())
        D = D + col[3] * t
        eD = eD + C * col[3] * mag
        g["dpre_gamma"], e["dpre_gamma"] = (dy * hhat).sum(lead), CSUM * (dy * hhat).abs().sum(lead)
        g["dpre_beta"], e["dpre_beta"] = dy.sum(lead), CSUM * dy.abs().sum(lead)
    else:
        z = torch.zeros(some.shape[-1], dtype=torch.float64)
        g.update(dpre_gamma=z, dpre_beta=z)
        e.update(dpre_gamma=z, dpre_beta=z)
    g["dx"], e["dx"] = a * D, abs(a) * (eD + U * D.abs())
    fd = full if f is None else f.double()
    fhat = (fd - (col[0] if post == "layer" else 0)) * col[1] if post is not None else fd
    n = fhat * pg + pb
    nmag = fhat.abs() * pg.abs() + pb.abs()
    sD, esD = s * D, abs(s) * (eD + 2 * U * D.abs())
    gt = p.get("gate")
    if gt is not None:
        d, ed = sD * n, esD * nmag + 4 * U * sD.abs() * nmag
        if gt.dim() == 1:
            g["dgate"] = d.sum(lead)
            # by way of sum s D fhat and sum s D
            e["dgate"] = ed.sum(lead) + CSUM * (sD.abs() * nmag).sum(lead)
        else:
            dims = tuple(i for i in range(d.dim() - 1) if gt.shape[i] == 1 and d.shape[i] != 1)
            if dims:
                g["dgate"] = d.sum(dims, keepdim=True)
                e["dgate"] = ed.sum(dims, keepdim=True) + CSUM * (sD.abs() * nmag).sum(dims, keepdim=True)
            else:
                g["dgate"], e["dgate"] = d, ed
    dn, edn = sD * gate, (esD + U * sD.abs()) * gate.abs()
    if post is not None:
        g["dpost_gamma"] = (dn * fhat).sum(lead)
        e["dpost_gamma"] = (edn * fhat.abs()).sum(lead) + CSUM * (dn * fhat).abs().sum(lead)
        g["dpost_beta"], e["dpost_beta"] = dn.sum(lead), edn.sum(lead) + CSUM * dn.abs().sum(lead)
        v, ev = dn * pg, edn * pg.abs()
        t = v - fhat * mean(v * fhat)
        mag = v.abs() + fhat.abs() * mean((v * fhat).abs())
        et = ev + fhat.abs() * mean(ev * fhat.abs())
        if post == "layer":
            t = t - mean(v)
            mag = mag + mean(v.abs())
            et = et + mean(ev)
        g["df"], e["df"] = col[1] * t, col[1] * (et + C * mag)
    else:
        g["df"], e["df"] = dn, edn
    return g, e


def assert_within(got, want, err, what):
    """|got - want| <= err + the output's own rounding, element by element."""
    bound = err + rounding(want.abs() + err, got.dtype)
    d = (got.detach().cpu().double().reshape(want.shape) - want).abs()
    bad = ~(d <= bound)
    if bad.any():
        i = int((d - bound).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound; worst at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, want {want.reshape(-1)[i].item()!r}, bound "
                             f"{bound.expand_as(want).reshape(-1)[i].item():.3g}")
