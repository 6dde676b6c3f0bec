"""Plain 64-bit forms of the dropout operators, and their error bounds.

The mask is made here from the published generator (Philox 4x32-10) in numpy.
The boundary's own values and bounds are those of _block_ref with f replaced by
d = dropout(f + bias): d is off by the sum's, the scale's and the product's
rounding, 3 u |d| with u = 2^-24, which the 32 u (|x| + |d|) that _block_ref
grants h contain beside the last sum's u |h| and, for y, the statistics.
"""
from __future__ import annotations

import numpy as np
import torch

from _block_ref import CSUM, U, backward, forward

LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """counter: four uint64 arrays of 32-bit words; key: two numbers."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) & 0xFFFFFFFF for v in key]
    sh = np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & LOW, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return round(p * 65536)  # ties to even


def keep(n, p, rng, start=0):
    """Whether elements start .. start + n - 1 are kept (bool tensor)."""
    seed, offset = (int(v) & (2 ** 64 - 1) for v in rng)
    b = np.arange(start // 8, (start + n + 7) // 8, dtype=np.uint64)
    full = lambda v: np.full_like(b, v)  # noqa: E731
    w = philox([b & LOW, b >> np.uint64(32), full(offset & 0xFFFFFFFF), full(offset >> 32)],
               (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1).reshape(-1)
    return torch.from_numpy(halves[start % 8:start % 8 + n] >= threshold(p))


def scale(p):
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def dropped(v, p, rng, start=0):
    """dropout(v) in 64 bits."""
    k = keep(v.numel(), p, rng, start).view(v.shape)
    return torch.where(k, v.double() * scale(p), torch.zeros((), dtype=torch.float64))


def drop_forward(f, x, bias, p, rng, norm, gamma, beta, eps, start=0):
    """h, y, (mean, rstd) and the errors of h and y before the last rounding."""
    z = f.double() if bias is None else f.double() + bias.double()
    d = dropped(z, p, rng, start)
    h, y, st, eh, ey = forward(d, torch.zeros_like(d) if x is None else x, {"pre_gamma": gamma, "pre_beta": beta}, None,
                               norm, 1.0, 1.0, eps)
    return h, y, st[2:], eh, ey


def drop_backward(dy, dh, h, stats, p, rng, norm, gamma):
    """Gradients and, for each, the error before the last rounding."""
    g, e = backward(dy, dh, None, h, (None, None, *stats), {"pre_gamma": gamma}, None, norm, 1.0, 1.0)
    D, eD = g["dx"], e["dx"]
    k = keep(D.numel(), p, rng).view(D.shape) * scale(p)
    df, edf = k * D, k * (eD + 3 * U * D.abs())
    lead = tuple(range(D.dim() - 1))
    want = {"df": df, "dx": D, "dbias": df.sum(lead), "dgamma": g["dpre_gamma"], "dbeta": g["dpre_beta"]}
    err = {"df": edf, "dx": eD, "dbias": edf.sum(lead) + CSUM * df.abs().sum(lead), "dgamma": e["dpre_gamma"],
           "dbeta": e["dpre_beta"]}
    return want, err
