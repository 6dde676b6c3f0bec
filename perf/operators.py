"""What is measured of the block-boundary and gradient operators.

Three operators:

``fwd``   the boundary between two blocks, forward: the block's output f is
          normalised (post norm), gated, scaled and added to the residual
          stream x, and the new stream h is normalised for the next block:
              n = post(f);  h = a x + s (gate . n);  y = pre(h)
``bwd``   its gradients: df, dx and the gradients of both norms' parameters
          and of the gate
``clip``  the norm over all of a model's gradients, and the gradients scaled
          so that their norm is at most max_norm

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits (64 for the long sum of the gradient norm), rounded once at the end;
with ``own`` true it makes the calls of ``memory_bound_add_gb300``.
"""
import itertools
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases
def _block(name, op, rows, H, dtype, post, pre, gate="none", rpg=0, beta=False, a=1.0, s=1.0,
           eps=1e-5, train=False):
    """post, pre: "rms", "layer" or "none"; gate: "none", "channel" (fp32 [H])
    or "rows" (one row of dtype for every rpg rows); beta: the norms have
    biases; train: the forward also returns what the backward needs."""
    return {"name": name, "op": op, "rows": rows, "H": H, "dtype": dtype, "post": post,
            "pre": pre, "gate": gate, "rpg": rpg, "beta": beta, "a": a, "s": s, "eps": eps,
            "train": train}


def _clip(name, hidden, ffn, layers, vocab, dtype, out, max_norm, scale):
    """Gradients of a decoder of `layers` blocks. out: "fp32" or "same" (a
    buffer of fp32 or of the gradients' dtype beside them), "inplace" (the
    gradients themselves; max_norm is above the norm, so they stay)."""
    return {"name": name, "op": "clip", "hidden": hidden, "ffn": ffn, "layers": layers,
            "vocab": vocab, "dtype": dtype, "out": out, "max_norm": max_norm, "scale": scale}


def listed():
    return [
        # one token of a served model: latency
        _block("fwd_token_1x4096_bf16", "fwd", 1, 4096, "bf16", "rms", "rms"),
        # BERT-base rows in training: layer norms on both sides, a learnt gate
        # per channel, statistics kept for the backward
        _block("fwd_bert_4096x768_fp16", "fwd", 4096, 768, "fp16", "layer", "layer", "channel",
               beta=True, eps=1e-12, train=True),
        # one prompt of 2048 tokens, the block's output scaled before the sum
        _block("fwd_pages_2048x4096_fp16", "fwd", 2048, 4096, "fp16", "rms", "rms", s=0.5),
        # odd rows and width (rows start misaligned), a gate of its own for every row
        _block("fwd_ragged_4097x1001_bf16", "fwd", 4097, 1001, "bf16", "none", "layer", "rows",
               rpg=1, beta=True, a=0.9),
        # the largest activations: 8 sequences of 4096, a gate for each sequence
        _block("fwd_large_32768x8192_bf16", "fwd", 32768, 8192, "bf16", "rms", "rms", "rows",
               rpg=4096, train=True),
        # the smallest training step
        _block("bwd_tiny_64x768_fp32", "bwd", 64, 768, "fp32", "none", "layer", "none", beta=True),
        _block("bwd_bert_4096x768_fp16", "bwd", 4096, 768, "fp16", "layer", "layer", "channel",
               beta=True, eps=1e-12),
        _block("bwd_pages_2048x4096_fp16", "bwd", 2048, 4096, "fp16", "rms", "rms", "rows", rpg=1,
               s=0.5),
        _block("bwd_large_32768x8192_bf16", "bwd", 32768, 8192, "bf16", "rms", "rms", "rows",
               rpg=4096),
        # one block's gradients, fp32, mostly below the limit: nothing to scale
        _clip("clip_block_fp32_inplace", 768, 2048, 1, 0, "fp32", "inplace", 1e4, 1.0),
        # a model of about 130 million parameters, loss-scaled fp16 gradients
        # unscaled and clipped into fp32 (its width is odd, so most gradients
        # begin at odd addresses of the buffer)
        _clip("clip_model_fp16_to_fp32", 1001, 2730, 8, 32000, "fp16", "fp32", 1.0, 1.0 / 1024),
        # about 1.7 billion parameters in bf16
        _clip("clip_large_bf16", 4096, 11008, 8, 32000, "bf16", "same", 1.0, 1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "clip"])
    dtype = rng.choice(["fp32", "fp16", "bf16", "bf16"])
    if op == "clip":
        hidden = _log_int(rng, 64, 4096)
        out = rng.choice(["fp32", "same", "inplace"])
        c = _clip("", hidden, hidden * rng.randint(2, 4) + rng.randint(0, 9),
                  _log_int(rng, 1, 8), rng.choice([0, _log_int(rng, 100, 32000)]), dtype, out,
                  1e4 if out == "inplace" else rng.choice([0.5, 1.0]),
                  1.0 / 1024 if dtype == "fp16" and out != "inplace" else 1.0)
        del c["name"]
        return c
    H = _log_int(rng, 32, 8192)
    if rng.random() < 0.75:
        H = max(8, H // 8 * 8)
    rows = _log_int(rng, 1, 8192)
    gate = rng.choice(["none", "channel", "rows"])
    rpg = 0
    if gate == "rows":
        rpg = rng.choice([1, _log_int(rng, 1, rows)])
        rows = max(1, rows // rpg) * rpg
    post = rng.choice(["rms", "layer", "none"])
    pre = rng.choice(["rms", "layer"])
    c = _block("", op, rows, H, dtype, post, pre, gate, rpg, beta="layer" in (post, pre),
               a=rng.choice([1.0, 0.9]), s=rng.choice([1.0, 0.5]), train=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """The parameters of a decoder: embedding, then in every block the four
    attention projections, three of the feed-forward layer and two norms, then
    the last norm."""
    d, f = case["hidden"], case["ffn"]
    block = [d * d] * 4 + [d * f] * 3 + [d] * 2
    return ([case["vocab"] * d] if case["vocab"] else []) + block * case["layers"] + [d]


def _offsets(sizes):
    at = [0, *itertools.accumulate(sizes)]
    return at[:-1], at[-1]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = {"case": case}

    def normal(shape, scale=1.0, loc=0.0, dtype=torch.float32):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for part in out.view(-1).split(1 << 26):
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(scale).add_(loc))
        return out

    if case["op"] == "clip":
        sizes = _sizes(case)
        at, total = _offsets(sizes)
        # gradients lie one after another in one buffer, as a training program
        # keeps them; their sizes of value differ from tensor to tensor
        flat = torch.empty(total, dtype=dt, device="cuda")
        std = torch.rand(len(sizes), generator=g, device="cuda").mul_(4.0).sub_(2.0).exp_()
        std = std * (3.0 / math.sqrt(total)) / case["scale"]
        std = std.tolist()
        for o, n, k in zip(at, sizes, range(len(sizes))):
            for i in range(0, n, 1 << 26):
                m = min(1 << 26, n - i)
                flat[o + i:o + i + m] = torch.randn(m, generator=g, device="cuda").mul_(std[k])
        s["flat"] = flat
        s["grads"] = [flat[o:o + n] for o, n in zip(at, sizes)]
        if case["out"] == "inplace":
            s["out"], s["out_flat"] = None, flat
        else:
            s["out_flat"] = torch.empty(total, dtype=torch.float32 if case["out"] == "fp32" else dt,
                                        device="cuda")
            s["out"] = [s["out_flat"][o:o + n] for o, n in zip(at, sizes)]
        return s
    rows, H = case["rows"], case["H"]
    s["f"] = normal((rows, H), 0.7, 0.1, dt)
    s["x"] = normal((rows, H), 1.5, 0.0, dt)
    par = {}
    for side in ("post", "pre"):
        if case[side] != "none":
            par[side + "_gamma"] = normal((H,), 0.1, 1.0)
            if case["beta"] and case[side] == "layer":
                par[side + "_beta"] = normal((H,), 0.1)
    if case["gate"] == "channel":
        par["gate"] = normal((H,), 0.2, 0.5)
    elif case["gate"] == "rows":
        G = rows // case["rpg"]
        par["gate"] = normal((G, 1, H) if case["rpg"] > 1 else (G, H), 0.5, 0.2, dt)
        if case["rpg"] > 1:
            s["f"], s["x"] = s["f"].view(G, case["rpg"], H), s["x"].view(G, case["rpg"], H)
    s["par"] = par
    if case["op"] == "bwd":
        shape = s["f"].shape
        s["dy"] = normal(shape, 1.0, 0.0, dt)
        s["dh"] = normal(shape, 0.5, 0.0, dt)
        # what the forward left: the rounded stream and the statistics
        h = torch.empty_like(s["x"])
        st = [torch.empty(rows, device="cuda") for _ in range(4)]
        f2, x2, h2 = s["f"].view(rows, H), s["x"].view(rows, H), h.view(rows, H)
        step = max(1, (1 << 26) // H)
        for i in range(0, rows, step):
            e = min(rows, i + step)
            hh, _, stats = _plain_fwd(case, f2[i:e], x2[i:e], _rows_of(case, par, i, e), stats=True)
            h2[i:e] = hh
            for t, v in zip(st, stats):
                if v is not None:
                    t[i:e] = v
        s["h"] = h
        s["stats"] = tuple(t if v is not None else None for t, v in zip(st, stats))
        del s["x"]
    return s


def _rows_of(case, par, i, e):
    """The parameters as rows i..e of the flattened batch see them."""
    if case["gate"] != "rows":
        return par
    G = par["gate"].reshape(-1, case["H"])
    idx = torch.arange(i, e, device="cuda") // case["rpg"]
    return {**par, "gate": G[idx]}


# -------------------------------------------------------------- plain forms
def _norm(v, kind, gamma, beta, eps):
    """(normalised, hat, mean or None, rstd) over the last dimension."""
    mean = None
    if kind == "layer":
        mean = v.mean(-1, keepdim=True)
        v = v - mean
    rstd = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    hat = v * rstd
    out = hat * gamma
    if beta is not None:
        out = out + beta
    return out, hat, mean, rstd


def _plain_fwd(case, f, x, par, stats=False):
    """h, y and (post mean, post rstd, pre mean, pre rstd), all in 32 bits."""
    n, pm, pr = f.float(), None, None
    if case["post"] != "none":
        n, _, pm, pr = _norm(n, case["post"], par["post_gamma"], par.get("post_beta"), case["eps"])
    if case["gate"] != "none":
        n = n * par["gate"].float()
    h = case["a"] * x.float() + case["s"] * n
    y, hm, hr = None, None, None
    if case["pre"] != "none":
        y, _, hm, hr = _norm(h, case["pre"], par["pre_gamma"], par.get("pre_beta"), case["eps"])
    st = tuple(None if v is None else v.reshape(-1) for v in (pm, pr, hm, hr)) if stats else None
    return h, y, st


def _plain_bwd(case, s):
    f, h, dy, dh, par = s["f"].float(), s["h"].float(), s["dy"].float(), s["dh"].float(), s["par"]
    pm, pr, hm, hr = [None if v is None else v.view(*f.shape[:-1], 1) for v in s["stats"]]
    lead = tuple(range(f.dim() - 1))
    out = {}
    hhat = (h - hm if hm is not None else h) * hr
    u = dy * par["pre_gamma"]
    t = u - hhat * (u * hhat).mean(-1, keepdim=True)
    if hm is not None:
        t = t - u.mean(-1, keepdim=True)
    D = hr * t + dh
    out["dpre_gamma"] = (dy * hhat).sum(lead)
    if "pre_beta" in par:
        out["dpre_beta"] = dy.sum(lead)
    out["dx"] = case["a"] * D
    sD = case["s"] * D
    if case["post"] != "none":
        fhat = (f - pm if pm is not None else f) * pr
        n = fhat * par["post_gamma"]
        if "post_beta" in par:
            n = n + par["post_beta"]
    else:
        n = f
    dn = sD
    if case["gate"] != "none":
        dn = sD * par["gate"].float()
        dg = sD * n
        if case["gate"] == "channel":
            dg = dg.sum(lead)
        elif case["rpg"] > 1:
            dg = dg.sum(1, keepdim=True)
        out["dgate"] = dg
    if case["post"] != "none":
        out["dpost_gamma"] = (dn * fhat).sum(lead)
        if "post_beta" in par:
            out["dpost_beta"] = dn.sum(lead)
        v = dn * par["post_gamma"]
        t = v - fhat * (v * fhat).mean(-1, keepdim=True)
        if pm is not None:
            t = t - v.mean(-1, keepdim=True)
        out["df"] = pr * t
    else:
        out["df"] = dn
    dt = DTYPES[case["dtype"]]
    half = {"df", "dx"} | ({"dgate"} if case["gate"] == "rows" else set())
    return {k: v.to(dt) if k in half else v for k, v in out.items()}


def _plain_clip(case, s):
    c = case["scale"]
    sq = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = (sq.sqrt() * c).float()
    coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0) * c
    if s["out"] is None:
        # rounded to the buffer's own type, as a scaling in place is
        done = [g.copy_(g.float() * coef) for g in s["grads"]]
    else:
        done = [o.copy_(g.float() * coef) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm, "grads": s["out_flat"]} if done else None


# --------------------------------------------------------------------- run
def run(state):
    s = state
    case = s["case"]
    if own:
        import memory_bound_add_gb300 as mba
        if case["op"] == "clip":
            norm = mba.clip_grads(s["grads"], case["max_norm"], out=s["out"], scale=case["scale"])
            return {"norm": norm, "grads": s["out_flat"]}
        kw = dict(post=None if case["post"] == "none" else case["post"],
                  pre=None if case["pre"] == "none" else case["pre"],
                  residual_scale=case["a"], block_scale=case["s"], **s["par"])
        if case["op"] == "fwd":
            h, y, stats = mba.block_norm(s["f"], s["x"], eps=case["eps"],
                                          want_stats=case["train"], **kw)
            return _fwd_out(case, h, y, stats)
        g = mba.block_norm_backward(s["dy"], s["dh"], s["f"], s["h"], s["stats"], **kw)
        return {k: v for k, v in g._asdict().items() if v is not None}
    if case["op"] == "clip":
        return _plain_clip(case, s)
    if case["op"] == "bwd":
        return _plain_bwd(case, s)
    dt = DTYPES[case["dtype"]]
    h, y, stats = _plain_fwd(case, s["f"], s["x"], s["par"], stats=case["train"])
    return _fwd_out(case, h.to(dt), y.to(dt), stats)


def _fwd_out(case, h, y, stats):
    out = {"h": h, "y": y}
    if case["train"]:
        out.update({k: v for k, v in zip(("post_mean", "post_rstd", "pre_mean", "pre_rstd"), stats)
                    if v is not None})
    return out


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The same values from the definitions, in 64 bits, chunk by chunk."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        c = float(case["scale"])
        sq = 0.0
        for g in s["grads"]:
            for part in g.split(1 << 26):
                sq += float((part.double() ** 2).sum())
        norm = math.sqrt(sq) * c
        k = c * min(1.0, case["max_norm"] / (norm + 1e-6))
        # in 32 bits where the whole in 64 would not leave room for the rest
        big = s["flat"].numel() > 1 << 29
        res = torch.empty(s["flat"].numel(), dtype=torch.float32 if big else torch.float64, device="cuda")
        for i in range(0, res.numel(), 1 << 26):
            res[i:i + (1 << 26)] = s["flat"][i:i + (1 << 26)].double() * k
        return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": res}
    rows, H = case["rows"], case["H"]
    par = {k: v.double().reshape(-1, H) for k, v in s["par"].items()}
    step = max(1, (1 << 25) // H)
    a, b, eps = float(case["a"]), float(case["s"]), float(case["eps"])
    gate = par.get("gate")

    def gates(i, e):
        if gate is None:
            return torch.ones(1, H, dtype=torch.float64, device="cuda")
        if case["gate"] == "channel":
            return gate
        return gate[torch.arange(i, e, device="cuda") // case["rpg"]]

    one = torch.ones(1, H, dtype=torch.float64, device="cuda")
    pg, pb = par.get("post_gamma", one), par.get("post_beta", one * 0)
    ng, nb = par.get("pre_gamma", one), par.get("pre_beta", one * 0)
    big = rows * H > 1 << 27
    wide = dict(dtype=torch.float32 if big else torch.float64, device="cuda")
    if case["op"] == "fwd":
        h, y = torch.empty(rows, H, **wide), torch.empty(rows, H, **wide)
        st = torch.zeros(4, rows, dtype=torch.float64, device="cuda")
        for i in range(0, rows, step):
            e = min(rows, i + step)
            n = s["f"].view(rows, H)[i:e].double()
            if case["post"] != "none":
                if case["post"] == "layer":
                    st[0, i:e] = n.mean(1)
                n = n - st[0, i:e, None]
                st[1, i:e] = (n.pow(2).mean(1) + eps).rsqrt()
                n = n * st[1, i:e, None] * pg + pb
            v = a * s["x"].view(rows, H)[i:e].double() + b * gates(i, e) * n
            h[i:e] = v
            if case["pre"] == "layer":
                st[2, i:e] = v.mean(1)
            v = v - st[2, i:e, None]
            st[3, i:e] = (v.pow(2).mean(1) + eps).rsqrt()
            y[i:e] = v * st[3, i:e, None] * ng + nb
        out = {"h": h.view(s["f"].shape), "y": y.view(s["f"].shape)}
        if case["train"]:
            keep = {"post_mean": case["post"] == "layer", "post_rstd": case["post"] != "none",
                    "pre_mean": case["pre"] == "layer", "pre_rstd": True}
            out.update({k: st[j] for j, (k, w) in enumerate(keep.items()) if w})
        return out
    dx, df = torch.empty(rows, H, **wide), torch.empty(rows, H, **wide)
    z = lambda n=1: torch.zeros(n, H, dtype=torch.float64, device="cuda")  # noqa: E731
    dng, dnb, dpg, dpb, dgc = z(), z(), z(), z(), z()
    dgr = z(rows // case["rpg"]) if case["gate"] == "rows" else None
    S = [torch.zeros(rows, dtype=torch.float64, device="cuda") if v is None else v.double() for v in s["stats"]]
    for i in range(0, rows, step):
        e = min(rows, i + step)
        part = lambda k: s[k].view(rows, H)[i:e].double()  # noqa: E731
        col = lambda j: S[j][i:e, None]  # noqa: E731
        dy, hh = part("dy"), (part("h") - col(2)) * col(3)
        w = dy * ng
        D = w - hh * (w * hh).mean(1, keepdim=True)
        if case["pre"] == "layer":
            D = D - w.mean(1, keepdim=True)
        D = D * col(3) + part("dh")
        dng += (dy * hh).sum(0)
        dnb += dy.sum(0)
        dx[i:e] = a * D
        f = part("f")
        fh = (f - col(0)) * col(1) if case["post"] != "none" else f
        dgn = b * D * (fh * pg + pb)
        if dgr is not None:
            dgr.index_add_(0, torch.arange(i, e, device="cuda") // case["rpg"], dgn)
        else:
            dgc += dgn.sum(0)
        dn = b * D * gates(i, e)
        dpg += (dn * fh).sum(0)
        dpb += dn.sum(0)
        if case["post"] != "none":
            w = dn * pg
            dn = w - fh * (w * fh).mean(1, keepdim=True)
            if case["post"] == "layer":
                dn = dn - w.mean(1, keepdim=True)
            dn = dn * col(1)
        df[i:e] = dn
    out = {"df": df.view(s["f"].shape), "dx": dx.view(s["f"].shape), "dpre_gamma": dng[0]}
    if "pre_beta" in par:
        out["dpre_beta"] = dnb[0]
    if "post_gamma" in par:
        out["dpost_gamma"] = dpg[0]
    if "post_beta" in par:
        out["dpost_beta"] = dpb[0]
    if gate is not None:
        out["dgate"] = dgc[0] if case["gate"] == "channel" else dgr.view(s["par"]["gate"].shape)
    return out


# -------------------------------------------------------------------- work
def work(case):
    S = BYTES[case["dtype"]]
    if case["op"] == "clip":
        n = sum(_sizes(case))
        # gradients at or under the limit in place: nothing has to be written
        wr = {"fp32": 4, "same": S, "inplace": 0}[case["out"]]
        return {"bytes": n * (S + wr) + 4, "flops": 2 * n + (n if wr else 0)}
    rows, H = case["rows"], case["H"]
    N = rows * H
    params = sum(H * 4 * (1 + (case["beta"] and case[k] == "layer"))
                 for k in ("post", "pre") if case[k] != "none")
    gate = {"none": 0, "channel": 4 * H, "rows": S * N // max(1, case["rpg"])}[case["gate"]]
    stat = 4 * rows * sum({"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("post", "pre"))
    if case["op"] == "fwd":
        return {"bytes": 4 * N * S + params + gate + (stat if case["train"] else 0), "flops": 16 * N}
    # f is needed for the post norm's gradients and the gate's alone
    reads = 4 if case["post"] != "none" or case["gate"] != "none" else 3
    return {"bytes": (reads + 2) * N * S + 2 * params + 2 * gate + stat, "flops": 40 * N}
