"""What is measured of the 8-bit norm and the dropout operators.

Four operators:

``quant``  residual sum and norm with an output in 8 bits, and the values
           that it stands for, read back:
               h = x + residual;  y = norm(h);  q = round(y / scale)
``fwd``    dropout, residual sum and norm, forward:
               d = keep ? (f + bias) / (1 - p) : 0;  h = x + d;  y = norm(h)
``bwd``    its gradients: df, dx and those of the bias and the norm
``drop``   dropout alone (its backward is the same call on the gradient)

A dropout mask is a function of (seed, offset, flat index): Philox 4x32-10
(Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011) with the seed as key and (index / 8, offset), 64 bits each, as counter;
its 128 bits serve 8 elements with 16 bits each, the lowest first.  An element
is kept where its 16 bits are at least t = round(65536 p), and scaled by
65536 / (65536 - t).

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it makes the calls of
``memory_bound_add_gb300``.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
# largest value of each 8-bit format
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------- cases
def _quant(name, rows, H, dtype, norm, format, scaling, group=0, beta=False, residual=True, eps=1e-5):
    """scaling: "row" (one scale a row), "group" (one for each `group` columns
    of a row) or "pow2" (the same, each a power of two)."""
    return {"name": name, "op": "quant", "rows": rows, "H": H, "dtype": dtype, "norm": norm,
            "format": format, "scaling": scaling, "group": group, "beta": beta,
            "residual": residual, "eps": eps}


def _block(name, op, rows, H, dtype, norm, p, bias=False, beta=False, dh=True, train=True,
           rng="host", eps=1e-5):
    """norm: "rms", "layer" or "none"; bias: f has a bias that is added before
    the dropout; dh (backward): a gradient reaches h beside y's; train: the
    forward also returns what the backward needs; rng: seed and offset are
    numbers of the host, or in device memory ("device")."""
    return {"name": name, "op": op, "rows": rows, "H": H, "dtype": dtype, "norm": norm, "p": p,
            "bias": bias, "beta": beta, "dh": dh, "train": train, "rng": rng, "eps": eps}


def _drop(name, rows, H, dtype, p, rng="host"):
    return {"name": name, "op": "drop", "rows": rows, "H": H, "dtype": dtype, "p": p, "rng": rng}


def listed():
    return [
        # one token of a served model, a scale for the row: latency
        _quant("quant_token_1x4096_bf16", 1, 4096, "bf16", "rms", "e4m3", "row"),
        # a prompt of 2048 tokens, a power of two for every 32 columns
        _quant("quant_pages_2048x4096_fp16", 2048, 4096, "fp16", "rms", "e4m3", "pow2", 32),
        # odd rows and width (rows start misaligned), integers, a layer norm
        _quant("quant_ragged_4097x1001_bf16", 4097, 1001, "bf16", "layer", "int8", "row", beta=True),
        # the largest activations, a scale for every 128 columns
        _quant("quant_large_32768x8192_bf16", 32768, 8192, "bf16", "rms", "e4m3", "group", 128),
        # BERT-base rows in training: a bias, a layer norm, statistics kept
        _block("fwd_bert_4096x768_fp16", "fwd", 4096, 768, "fp16", "layer", 0.1, bias=True,
               beta=True, rng="device", eps=1e-12),
        # odd rows and width
        _block("fwd_ragged_4097x1001_bf16", "fwd", 4097, 1001, "bf16", "rms", 0.25),
        # the largest activations: 8 sequences of 4096
        _block("fwd_large_32768x8192_bf16", "fwd", 32768, 8192, "bf16", "rms", 0.1, rng="device"),
        # the smallest training step
        _block("bwd_tiny_64x768_fp32", "bwd", 64, 768, "fp32", "layer", 0.1, bias=True, beta=True,
               dh=False),
        _block("bwd_bert_4096x768_fp16", "bwd", 4096, 768, "fp16", "layer", 0.1, bias=True,
               beta=True, dh=False, rng="device", eps=1e-12),
        _block("bwd_large_32768x8192_bf16", "bwd", 32768, 8192, "bf16", "rms", 0.1),
        # one layer's activations, and the largest
        _drop("drop_bert_4096x768_fp16", 4096, 768, "fp16", 0.1, rng="device"),
        _drop("drop_large_32768x8192_bf16", 32768, 8192, "bf16", 0.1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "quant", "fwd", "bwd", "drop"])
    dtype = rng.choice(["fp32", "fp16", "bf16", "bf16"])
    H = _log_int(rng, 32, 8192)
    if rng.random() < 0.75:
        H = max(8, H // 8 * 8)
    rows = _log_int(rng, 1, 8192)
    p = rng.choice([0.1, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 3)])
    where = rng.choice(["host", "device"])
    if op == "quant":
        norm = rng.choice(["rms", "rms", "layer", "none"])
        scaling = rng.choice(["row", "group", "pow2"])
        c = _quant("", rows, H, dtype, norm, rng.choice(["e4m3", "e4m3", "e5m2", "int8"]), scaling,
                   0 if scaling == "row" else rng.choice([32, 64, 128]), beta=norm == "layer",
                   residual=rng.random() < 0.75)
    elif op == "drop":
        c = _drop("", rows, H, dtype, p, where)
    else:
        norm = rng.choice(["rms", "layer", "layer", "none"])
        c = _block("", op, rows, H, dtype, norm, p, bias=rng.random() < 0.5, beta=norm == "layer",
                   dh=norm == "none" or rng.random() < 0.5, train=rng.random() < 0.5, rng=where)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    rows, H = case["rows"], case["H"]

    def normal(shape, scale=1.0, loc=0.0, dtype=torch.float32):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for part in out.view(-1).split(1 << 26):
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(scale).add_(loc))
        return out

    s = {"case": case}
    par = s["par"] = {}
    if case["op"] != "drop" and case["norm"] != "none":
        par["gamma"] = normal((H,), 0.1, 1.0)
        if case["beta"]:
            par["beta"] = normal((H,), 0.1)
    if case["op"] == "quant":
        s["x"] = normal((rows, H), 0.7, 0.1, dt)
        s["residual"] = normal((rows, H), 1.5, 0.0, dt) if case["residual"] else None
        return s
    # a program's seed, and the number of the call
    pair = [(0x5DEECE66D * (int(seed) + 1) + 11) % (1 << 62), 40 + int(seed) % 1000]
    s["rng"] = torch.tensor(pair, device="cuda") if case["rng"] == "device" else tuple(pair)
    if case["op"] == "drop":
        s["x"] = normal((rows, H), 1.0, 0.0, dt)
        return s
    s["bias"] = normal((H,), 0.2) if case["bias"] else None
    if case["op"] == "fwd":
        s["f"] = normal((rows, H), 0.7, 0.1, dt)
        s["x"] = normal((rows, H), 1.5, 0.0, dt)
        return s
    has = case["norm"] != "none"
    s["dy"] = normal((rows, H), 1.0, 0.0, dt) if has else None
    s["dh"] = normal((rows, H), 0.5, 0.0, dt) if case["dh"] else None
    s["h"] = normal((rows, H), 1.7, 0.1, dt) if has else None
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    step = max(1, (1 << 26) // H)
    for i in range(0, rows if has else 0, step):
        v = s["h"][i:i + step].float()
        m = v.mean(1, keepdim=True) if case["norm"] == "layer" else 0.0
        mean[i:i + step] = m.squeeze(1) if case["norm"] == "layer" else 0.0
        rstd[i:i + step] = ((v - m).square().mean(1) + case["eps"]).rsqrt()
    s["stats"] = (mean if case["norm"] == "layer" else None, rstd if has else None)
    return s


# -------------------------------------------------------------- plain forms
_LOW = 0xFFFFFFFF


def _random_words(block, rng):
    """The four 32-bit words of Philox for each of these counters, in int64."""
    seed, offset = rng[0], rng[1]
    c = [block & _LOW, (block >> 32) & _LOW, offset & _LOW, (offset >> 32) & _LOW]
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & _LOW) ^ c[1] ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c[3] ^ k1, a & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c


def _keep(shape, p, rng):
    """(which elements are kept, what they are multiplied by)"""
    n = math.prod(shape)
    t = round(65536 * p)
    words = _random_words(torch.arange(-(-n // 8), device="cuda"), rng)
    bits = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], -1)
    return (bits.view(-1)[:n] >= t).view(shape), 65536.0 / (65536 - t)


def _norm(v, case, par):
    """(normalised, mean or None, rstd or None) over the last dimension."""
    if case["norm"] == "none":
        return v, None, None
    mean = None
    if case["norm"] == "layer":
        mean = v.mean(-1, keepdim=True)
        v = v - mean
    rstd = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + case["eps"])
    out = v * rstd * par["gamma"]
    if "beta" in par:
        out = out + par["beta"]
    return out, mean, rstd


def _plain_quant(case, s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y, _, _ = _norm(h, case, s["par"])
    rows, H = y.shape
    g = case["group"] if case["scaling"] != "row" else H
    G = -(-H // g)
    pad = torch.zeros(rows, G * g, device="cuda")
    pad[:, :H] = y
    parts = pad.view(rows, G, g)
    amax = parts.abs().amax(-1)
    top = QMAX[case["format"]]
    if case["scaling"] == "pow2":
        # the least power of two that leaves nothing above the largest value
        m, e = torch.frexp(amax)
        mt, et = math.frexp(top)
        e = torch.where(amax > 0, e - et + (m > mt), -126).clamp(min=-126)
        scale = torch.ldexp(torch.ones_like(amax), e)
        out_scale = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        scale = (amax / top).clamp(min=2.0 ** -126)
        out_scale = scale
    v = (parts / scale[..., None]).clamp(-top, top)
    q = v.to(FLOAT8[case["format"]]).float() if case["format"] in FLOAT8 else v.round()
    values = (q * scale[..., None]).view(rows, G * g)[:, :H].to(_values_dtype(case))
    out = {"scale": out_scale, "values": values}
    if s["residual"] is not None:
        out["h"] = h.to(s["x"].dtype)
    return out


def _values_dtype(case):
    """What the 8 bits are read back as: a product's 16-bit operand."""
    return torch.bfloat16 if case["dtype"] == "fp32" else DTYPES[case["dtype"]]


def _plain_fwd(case, s):
    z = s["f"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    keep, scale = _keep(z.shape, case["p"], s["rng"])
    h = s["x"].float() + torch.where(keep, z * scale, 0.0)
    y, mean, rstd = _norm(h, case, s["par"])
    return _fwd_out(case, h.to(s["f"].dtype), y.to(s["f"].dtype), (mean, rstd))


def _plain_bwd(case, s):
    out = {}
    dt = DTYPES[case["dtype"]]
    if case["norm"] != "none":
        dy, h = s["dy"].float(), s["h"].float()
        mean, rstd = [None if v is None else v.view(-1, 1) for v in s["stats"]]
        hat = (h if mean is None else h - mean) * rstd
        u = dy * s["par"]["gamma"]
        t = u - hat * (u * hat).mean(-1, keepdim=True)
        if mean is not None:
            t = t - u.mean(-1, keepdim=True)
        D = rstd * t
        out["dgamma"] = (dy * hat).sum(0)
        if "beta" in s["par"]:
            out["dbeta"] = dy.sum(0)
        if s["dh"] is not None:
            D = D + s["dh"].float()
    else:
        D = s["dh"].float()
    keep, scale = _keep(D.shape, case["p"], s["rng"])
    df = torch.where(keep, D * scale, 0.0)
    if s["bias"] is not None:
        out["dbias"] = df.sum(0)
    out["df"] = df.to(dt)
    out["dx"] = D.to(dt)
    return out


def _plain_drop(case, s):
    keep, scale = _keep(s["x"].shape, case["p"], s["rng"])
    return {"y": torch.where(keep, s["x"].float() * scale, 0.0).to(s["x"].dtype)}


# --------------------------------------------------------------------- run
def run(state):
    s = state
    case = s["case"]
    if own:
        import memory_bound_add_gb300 as mba
        if case["op"] == "drop":
            return {"y": mba.dropout(s["x"], case["p"], s["rng"])}
        norm = None if case["norm"] == "none" else case["norm"]
        if case["op"] == "quant":
            r = mba.norm_quant(s["x"], s["residual"], norm=norm, eps=case["eps"], format=case["format"],
                               scaling=case["scaling"], group=case["group"] or None, **s["par"])
            out = {"scale": r.scale, "values": mba.dequantise(r.q, r.scale, dtype=_values_dtype(case))}
            if r.h is not None:
                out["h"] = r.h
            return out
        kw = dict(p=case["p"], rng=s["rng"], bias=s["bias"], norm=norm, **s["par"])
        if case["op"] == "fwd":
            h, y, stats = mba.dropout_add_norm(s["f"], s["x"], eps=case["eps"], want_stats=case["train"], **kw)
            return _fwd_out(case, h, y, stats)
        g = mba.dropout_add_norm_backward(s["dy"], s["dh"], s["h"], s["stats"], **kw)
        return {k: v for k, v in g._asdict().items() if v is not None}
    return {"quant": _plain_quant, "fwd": _plain_fwd, "bwd": _plain_bwd, "drop": _plain_drop}[case["op"]](case, s)


def _fwd_out(case, h, y, stats):
    out = {"h": h}
    if case["norm"] != "none":
        out["y"] = y
        if case["train"]:
            out.update({k: v.view(-1) for k, v in zip(("mean", "rstd"), stats) if v is not None})
    return out


# ------------------------------------------------------------------- exact
def _mul32(a, b):
    """(high, low) 32 bits of the product of 32-bit numbers, from 16-bit halves."""
    lo, mid = (a & 0xFFFF) * b, (a >> 16) * b
    hi = (mid + (lo >> 16)) >> 16
    return hi, ((mid << 16) + lo) & _LOW


def _kept_range(a, b, t, rng):
    """Which of the elements a .. b - 1 of a tensor are kept, by their indexes."""
    seed, offset = (int(v) for v in rng)
    i = torch.arange(a // 8, (b + 7) // 8, device="cuda")
    x0, x1 = i % (1 << 32), i // (1 << 32)
    x2, x3 = (torch.full_like(i, v) for v in (offset % (1 << 32), offset // (1 << 32)))
    for r in range(10):
        h0, l0 = _mul32(x0, 0xD2511F53)
        h1, l1 = _mul32(x2, 0xCD9E8D57)
        x0, x2 = h1 ^ x1 ^ ((seed + r * 0x9E3779B9) % (1 << 32)), h0 ^ x3 ^ ((seed // (1 << 32) + r * 0xBB67AE85) % (1 << 32))
        x1, x3 = l1, l0
    words = torch.stack((x0, x1, x2, x3), 1).view(-1)
    u = torch.arange(a, b, device="cuda")
    return ((words[u // 2 - a // 8 * 4] >> (u % 2 * 16)) % 65536) >= t


def _grid(v, fmt):
    """v to the nearest value of an 8-bit format, ties to even, in 64 bits."""
    top = QMAX[fmt]
    if fmt == "int8":
        return v.round().clamp(-top, top)
    bits, least = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v)[1].double() - 1
    step = torch.exp2(e.clamp(min=least) - bits)
    return (torch.round(v / step) * step).clamp(-top, top)


def exact(case, seed):
    """The same values from the definitions, in 64 bits, some rows at a time."""
    s = prepare(case, seed)
    rows, H = case["rows"], case["H"]
    step = max(1, (1 << 24) // H)
    wide = dict(dtype=torch.float32 if rows * H > 1 << 27 else torch.float64, device="cuda")
    par = {k: v.double() for k, v in s["par"].items()}
    if case["op"] != "quant":
        t = round(65536 * case["p"])
        times = 65536 / (65536 - t)

        def dropped(v, i):
            return v * _kept_range(i * H, i * H + v.numel(), t, s["rng"]).view(v.shape) * times

    def normed(v):
        if case["norm"] == "none":
            return v, None, None
        m = v.mean(1) if case["norm"] == "layer" else torch.zeros_like(v[:, 0])
        v = v - m[:, None]
        r = (v.pow(2).mean(1) + case["eps"]).rsqrt()
        return v * r[:, None] * par["gamma"] + par.get("beta", 0.0), m, r

    new = lambda *k: {n: torch.empty(rows, H, **wide) for n in k}  # noqa: E731
    if case["op"] == "drop":
        out = new("y")
        for i in range(0, rows, step):
            out["y"][i:i + step] = dropped(s["x"][i:i + step].double(), i)
        return out
    if case["op"] == "quant":
        g = case["group"] if case["scaling"] != "row" else H
        G, top = -(-H // g), QMAX[case["format"]]
        out = new("values", "h")
        out["scale"] = torch.empty(rows, G, dtype=torch.float64, device="cuda")
        for i in range(0, rows, step):
            v = s["x"][i:i + step].double()
            if s["residual"] is not None:
                v = v + s["residual"][i:i + step].double()
            out["h"][i:i + step] = v
            y = normed(v)[0]
            for k in range(G):
                w = y[:, k * g:(k + 1) * g]
                sc = w.abs().amax(1) / top
                if case["scaling"] == "pow2":
                    m, e = torch.frexp(sc)
                    sc = torch.where(sc > 0, torch.exp2((e - (m == 0.5).int()).double()), 0.0)
                sc = sc.clamp(min=2.0 ** -126)
                out["scale"][i:i + step, k] = sc
                out["values"][i:i + step, k * g:(k + 1) * g] = _grid(w / sc[:, None], case["format"]) * sc[:, None]
        if s["residual"] is None:
            del out["h"]
        return out
    if case["op"] == "fwd":
        out = new("h", "y") if case["norm"] != "none" else new("h")
        st = torch.zeros(2, rows, dtype=torch.float64, device="cuda")
        for i in range(0, rows, step):
            z = s["f"][i:i + step].double()
            if s["bias"] is not None:
                z = z + s["bias"].double()
            h = s["x"][i:i + step].double() + dropped(z, i)
            y, m, r = normed(h)
            out["h"][i:i + step] = h
            if m is not None:
                out["y"][i:i + step], st[0, i:i + step], st[1, i:i + step] = y, m, r
        if case["train"] and case["norm"] != "none":
            out["rstd"] = st[1]
            if case["norm"] == "layer":
                out["mean"] = st[0]
        return out
    out = new("df", "dx")
    sums = torch.zeros(3, H, dtype=torch.float64, device="cuda")
    mean, rstd = s["stats"]
    for i in range(0, rows, step):
        D = 0.0 if s["dh"] is None else s["dh"][i:i + step].double()
        if case["norm"] != "none":
            dy, hat = s["dy"][i:i + step].double(), s["h"][i:i + step].double()
            if mean is not None:
                hat = hat - mean[i:i + step, None].double()
            r = rstd[i:i + step, None].double()
            hat = hat * r
            u = dy * par["gamma"]
            w = u - hat * (u * hat).mean(1, keepdim=True)
            if mean is not None:
                w = w - u.mean(1, keepdim=True)
            D = D + r * w
            sums[0] += (dy * hat).sum(0)
            sums[1] += dy.sum(0)
        df = dropped(D, i)
        sums[2] += df.sum(0)
        out["dx"][i:i + step], out["df"][i:i + step] = D, df
    for k, name, there in ((0, "dgamma", "gamma" in par), (1, "dbeta", "beta" in par), (2, "dbias", case["bias"])):
        if there:
            out[name] = sums[k]
    return out


# -------------------------------------------------------------------- work
def work(case):
    S = BYTES[case["dtype"]]
    rows, H = case["rows"], case["H"]
    N = rows * H
    if case["op"] == "drop":
        return {"bytes": 2 * N * S, "flops": N}
    has = case["norm"] != "none"
    vectors = 4 * H * (has + case["beta"])
    if case["op"] == "quant":
        # the 8 bits are written, and so are the 16-bit values that they stand for
        G = 1 if case["scaling"] == "row" else -(-H // case["group"])
        scales = rows * G * (1 if case["scaling"] == "pow2" else 4)
        return {"bytes": N * S * (3 if case["residual"] else 1) + N + 2 * N + scales + vectors, "flops": 12 * N}
    vectors += 4 * H * case["bias"]
    stat = 4 * rows * {"none": 0, "rms": 1, "layer": 2}[case["norm"]]
    if case["op"] == "fwd":
        return {"bytes": N * S * (3 + has) + vectors + (stat if case["train"] else 0), "flops": 12 * N}
    # without a norm dx is dh itself: nothing has to be written
    moved = (2 * has + case["dh"]) + (2 if has else 1)
    return {"bytes": moved * N * S + 2 * vectors + stat, "flops": 20 * N}
