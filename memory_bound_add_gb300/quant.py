"""Residual sum and norm with an output in 8 bits and its scales.

Binding of ``include/addln_quant.h`` (argument marshalling only, like
``binding``): for the rows of x and the residual stream,

    h = x + residual;  y = norm(h);  q = round(y / scale)

so that q * scale stands for y.  ``norm`` is ``None``, ``"rms"`` or ``"layer"``.
x and residual are contiguous ``[..., H]`` CUDA tensors of one dtype (fp32, fp16
or bf16); gamma and beta are fp32 ``[H]``.

``format``   ``"e4m3"``, ``"e5m2"`` or ``"int8"``: q is a ``torch.float8_e4m3fn``,
             ``torch.float8_e5m2`` or ``torch.int8`` tensor of x's shape
``scaling``  ``"row"``     fp32 scales ``[..., 1]``
             ``"group"``   fp32 ``[..., groups]``, one for every `group` columns
             ``"pow2"``    the same, powers of two, ``torch.float8_e8m0fnu``
             ``"tensor"``  one given fp32 scale

Training with the values that q stands for: ``block_norm_backward(dy, dh, None,
h, (None, None, mean, rstd), pre=norm, pre_gamma=gamma, pre_beta=beta)`` gives
the gradients (h: x where there is no residual).
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import binding, fast
from .binding import DTYPE_CODE, AddLNError
from .block import (NORM_LAYER, _F32, _F, _I, _I64, _P, _beside, _current_device, _current_stream, _norm_kind, _rows_tensor, _same_rows,
                    _tensor, changed, on_stream)

Q_E4M3, Q_E5M2, Q_INT8 = 0, 1, 2
SCALE_ROW, SCALE_GROUP, SCALE_POW2, SCALE_TENSOR = 0, 1, 2, 3

_FORMATS = {"e4m3": (Q_E4M3, torch.float8_e4m3fn), "e5m2": (Q_E5M2, torch.float8_e5m2), "int8": (Q_INT8, torch.int8)}
_CODES = {t: c for c, t in _FORMATS.values()}
_SCALINGS = {"row": SCALE_ROW, "group": SCALE_GROUP, "pow2": SCALE_POW2, "tensor": SCALE_TENSOR}
_E8 = torch.float8_e8m0fnu

# Every symbol include/addln_quant.h declares, with its ctypes signature.
SIGNATURES = {
    "norm_quant_fwd": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I64, _I, _P, _P, _P, _P, _I64, _I64, _F, _I, _P]),
    "dequant_rows": (_I, [_P, _I, _I, _I64, _I, _P, _P, _I64, _I64, _I, _P]),
}

_lib = None
_fast = None  # fast.py's extension, from the first call on


def bind(handle):
    """Sets these signatures on a library handle and returns it."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    return handle


def lib():
    global _lib, _fast
    if _lib is None:
        _lib = bind(binding.lib())
        _fast = fast.module()
    return _lib


def _format(name):
    f = _FORMATS.get(name)
    if f is None:
        raise ValueError(f'format must be "e4m3", "e5m2" or "int8", got {name!r}')
    return f


def _group_of(scaling, group):
    """The scaling's code and its group (0 without groups)."""
    code = _SCALINGS.get(scaling)
    if code is None:
        raise ValueError(f'scaling must be "row", "group", "pow2" or "tensor", got {scaling!r}')
    if code in (SCALE_ROW, SCALE_TENSOR):
        if group is not None:
            raise ValueError(f'a group beside scaling "{scaling}"')
        return code, 0
    if group is None:
        group = 32 if code == SCALE_POW2 else 128
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group!r}")
    return code, int(group)


def scale_layout(scale, shape):
    """(scaling, group, group_major) of the scales of a q of this shape;
    ValueError where they do not fit."""
    return _layout(scale.dtype, scale.shape, scale.stride(), shape)


@functools.lru_cache(maxsize=256)
def _layout(dtype, scale_shape, scale_stride, shape):
    """scale_layout of a tensor of these sizes and strides.  A row's groups are told from how many
    there are: no two of 32, 64 and 128 columns cut a row into the same number,
    but for one."""
    H = shape[-1]
    scale = torch.empty_strided(scale_shape, scale_stride, dtype=dtype, device="meta")
    if scale.dtype not in (_F32, _E8):
        raise ValueError(f"scale must be {_F32} or {_E8}, got {scale.dtype}")
    if scale.numel() == 1 and scale.dim() <= 1 and not (scale.dtype is _E8 and len(shape) == scale.dim() == 1):
        if scale.dtype is not _F32:
            raise ValueError(f"a scale for the whole tensor must be {_F32}")
        return SCALE_TENSOR, 0, 0
    bad = ValueError(f"scale of shape {tuple(scale.shape)} does not fit {tuple(shape)}")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    if not scale.dim() or not _same_rows((*scale.shape[:-1], H), shape):
        raise bad
    G = scale.shape[-1]
    pow2 = scale.dtype is _E8
    if G == 1 and not pow2:
        scaling, group = SCALE_ROW, 0
    else:
        for group in (128, 64, 32):
            if G == -(-H // group):
                break
        else:
            raise bad
        scaling = SCALE_POW2 if pow2 else SCALE_GROUP
    if scale.is_contiguous():
        return scaling, group, 0
    # [groups, rows] in memory: rows lie side by side
    if scaling != SCALE_ROW and scale.movedim(-1, 0).is_contiguous():
        return scaling, group, 1
    raise ValueError("scale must be contiguous, or contiguous with its groups first")


# ------------------------------------------------------------------ forward
def _forward(s, x, residual, q, scale, h, mean, rstd, rows, H, norm, gamma, beta, eps, fmt, scaling, group, group_major):
    """q, scale, h, mean and rstd are addresses, checked."""
    dev = x.get_device()
    rc = (_lib or lib()).norm_quant_fwd(
        x.data_ptr(), None if residual is None else _beside(residual, "residual", x, dev), _norm_kind(norm, "norm"),
        None if gamma is None else _tensor(gamma, "gamma", _F32, H, dev),
        None if beta is None else _tensor(beta, "beta", _F32, H, dev), q, fmt, scaling, group, group_major, scale, h,
        mean, rstd, rows, H, eps, DTYPE_CODE[x.dtype], s)
    if rc:
        raise AddLNError(rc, "norm_quant_fwd")


def _q_tensor(q, name, shape, index):
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if q.dtype not in _CODES:
        raise ValueError(f"{name} must be one of {', '.join(map(str, _CODES))}, got {q.dtype}")
    if q.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {q.device}")
    if not q.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if q.shape != shape and not (q.dim() and _same_rows(q.shape, shape)):
        raise ValueError(f"{name} of shape {tuple(q.shape)} beside {tuple(shape)}")
    return q.data_ptr()


def norm_quant_fwd(x, residual, q, scale, h=None, stats=None, *, norm="rms", gamma=None, beta=None, eps: float = 1e-5,
                   stream=None):
    """Into caller-provided q (its dtype says the format) and scale (its dtype,
    shape and strides say the scaling; fp32 of one element and at most one
    dimension: a given scale, which is read), and h (None: not written; it may
    be x or residual itself) and stats = (mean, rstd), [rows] fp32 (None: not
    written)."""
    rows, H = _rows_tensor(x, "x")
    dev = x.get_device()
    at = _q_tensor(q, "q", x.shape, dev)
    if not isinstance(scale, torch.Tensor):
        raise TypeError("scale must be a torch.Tensor")
    if scale.get_device() != dev:
        raise ValueError(f"scale must be on cuda:{dev}, got {scale.device}")
    scaling, group, group_major = scale_layout(scale, x.shape)
    mean, rstd = stats or (None, None)
    hp = _beside(h, "h", x, dev)
    mp, rp = _tensor(mean, "mean", _F32, rows, dev), _tensor(rstd, "rstd", _F32, rows, dev)
    on_stream(x.device, stream, lambda s: _forward(s, x, residual, at, scale.data_ptr(), hp, mp, rp, rows, H, norm, gamma,
                                                   beta, eps, _CODES[q.dtype], scaling, group, group_major))
    written = [q, h, mean, rstd] + ([scale] if scaling != SCALE_TENSOR else [])
    changed([t for t in written if t is not None])


class NormQuant(NamedTuple):
    """q and its scales; h where there is a residual, mean and rstd (flat
    [rows]) where statistics are wanted and the norm has them."""
    q: torch.Tensor
    scale: torch.Tensor
    h: Optional[torch.Tensor]
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


def norm_quant(x, residual=None, *, norm="rms", gamma=None, beta=None, eps: float = 1e-5, format: str = "e4m3",
               scaling: str = "row", group: Optional[int] = None, scale=None, group_major: bool = False,
               want_stats: bool = False, stream=None) -> NormQuant:
    """Allocate the outputs with PyTorch and run norm_quant_fwd.  group: 128 by
    default, 32 for "pow2".  scale: the given one, for scaling "tensor" alone.
    group_major: the scales of groups lie as [groups, rows] in memory (the
    tensor returned has the same shape and other strides)."""
    spec = _spec(norm, format, scaling, group, bool(group_major))
    if _fast is not None and stream is None and scale is None and not spec[5]:
        out = _fast.norm_quant(x, residual, gamma, beta, eps, spec[0], spec[1], spec[3], spec[4], want_stats)
        if out is not None:
            return tuple.__new__(NormQuant, out)
    rows, H = _rows_tensor(x, "x")
    if spec[3] == SCALE_TENSOR:
        if not isinstance(scale, torch.Tensor):
            raise TypeError('scaling "tensor" needs a scale: an fp32 tensor of one element')
        _tensor(scale, "scale", _F32, 1, x.get_device())
    elif scale is not None:
        raise ValueError(f'a scale beside scaling "{scaling}"')
    # the commonest call without on_stream's detour
    if stream is None and (index := x.get_device()) == _current_device():
        return _norm_quant(_current_stream(index), x, residual, rows, H, gamma, beta, eps, spec, scale, want_stats)
    return on_stream(x.device, stream, lambda s: _norm_quant(s, x, residual, rows, H, gamma, beta, eps, spec, scale,
                                                             want_stats))


@functools.lru_cache(maxsize=256)
def _spec(norm, format, scaling, group, group_major):
    """(norm's code, format's code, q's dtype, scaling's code, group, whether
    the groups come first, the scales' dtype) of a call's choices."""
    code, g = _group_of(scaling, group)
    return (_norm_kind(norm, "norm"), *_format(format), code, g, group_major and g != 0,
            _E8 if code == SCALE_POW2 else _F32)


def _norm_quant(s, x, residual, rows, H, gamma, beta, eps, spec, scale, want_stats):
    norm, fmt, qt, code, g, major, st = spec
    dev = x.get_device()
    new = torch.empty
    q = torch.empty_like(x, dtype=qt)
    if code != SCALE_TENSOR:
        G = -(-H // g) if g else 1
        lead = x.shape[:-1]
        scale = new((G, *lead), dtype=st, device=x.device).movedim(0, -1) if major else \
            new((*lead, G), dtype=st, device=x.device)
    h = mean = rstd = rp = hp = None
    if residual is not None:
        rp = _beside(residual, "residual", x, dev)
        h = torch.empty_like(x)
        hp = h.data_ptr()
    if want_stats and norm:
        rstd = new(rows, dtype=_F32, device=x.device)
        if norm == NORM_LAYER:
            mean = new(rows, dtype=_F32, device=x.device)
    rc = (_lib or lib()).norm_quant_fwd(
        x.data_ptr(), rp, norm, None if gamma is None else _tensor(gamma, "gamma", _F32, H, dev),
        None if beta is None else _tensor(beta, "beta", _F32, H, dev), q.data_ptr(), fmt, code, g, major,
        scale.data_ptr(), hp, None if mean is None else mean.data_ptr(), None if rstd is None else rstd.data_ptr(), rows,
        H, eps, DTYPE_CODE[x.dtype], s)
    if rc:
        raise AddLNError(rc, "norm_quant_fwd")
    return NormQuant(q, scale, h, mean, rstd)


# ------------------------------------------------------------------ read back
def _dequant(s, q, scale, out, layout, dtype):
    H = q.shape[-1]
    rc = (_lib or lib()).dequant_rows(q.data_ptr(), _CODES[q.dtype], *layout, scale.data_ptr(), out, q.numel() // H, H,
                                      DTYPE_CODE[dtype], s)
    if rc:
        raise AddLNError(rc, "dequant_rows")


def _check_pair(q, scale):
    if not isinstance(q, torch.Tensor) or not isinstance(scale, torch.Tensor):
        raise TypeError("q and scale must be torch.Tensors")
    index = q.get_device()
    if index >= 0 and q.dtype in _CODES and q.is_contiguous() and scale.get_device() == index and q.dim() and q.shape[-1]:
        return scale_layout(scale, q.shape)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if not q.dim() or q.shape[-1] < 1:
        raise ValueError("q must have a last dimension of at least 1")
    _q_tensor(q, "q", q.shape, q.get_device())
    raise ValueError(f"scale must be on {q.device}, got {scale.device}")


def dequant_rows(q, scale, out, *, stream=None):
    """What q stands for, into out ([..., H], fp32, fp16 or bf16)."""
    layout = _check_pair(q, scale)
    _rows_tensor(out, "out")
    at = _tensor(out, "out", out.dtype, q.numel(), q.get_device())
    if not _same_rows(out.shape, q.shape):
        raise ValueError(f"out of shape {tuple(out.shape)} beside {tuple(q.shape)}")
    on_stream(q.device, stream, lambda s: _dequant(s, q, scale, at, layout, out.dtype))
    changed([out])


def dequantise(q, scale, *, dtype=torch.bfloat16, stream=None):
    """What q stands for, q * scale, as a tensor of this dtype.  The scaling is
    told from scale, as norm_quant returns it (fp32 of one element and at most
    one dimension: a scale for the whole tensor)."""
    if _fast is not None and stream is None:
        out = _fast.dequantise(q, scale, DTYPE_CODE.get(dtype))
        if out is not None:
            return out
    layout = _check_pair(q, scale)
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")

    def call(s):
        out = torch.empty_like(q, dtype=dtype)
        _dequant(s, q, scale, out.data_ptr(), layout, dtype)
        return out

    if stream is None and (index := q.get_device()) == _current_device():
        return call(_current_stream(index))
    return on_stream(q.device, stream, call)
