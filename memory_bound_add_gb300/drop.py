"""Dropout with a mask that is never stored, alone and at the block boundary.

Binding of ``include/addln_dropout.h`` (argument marshalling only, like
``binding``), with its training use: for the rows of a block's output f and
the residual stream x,

    d = dropout(f + bias);  h = x + d;  y = norm(h)

``norm`` is ``None``, ``"rms"`` or ``"layer"``.  f and x are contiguous
``[..., H]`` CUDA tensors of one dtype (fp32, fp16 or bf16); bias, gamma and
beta are fp32 ``[H]``.  What stands beside f row for row has f's shape, but that
leading sizes may be joined.

A mask is a function of ``rng`` and of the elements' indexes (the header says
which): the call's backward, given the same ``rng``, makes it again.  ``rng`` is

    (seed, offset)          two whole numbers of up to 64 bits
    an int64 CUDA tensor    of two elements, seed and offset, which the kernel
                            reads when it runs: a captured graph can advance it

Use another offset for every call.  p counts in steps of 2^-16.
"""
from __future__ import annotations

import contextlib
import copy
import ctypes
import functools
import operator
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import binding, fast
from .binding import DTYPE_CODE, AddLNError
from .block import (_F32, _F, _I, _I64, _NORMS, _P, _addresses, _beside, _current_device, _current_stream, _norm_kind,
                    _rows_tensor, _tensor, changed, on_stream)

_D, _U64 = ctypes.c_double, ctypes.c_uint64
# Every symbol include/addln_dropout.h declares, with its ctypes signature.
SIGNATURES = {
    "dropout_fwd": (_I, [_P, _P, _I64, _D, _P, _U64, _U64, _I, _P]),
    "dropout_add_norm_fwd": (_I, [_P, _P, _P, _D, _P, _U64, _U64, _I, _P, _P, _P, _P, _P, _P, _I64, _I64, _F, _I, _P]),
    "dropout_add_norm_bwd": (_I, [_P, _P, _P, _D, _P, _U64, _U64, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I,
                                  _P, _I64, _P]),
    "dropout_add_norm_bwd_workspace_size": (_I64, [_I64, _I64, _I]),
}

_MOST = (1 << 64) - 1

_lib = None
_fast = None  # fast.py's extension, from the first call on
_NONE = (None, None)


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


def _rng_args(rng, index):
    """(address or None, seed, offset) of an rng for device number `index`."""
    if isinstance(rng, torch.Tensor):
        return _tensor(rng, "rng", torch.int64, 2, index), 0, 0
    if type(rng) is tuple and len(rng) == 2:
        seed, offset = rng
        if type(seed) is int and type(offset) is int and 0 <= seed <= _MOST and 0 <= offset <= _MOST:
            return None, seed, offset
    try:
        seed, offset = map(operator.index, rng)
    except TypeError:
        raise TypeError("rng must be two whole numbers (seed, offset) or an int64 tensor of two") from None
    for v in (seed, offset):
        if not -(1 << 63) <= v < 1 << 64:
            raise ValueError(f"rng: {v} has more than 64 bits")
    return None, seed, offset


def _activation(x, name):
    """The dtype's code of a contiguous CUDA tensor of any shape."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = DTYPE_CODE.get(x.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def _on(x, stream, call):
    """on_stream, without its detours in the commonest case."""
    if stream is None and (index := x.get_device()) == _current_device():
        return call(_current_stream(index))
    return on_stream(x.device, stream, call)


# ------------------------------------------------------------------ dropout
def _dropout(s, x, y, p, rng, code):
    rc = (_lib or lib()).dropout_fwd(x.data_ptr(), y, x.numel(), p, *_rng_args(rng, x.get_device()), code, s)
    if rc:
        raise AddLNError(rc, "dropout_fwd")


def dropout_fwd(x, y, p, rng, *, stream=None):
    """Dropout of x (any shape, contiguous) into y, which may be x itself."""
    code = _activation(x, "x")
    at = _tensor(y, "y", x.dtype, x.numel(), x.get_device())
    on_stream(x.device, stream, lambda s: _dropout(s, x, at, p, rng, code))
    changed([y])


def dropout(x, p, rng, *, stream=None):
    """Dropout of x; its backward is the same call on the gradient (no graph is
    made here: dropout_train makes one)."""
    if _fast is not None and stream is None:
        y = _fast.dropout(x, p, rng)
        if y is not None:
            return y
    code = _activation(x, "x")

    def call(s):
        y = torch.empty_like(x)
        _dropout(s, x, y.data_ptr(), p, rng, code)
        return y

    return _on(x, stream, call)


# ------------------------------------------------------------------ forward
def _forward(s, f, x, outs, rows, H, p, rng, bias, norm, gamma, beta, eps):
    """f, and outs, the addresses of h, y and the statistics, are checked."""
    dev = f.get_device()
    rc = (_lib or lib()).dropout_add_norm_fwd(
        f.data_ptr(), None if x is None else _beside(x, "x", f, dev),
        None if bias is None else _tensor(bias, "bias", _F32, H, dev), p, *_rng_args(rng, dev),
        _norm_kind(norm, "norm"), None if gamma is None else _tensor(gamma, "gamma", _F32, H, dev),
        None if beta is None else _tensor(beta, "beta", _F32, H, dev), *outs, rows, H, eps, DTYPE_CODE[f.dtype], s)
    if rc:
        raise AddLNError(rc, "dropout_add_norm_fwd")


def dropout_add_norm_fwd(f, x, h, y=None, stats=None, *, p, rng, bias=None, norm="layer", gamma=None, beta=None,
                         eps: float = 1e-5, stream=None):
    """The boundary into caller-provided h (None: not written) and y ([..., H],
    f's dtype; each may be f or x itself) and, with stats = (mean, rstd), into
    [rows] fp32 tensors (None: not written).  x None: h = dropout(f + bias)."""
    rows, H = _rows_tensor(f, "f")
    dev = f.get_device()
    mean, rstd = stats or _NONE
    outs = (_beside(h, "h", f, dev), _beside(y, "y", f, dev), _tensor(mean, "mean", _F32, rows, dev),
            _tensor(rstd, "rstd", _F32, rows, dev))
    on_stream(f.device, stream, lambda s: _forward(s, f, x, outs, rows, H, p, rng, bias, norm, gamma, beta, eps))
    changed([t for t in (h, y, mean, rstd) if t is not None])


def dropout_add_norm(f, x=None, *, p, rng, bias=None, norm="layer", gamma=None, beta=None, eps: float = 1e-5,
                     want_stats: bool = False, stream=None):
    """Allocate the outputs with PyTorch and run dropout_add_norm_fwd (no graph
    is made here: dropout_add_norm_train makes one).

    Returns (h, y or None, stats or None), stats = (mean, rstd), each [rows]
    fp32 or None where the norm has none.
    """
    if _fast is not None and stream is None:
        out = _fast.dropout_add_norm(f, x, p, rng, bias, _NORMS.get(norm), gamma, beta, eps, want_stats)
        if out is not None:
            return out[0], out[1], out[2:] if want_stats else None
    rows, H = _rows_tensor(f, "f")

    def call(s):
        h = torch.empty_like(f)
        y = torch.empty_like(f) if norm is not None else None
        stats = None
        mp = rp = None
        if want_stats:
            mean = rstd = None
            if norm is not None:
                rstd = torch.empty(rows, dtype=_F32, device=f.device)
                rp = rstd.data_ptr()
                if norm == "layer":
                    mean = torch.empty(rows, dtype=_F32, device=f.device)
                    mp = mean.data_ptr()
            stats = (mean, rstd)
        _forward(s, f, x, (h.data_ptr(), None if y is None else y.data_ptr(), mp, rp), rows, H, p, rng, bias, norm, gamma,
                 beta, eps)
        return h, y, stats

    return _on(f, stream, call)


# ----------------------------------------------------------------- backward
class DropoutAddNormGrads(NamedTuple):
    """Gradients of the boundary; None where there is no such input.  Without
    a norm dx is dh itself."""
    df: torch.Tensor
    dx: torch.Tensor
    dbias: Optional[torch.Tensor]
    dgamma: Optional[torch.Tensor]
    dbeta: Optional[torch.Tensor]


def dropout_add_norm_bwd_workspace_size(rows: int, H: int, dtype: int) -> int:
    n = int(lib().dropout_add_norm_bwd_workspace_size(int(rows), int(H), int(dtype)))
    if n < 0:
        raise AddLNError(n, "dropout_add_norm_bwd_workspace_size")
    return n


@functools.lru_cache(maxsize=256)
def _workspace_size(rows, H, code, index):
    """dropout_add_norm_bwd_workspace_size on device number `index`, which is
    current: a number that these arguments alone decide."""
    return dropout_add_norm_bwd_workspace_size(rows, H, code)


def _given(dy, dh):
    """The gradient that is given, with its rows and H."""
    some, name = (dy, "dy") if dy is not None else (dh, "dh")
    return (some, *_rows_tensor(some, name))


def _backward(s, some, rows, H, dy, dh, h, stats, outs, p, rng, norm, gamma, workspace):
    """outs: the addresses of df, dx and the vectors' gradients, checked."""
    dev, code = some.get_device(), DTYPE_CODE[some.dtype]
    mean, rstd = stats or _NONE
    size = 0
    if workspace is None:
        if any(outs[2:]):
            size = _workspace_size(rows, H, code, dev)
            workspace = torch.empty(size, dtype=torch.uint8, device=some.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    else:
        size = workspace.numel() * workspace.element_size()
    rc = (_lib or lib()).dropout_add_norm_bwd(
        None if dy is None else _beside(dy, "dy", some, dev), None if dh is None else _beside(dh, "dh", some, dev),
        None if h is None else _beside(h, "h", some, dev), p, *_rng_args(rng, dev), _norm_kind(norm, "norm"),
        None if gamma is None else _tensor(gamma, "gamma", _F32, H, dev),
        None if mean is None else _tensor(mean, "mean", _F32, rows, dev),
        None if rstd is None else _tensor(rstd, "rstd", _F32, rows, dev), *outs, rows, H, code,
        None if workspace is None else workspace.data_ptr(), size, s)
    if rc:
        raise AddLNError(rc, "dropout_add_norm_bwd")


def dropout_add_norm_bwd(dy, dh, h, stats, df, dx, *, p, rng, norm="layer", gamma=None, dbias=None, dgamma=None,
                         dbeta=None, workspace=None, stream=None):
    """Backward of dropout_add_norm_fwd into caller-provided df, dx (None: not
    written) and whichever of dbias, dgamma and dbeta are given.  dy or dh may
    be None (no gradient reaches y, or h from elsewhere); h is read for dy
    alone.  workspace: a CUDA tensor of at least
    dropout_add_norm_bwd_workspace_size(...) bytes, reusable call after call
    (allocated here when None)."""
    some, rows, H = _given(dy, dh)
    dev = some.get_device()
    outs = (_beside(df, "df", some, dev), _beside(dx, "dx", some, dev), _tensor(dbias, "dbias", _F32, H, dev),
            _tensor(dgamma, "dgamma", _F32, H, dev), _tensor(dbeta, "dbeta", _F32, H, dev))
    on_stream(some.device, stream, lambda s: _backward(s, some, rows, H, dy, dh, h, stats, outs, p, rng, norm, gamma,
                                                       workspace))
    changed([t for t in (df, dx, dbias, dgamma, dbeta) if t is not None])


def dropout_add_norm_backward(dy, dh, h, stats, *, p, rng, bias=None, norm="layer", gamma=None, beta=None,
                              stream=None) -> DropoutAddNormGrads:
    """Allocate the gradients with PyTorch and run dropout_add_norm_bwd: the
    gradient of every input that is given."""
    if _fast is not None and stream is None:
        mean, rstd = stats or _NONE
        g = _fast.dropout_add_norm_backward(dy, dh, h, mean, rstd, p, rng, bias, _NORMS.get(norm), gamma, beta)
        if g is not None:
            return tuple.__new__(DropoutAddNormGrads, g if norm is not None else (g[0], dh, *g[2:]))
    some, rows, H = _given(dy, dh)
    dev = some.get_device()
    for t, name in ((bias, "bias"), (beta, "beta")):
        if t is not None:
            _tensor(t, name, _F32, H, dev)
    dx_is_dh = norm is None

    def call(s):
        g = (torch.empty_like(some), None if dx_is_dh else torch.empty_like(some),
             None if bias is None else torch.empty_like(bias), None if gamma is None else torch.empty_like(gamma),
             None if beta is None else torch.empty_like(beta))
        _backward(s, some, rows, H, dy, dh, h, stats, _addresses(g), p, rng, norm, gamma, None)
        return DropoutAddNormGrads(g[0], dh if dx_is_dh else g[1], *g[2:])

    return _on(some, stream, call)


# ----------------------------------------------------------------- training
def _frozen(rng):
    """rng as it is now: the backward has to make this call's mask, however
    the tensor (or list, or array) is advanced meanwhile."""
    if isinstance(rng, torch.Tensor):
        return rng.clone()
    try:
        return tuple(map(operator.index, rng))
    except TypeError:
        return rng  # refused where it is used


class DropoutFunction(torch.autograd.Function):
    """dropout with its gradient."""

    @staticmethod
    def forward(ctx, x, p, rng):
        ctx.p, ctx.rng = p, _frozen(rng)
        return dropout(x.contiguous(), p, ctx.rng)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return dropout(dy.contiguous(), ctx.p, ctx.rng), None, None


def dropout_train(x, p, rng):
    """dropout(x, p, rng) with a gradient for x (first order only)."""
    return DropoutFunction.apply(x, p, rng)


class DropoutAddNormFunction(torch.autograd.Function):
    """(h, y) of the boundary with gradients for f, x, bias, gamma and beta;
    without a norm y is None."""

    @staticmethod
    def forward(ctx, f, x, bias, gamma, beta, p, rng, norm, eps):
        if x is not None and f.shape != x.shape:
            raise ValueError(f"f of shape {tuple(f.shape)} beside x of {tuple(x.shape)}")
        cont = lambda t: None if t is None else t.contiguous()  # noqa: E731
        f, x, bias, gamma, beta = map(cont, (f, x, bias, gamma, beta))
        ctx.p, ctx.rng, ctx.norm = p, _frozen(rng), norm
        h, y, stats = dropout_add_norm(f, x, p=p, rng=ctx.rng, bias=bias, norm=norm, gamma=gamma, beta=beta,
                                       eps=float(eps), want_stats=True)
        ctx.save_for_backward(h if norm is not None else None, gamma, *stats)
        ctx.set_materialize_grads(False)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        if dh is None and dy is None:
            return (None,) * 9
        h, gamma, *stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        dh = None if dh is None else dh.contiguous()
        dy = None if dy is None else dy.contiguous()
        some = dy if dy is not None else dh
        H = some.shape[-1]
        new = lambda n: torch.empty(H, dtype=_F32, device=some.device) if need[n] else None  # noqa: E731
        dbias, dgamma, dbeta = new(2), new(3), new(4)
        df = torch.empty_like(some)
        # without dy the stream's gradient passes unchanged
        dx = torch.empty_like(some) if need[1] and dy is not None else None
        dropout_add_norm_bwd(dy, dh, h, stats, df, dx, p=ctx.p, rng=ctx.rng, norm=ctx.norm, gamma=gamma, dbias=dbias,
                             dgamma=dgamma, dbeta=dbeta)
        if need[1] and dy is None:
            dx = dh
        return (df if need[0] else None, dx if need[1] else None, dbias, dgamma, dbeta) + (None,) * 4


def dropout_add_norm_train(f, x=None, *, p, rng, bias=None, norm="layer", gamma=None, beta=None, eps: float = 1e-5):
    """(h, y or None) of the boundary, with gradients for every tensor argument
    but rng (first order only).  A tensor rng may be advanced at once: the
    backward uses a copy."""
    return DropoutAddNormFunction.apply(f, x, bias, gamma, beta, p, rng, norm, eps)


def _new_rng(device):
    """A seed from torch's generator and an offset of 0."""
    seed = int(torch.randint(0, (1 << 63) - 1, (), device="cpu"))
    return torch.tensor([seed, 0], dtype=torch.int64, device=device)


class FusedDropoutAddNorm(torch.nn.Module):
    """The boundary as a module: norm(x + dropout(f + input_bias)) with fp32
    parameters of size `hidden` (weight ones, bias zeros; input_bias zeros, with
    it only).  Returns (h, y).  Its seed and offset lie in the tensor `rng`,
    seeded from torch's generator; each training step takes the next offset, in
    device memory, so that a captured step draws a new mask at every replay.
    rng moves, is saved and is loaded with the module, but is no buffer, or
    DistributedDataParallel would give all ranks rank 0's masks; ranks whose masks
    are to differ need seeds that do (another torch.manual_seed, or rng[0] += rank,
    after loading a state too).
    forward's own rng replaces them.  A step that is computed again during the
    backward (activation checkpointing) would find the offset moved on, so there
    forward refuses to draw; pass rng to such steps:

        rng = m.rng.clone()
        m.rng[1] += 1
        h, y = checkpoint(m, f, x, rng, use_reentrant=False)

    A deepcopy draws a seed of its own, so that layers made as copies of one drop
    different places; a loaded state has the seed and offset that were saved.
    In eval() nothing is dropped."""

    def __init__(self, hidden: int, p: float = 0.1, norm: Optional[str] = "layer", bias: bool = True,
                 input_bias: bool = False, eps: float = 1e-5, device=None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be between 0 and 1, got {p}")
        _norm_kind(norm, "norm")
        self.p, self.norm, self.eps = float(p), norm, float(eps)
        new = lambda v, w: torch.nn.Parameter(  # noqa: E731
            torch.full((hidden,), float(v), dtype=torch.float32, device=device)) if w else None
        self.weight = new(1, norm is not None)
        self.bias = new(0, norm is not None and bias)
        self.input_bias = new(0, input_bias)
        self.rng = _new_rng(device)

    @contextlib.contextmanager
    def _rng_as_buffer(self):
        """What moves, saves and loads buffers takes rng for one inside."""
        self._buffers["rng"] = self.__dict__.pop("rng")
        try:
            yield
        finally:
            self.__dict__["rng"] = self._buffers.pop("rng")

    def _apply(self, *args, **kw):
        with self._rng_as_buffer():
            return super()._apply(*args, **kw)

    def _save_to_state_dict(self, *args, **kw):
        with self._rng_as_buffer():
            super()._save_to_state_dict(*args, **kw)

    def _load_from_state_dict(self, *args, **kw):
        with self._rng_as_buffer():
            super()._load_from_state_dict(*args, **kw)

    def __setstate__(self, state):
        super().__setstate__(state)
        if "rng" in self._buffers:  # pickled when it was a buffer
            self.rng = self._buffers.pop("rng")

    def __deepcopy__(self, memo):
        new = type(self).__new__(type(self))
        memo[id(self)] = new
        new.__dict__.update(copy.deepcopy(self.__dict__, memo))
        new.rng = _new_rng(self.rng.device)
        return new

    def forward(self, f, x=None, rng=None):
        p = self.p if self.training else 0.0
        advance = rng is None and p > 0.0
        if advance and torch._C._current_graph_task_id() != -1:
            raise RuntimeError("FusedDropoutAddNorm computed during a backward (checkpointing?) would draw another mask than "
                               "the step's first forward: pass rng")
        if rng is None:
            rng = self.rng if p > 0.0 else (0, 0)
        out = dropout_add_norm_train(f, x, p=p, rng=rng, bias=self.input_bias, norm=self.norm, gamma=self.weight,
                                     beta=self.bias, eps=self.eps)
        if advance:
            self.rng[1] += 1
        return out
