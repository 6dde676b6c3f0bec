"""The block boundary: post norm, gate, scaled residual sum and pre norm, fused.

Binding of ``include/addln_block.h`` (argument marshalling only, like
``binding``), with its training use: for the rows of the block's output f and
the residual stream x,

    n = post(f);  h = residual_scale * x + block_scale * gate * n;  y = pre(h)

``post`` and ``pre`` are ``None``, ``"rms"`` or ``"layer"``.  f and x are
contiguous ``[..., H]`` CUDA tensors of one dtype (fp32, fp16 or bf16); what
stands beside f row for row (x, h, y and the gradients) has f's shape, but that
leading sizes may be joined (``[B * S, H]`` beside ``[B, S, H]``).  The norms'
gamma and beta are fp32 ``[H]``.  ``gate`` is one of

    None                 no gate
    fp32 ``[H]``         one value a column (a learnt layer scale)
    ``[..., H]`` in f's dtype, with as many dimensions as f, whose leading
                         sizes are f's up to some dimension and 1 from there
                         on: a gate for every row (f's shape) or one for each
                         sequence (``[B, 1, H]`` for f ``[B, S, H]``).  Its rows
                         may lie apart (a slice of a wider projection).
"""
from __future__ import annotations

import ctypes
import functools
import itertools
import operator
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import DTYPE_CODE, AddLNError

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
GATE_NONE, GATE_CHANNEL, GATE_ROWS = 0, 1, 2
ERR_ALIGN, ERR_KIND, ERR_SCALE, ERR_HOST_MEMORY = -12, -13, -14, -15

_NORMS = {None: NORM_NONE, "rms": NORM_RMS, "layer": NORM_LAYER}

# Every symbol include/addln_block.h declares, with its ctypes signature.
_P, _I64, _F, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
SIGNATURES = {
    "block_norm_fwd": (_I, [_P, _P, _I, _P, _P, _P, _I, _I64, _I64, _F, _F, _I, _P, _P, _P, _P,
                            _P, _P, _P, _P, _I64, _I64, _F, _I, _P]),
    "block_norm_bwd": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I64, _I64, _F, _F, _I,
                            _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _P, _I64, _P]),
    "block_norm_bwd_workspace_size": (_I64, [_I64, _I64, _I, _I, _I64]),
}

_lib = None
_F32 = torch.float32


def bind(handle):
    """Sets these signatures on a library handle and returns it."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    return handle


def lib():
    global _lib
    if _lib is None:
        _lib = bind(binding.lib())
    return _lib


# ------------------------------------------------------------------ helpers
# The current device's index and a device's current stream as a raw handle,
# without the objects that torch.cuda's functions build around them (a few
# microseconds a call, as much as a small launch).
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def on_stream(device, stream, call):
    """call(raw stream handle) with `device` current; what it allocates
    belongs to the stream it launches on."""
    if stream is None:
        index = device.index
        if index == _current_device():
            return call(_current_stream(index))
        with torch.cuda.device(device):
            return call(_current_stream(index))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _tensor(t, name, dtype, n, index):
    """A contiguous CUDA tensor of this dtype, with n elements, on device
    number `index`: its address (None for None, which the library refuses
    where the tensor is required)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _same_rows(a, b) -> bool:
    """Whether these [..., H] shapes are the same rows in the same order: equal
    but for leading sizes that one of them has joined."""
    cuts = lambda s: set(itertools.accumulate(s[:-1], operator.mul)) - {1}  # noqa: E731
    return len(a) > 0 and len(b) > 0 and a[-1] == b[-1] and (cuts(a) <= cuts(b) or cuts(b) <= cuts(a))


def _beside(t, name, like, index):
    """_tensor for what stands row for row beside the activation `like`."""
    if isinstance(t, torch.Tensor) and t.shape == like.shape and t.dtype is like.dtype and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    at = _tensor(t, name, like.dtype, like.numel(), index)
    if t is not None and not _same_rows(t.shape, like.shape):
        raise ValueError(f"{name} of shape {tuple(t.shape)} beside {tuple(like.shape)}")
    return at


def _rows_tensor(t, name):
    """rows and H of a contiguous [..., H] activation."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if not t.dim() or t.shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension (the hidden one) of at least 1")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    H = t.shape[-1]
    return t.numel() // H, H


def _norm_kind(kind, name):
    code = _NORMS.get(kind)
    if code is None:
        raise ValueError(f'{name} must be None, "rms" or "layer", got {kind!r}')
    return code


def gate_layout(gate, shape):
    """(gate rows, row stride, rows per gate row) of a per-row gate for an
    activation of this shape; ValueError where it does not fit."""
    H = shape[-1]
    if gate.dim() != len(shape) or gate.shape[-1] != H:
        raise ValueError(f"gate of shape {tuple(gate.shape)} does not fit {tuple(shape)}")
    lead, want = tuple(gate.shape[:-1]), tuple(shape[:-1])
    k = 0
    while k < len(lead) and lead[k] == want[k]:
        k += 1
    if any(n != 1 for n in lead[k:]):
        raise ValueError(f"gate of shape {tuple(gate.shape)} does not fit {tuple(shape)}: its leading sizes "
                         "have to be the activation's up to some dimension and 1 from there on")
    rpg = 1
    for n in want[k:]:
        rpg *= n
    if gate.numel() == 0:
        return 0, H, max(rpg, 1)
    stride, rows = None, 1
    for n, st in zip(reversed(lead), reversed(gate.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * rows:
            raise ValueError("the gate's rows do not lie at one stride; make it contiguous")
        rows *= n
    if H > 1 and gate.stride(-1) != 1:
        raise ValueError("the gate's last dimension must be contiguous")
    if stride is None:
        stride = H
    if stride < H:
        raise ValueError("the gate's rows overlap (an expanded tensor); make it contiguous")
    return rows, stride, max(rpg, 1)


def _gate_args(gate, x):
    """(address, kind, stride, rows per gate row) of a gate for activation x."""
    if gate is None:
        return None, GATE_NONE, 0, 0
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dim() == 1 and (x.dim() > 1 or gate.dtype is _F32):
        return _tensor(gate, "gate", torch.float32, x.shape[-1], x.get_device()), GATE_CHANNEL, 0, 0
    if gate.dtype != x.dtype:
        raise ValueError(f"a gate with rows must be {x.dtype}, got {gate.dtype}")
    if gate.device != x.device:
        raise ValueError(f"gate must be on {x.device}, got {gate.device}")
    _, stride, rpg = gate_layout(gate, x.shape)
    return gate.data_ptr(), GATE_ROWS, stride, rpg


def changed(ts):
    """Autograd has to see that the tensors of this list were written, so that a
    graph that saved one of them refuses to use it.  Inference tensors have no
    versions."""
    if any(map(torch.Tensor.is_inference, ts)):
        ts = [t for t in ts if not t.is_inference()]
    torch.autograd.graph.increment_version(ts)


def _check(rc, where):
    if rc != binding.OK:
        raise AddLNError(rc, where)


# ------------------------------------------------------------------ forward
_NO_STATS = (None, None, None, None)


def _addresses(ts):
    """Addresses of tensors that were allocated here (None for None)."""
    return [None if t is None else t.data_ptr() for t in ts]


def _forward(s, f, x, outs, rows, H, post, post_gamma, post_beta, gate, pre, pre_gamma, pre_beta, residual_scale,
             block_scale, eps):
    """f, and outs, the addresses of h, y and the statistics, are checked."""
    dt, dev = f.dtype, f.get_device()
    gp, gk, gs, rpg = (None, GATE_NONE, 0, 0) if gate is None else _gate_args(gate, f)
    rc = (_lib or lib()).block_norm_fwd(
        f.data_ptr(), _beside(x, "x", f, dev), _norm_kind(post, "post"),
        None if post_gamma is None else _tensor(post_gamma, "post_gamma", _F32, H, dev),
        None if post_beta is None else _tensor(post_beta, "post_beta", _F32, H, dev),
        gp, gk, gs, rpg, residual_scale, block_scale, _norm_kind(pre, "pre"),
        None if pre_gamma is None else _tensor(pre_gamma, "pre_gamma", _F32, H, dev),
        None if pre_beta is None else _tensor(pre_beta, "pre_beta", _F32, H, dev),
        *outs, rows, H, eps, DTYPE_CODE[dt], s)
    if rc:
        raise AddLNError(rc, "block_norm_fwd")


def block_norm_fwd(f, x, h, y=None, stats=None, *, post=None, post_gamma=None, post_beta=None,
                   gate=None, pre="rms", pre_gamma=None, pre_beta=None, residual_scale: float = 1.0,
                   block_scale: float = 1.0, eps: float = 1e-5, stream=None):
    """The boundary into caller-provided h and y ([..., H], f's dtype; each
    may be f or x itself) and, with stats = (post_mean, post_rstd, pre_mean,
    pre_rstd), into [rows] fp32 tensors (None: not written)."""
    rows, H = _rows_tensor(f, "f")
    dev = f.get_device()
    pm, pr, nm, nr = stats or _NO_STATS
    outs = (_beside(h, "h", f, dev), _beside(y, "y", f, dev), _tensor(pm, "post_mean", _F32, rows, dev),
            _tensor(pr, "post_rstd", _F32, rows, dev), _tensor(nm, "pre_mean", _F32, rows, dev),
            _tensor(nr, "pre_rstd", _F32, rows, dev))
    on_stream(f.device, stream, lambda s: _forward(
        s, f, x, outs, rows, H, post, post_gamma, post_beta, gate, pre, pre_gamma, pre_beta, residual_scale,
        block_scale, eps))
    changed([t for t in (h, y, pm, pr, nm, nr) if t is not None])


def block_norm(f, x, *, post=None, post_gamma=None, post_beta=None, gate=None, pre="rms",
               pre_gamma=None, pre_beta=None, residual_scale: float = 1.0, block_scale: float = 1.0,
               eps: float = 1e-5, want_stats: bool = False, stream=None):
    """Allocate the outputs with PyTorch and run block_norm_fwd.

    Returns (h, y or None, stats or None), stats = (post_mean, post_rstd,
    pre_mean, pre_rstd), each [rows] fp32 or None where the norm has none.
    """
    rows, H = _rows_tensor(f, "f")

    def call(s):
        h = torch.empty_like(f)
        y = torch.empty_like(f) if pre is not None else None
        stats = None
        outs = [h.data_ptr(), None if y is None else y.data_ptr()]
        if want_stats:
            new = lambda w: torch.empty(rows, dtype=_F32, device=f.device) if w else None  # noqa: E731
            stats = (new(post == "layer"), new(post is not None), new(pre == "layer"), new(pre is not None))
        outs.extend(_addresses(stats or _NO_STATS))
        _forward(s, f, x, outs, rows, H, post, post_gamma, post_beta, gate, pre, pre_gamma, pre_beta,
                 residual_scale, block_scale, eps)
        return h, y, stats

    return on_stream(f.device, stream, call)


# ----------------------------------------------------------------- backward
class BlockNormGrads(NamedTuple):
    """Gradients of a block boundary; None where there is no such input."""
    df: torch.Tensor
    dx: torch.Tensor
    dpost_gamma: Optional[torch.Tensor]
    dpost_beta: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpre_gamma: Optional[torch.Tensor]
    dpre_beta: Optional[torch.Tensor]


def block_norm_bwd_workspace_size(rows: int, H: int, dtype: int, gate_kind: int = GATE_NONE,
                                  rows_per_gate: int = 1) -> int:
    n = int(lib().block_norm_bwd_workspace_size(int(rows), int(H), int(dtype), int(gate_kind),
                                                int(rows_per_gate)))
    if n < 0:
        raise AddLNError(n, "block_norm_bwd_workspace_size")
    return n


@functools.lru_cache(maxsize=256)
def _workspace_size(rows, H, code, gate_kind, rows_per_gate, index):
    """block_norm_bwd_workspace_size on device number `index`, which is
    current: a number that these arguments alone decide."""
    return block_norm_bwd_workspace_size(rows, H, code, gate_kind, rows_per_gate)


def _given(dy, dh):
    """The gradient that is given, with its rows and H."""
    some, name = (dy, "dy") if dy is not None else (dh, "dh")
    return (some, *_rows_tensor(some, name))


def _backward(s, some, rows, H, dy, dh, f, h, stats, outs, post, post_gamma, post_beta, gate_args, pre, pre_gamma,
              residual_scale, block_scale, workspace):
    """outs: the addresses of df, dx and the parameters' gradients, checked."""
    dev = some.get_device()
    code = DTYPE_CODE[some.dtype]
    pm, pr, nm, nr = stats or _NO_STATS
    gp, gk, gs, rpg = gate_args
    if workspace is None:
        size = _workspace_size(rows, H, code, gk, rpg or 1, dev)
        workspace = torch.empty(size, dtype=torch.uint8, device=some.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    else:
        size = workspace.numel() * workspace.element_size()
    rc = (_lib or lib()).block_norm_bwd(
        None if dy is None else _beside(dy, "dy", some, dev), None if dh is None else _beside(dh, "dh", some, dev),
        None if f is None else _beside(f, "f", some, dev), None if h is None else _beside(h, "h", some, dev),
        _norm_kind(post, "post"), None if post_gamma is None else _tensor(post_gamma, "post_gamma", _F32, H, dev),
        None if post_beta is None else _tensor(post_beta, "post_beta", _F32, H, dev),
        None if pm is None else _tensor(pm, "post_mean", _F32, rows, dev),
        None if pr is None else _tensor(pr, "post_rstd", _F32, rows, dev), gp, gk, gs, rpg, residual_scale,
        block_scale, _norm_kind(pre, "pre"),
        None if pre_gamma is None else _tensor(pre_gamma, "pre_gamma", _F32, H, dev),
        None if nm is None else _tensor(nm, "pre_mean", _F32, rows, dev),
        None if nr is None else _tensor(nr, "pre_rstd", _F32, rows, dev), *outs, rows, H, code,
        workspace.data_ptr(), size, s)
    if rc:
        raise AddLNError(rc, "block_norm_bwd")


def block_norm_bwd(dy, dh, f, h, stats, df, dx, *, post=None, post_gamma=None, post_beta=None,
                   gate=None, pre="rms", pre_gamma=None, residual_scale: float = 1.0,
                   block_scale: float = 1.0, dpost_gamma=None, dpost_beta=None, dgate=None,
                   dpre_gamma=None, dpre_beta=None, workspace=None, stream=None):
    """Backward of block_norm_fwd into caller-provided df, dx and whichever
    parameter gradients are given.  dy or dh may be None (no gradient reaches
    y, or h from elsewhere).  workspace: a CUDA tensor of at least
    block_norm_bwd_workspace_size(...) bytes, reusable call after call
    (allocated here when None)."""
    some, rows, H = _given(dy, dh)
    dt, dev = some.dtype, some.get_device()
    gate_args = _gate_args(gate, some)
    if dgate is not None and gate is None:
        raise ValueError("dgate without a gate")
    outs = (_beside(df, "df", some, dev), _beside(dx, "dx", some, dev),
            _tensor(dpost_gamma, "dpost_gamma", _F32, H, dev), _tensor(dpost_beta, "dpost_beta", _F32, H, dev),
            None if dgate is None else _tensor(dgate, "dgate", _F32 if gate_args[1] == GATE_CHANNEL else dt,
                                               gate.numel(), dev),
            _tensor(dpre_gamma, "dpre_gamma", _F32, H, dev), _tensor(dpre_beta, "dpre_beta", _F32, H, dev))
    if dgate is not None and dgate.shape != gate.shape and not _same_rows(dgate.shape, gate.shape):
        raise ValueError(f"dgate of shape {tuple(dgate.shape)} beside a gate of {tuple(gate.shape)}")

    def call(s):
        if rows == 0 and dgate is not None:
            dgate.zero_()  # gate rows of empty sequences, which the library does not know of
        _backward(s, some, rows, H, dy, dh, f, h, stats, outs, post, post_gamma, post_beta, gate_args, pre, pre_gamma,
                  residual_scale, block_scale, workspace)

    on_stream(some.device, stream, call)
    changed([t for t in (df, dx, dpost_gamma, dpost_beta, dgate, dpre_gamma, dpre_beta) if t is not None])


def block_norm_backward(dy, dh, f, h, stats, *, post=None, post_gamma=None, post_beta=None, gate=None,
                        pre="rms", pre_gamma=None, pre_beta=None, residual_scale: float = 1.0,
                        block_scale: float = 1.0, stream=None) -> BlockNormGrads:
    """Allocate the gradients with PyTorch and run block_norm_bwd: the
    gradient of every input that is given (beta's gradients where a beta is)."""
    some, rows, H = _given(dy, dh)
    gate_args = _gate_args(gate, some)
    if pre_beta is not None:
        _tensor(pre_beta, "pre_beta", _F32, H, some.get_device())

    def call(s):
        new = torch.empty_like if rows else torch.zeros_like
        g = [torch.empty_like(some), torch.empty_like(some), None if post_gamma is None else new(post_gamma),
             None if post_beta is None else new(post_beta), None if gate is None else
             new(gate) if gate.is_contiguous() else new(gate, memory_format=torch.contiguous_format),
             None if pre_gamma is None else new(pre_gamma), None if pre_beta is None else new(pre_beta)]
        _backward(s, some, rows, H, dy, dh, f, h, stats, _addresses(g), post, post_gamma, post_beta, gate_args, pre,
                  pre_gamma, residual_scale, block_scale, None)
        return BlockNormGrads(*g)

    return on_stream(some.device, stream, call)


# ----------------------------------------------------------------- training
class BlockNormFunction(torch.autograd.Function):
    """(h, y) of the block boundary with gradients for f, x, the norms'
    parameters and the gate; without a pre norm y is None."""

    @staticmethod
    def forward(ctx, f, x, post_gamma, post_beta, gate, pre_gamma, pre_beta, post, pre, residual_scale,
                block_scale, eps):
        if f.shape != x.shape:
            raise ValueError(f"f of shape {tuple(f.shape)} beside x of {tuple(x.shape)}")
        f, x = f.contiguous(), x.contiguous()
        cont = lambda t: None if t is None else t.contiguous()  # noqa: E731
        post_gamma, post_beta, pre_gamma, pre_beta = map(cont, (post_gamma, post_beta, pre_gamma, pre_beta))
        if gate is not None:
            try:
                _gate_args(gate, f)
            except ValueError:
                gate = gate.contiguous()
        ctx.kinds = dict(post=post, pre=pre, residual_scale=float(residual_scale), block_scale=float(block_scale))
        h, y, stats = block_norm(f, x, post_gamma=post_gamma, post_beta=post_beta, gate=gate,
                                 pre_gamma=pre_gamma, pre_beta=pre_beta, eps=float(eps), want_stats=True,
                                 **ctx.kinds)
        # f serves the post norm's and the gate's gradients, h the pre norm's
        ctx.save_for_backward(f if post is not None or gate is not None else None,
                              h if pre is not None else None, post_gamma, post_beta, gate, pre_gamma, pre_beta,
                              *stats)
        ctx.set_materialize_grads(False)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        if dh is None and dy is None:
            return (None,) * 12
        f, h, post_gamma, post_beta, gate, pre_gamma, pre_beta, *stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        some = dy if dy is not None else dh
        dh = None if dh is None else dh.contiguous()
        dy = None if dy is None else dy.contiguous()
        df, dx = torch.empty_like(some, memory_format=torch.contiguous_format), \
            torch.empty_like(some, memory_format=torch.contiguous_format)
        new = lambda t, n: torch.empty(t.shape, dtype=t.dtype, device=t.device) \
            if t is not None and need[n] else None  # noqa: E731
        dpg, dpb, dg, dng, dnb = (new(t, n + 2) for n, t in
                                  enumerate((post_gamma, post_beta, gate, pre_gamma, pre_beta)))
        block_norm_bwd(dy, dh, f, h, stats, df, dx, post_gamma=post_gamma, post_beta=post_beta, gate=gate,
                       pre_gamma=pre_gamma, dpost_gamma=dpg, dpost_beta=dpb, dgate=dg, dpre_gamma=dng,
                       dpre_beta=dnb, **ctx.kinds)
        return (df if need[0] else None, dx if need[1] else None, dpg, dpb, dg, dng, dnb) + (None,) * 5


def block_norm_train(f, x, *, post=None, post_gamma=None, post_beta=None, gate=None, pre="rms",
                     pre_gamma=None, pre_beta=None, residual_scale: float = 1.0, block_scale: float = 1.0,
                     eps: float = 1e-5):
    """(h, y or None) of the block boundary, with gradients for every tensor
    argument (first order only)."""
    return BlockNormFunction.apply(f, x, post_gamma, post_beta, gate, pre_gamma, pre_beta, post, pre,
                                   residual_scale, block_scale, eps)


class FusedBlockNorm(torch.nn.Module):
    """The block boundary as a module: learnable fp32 parameters of size
    `hidden` (norms: gamma ones, and beta zeros with bias; layer_scale: a
    per-channel gate that starts at this value).  A gate with rows is passed
    to forward instead.  Returns (h, y).  The parameters are fp32 whatever the
    activations (moved to a 16-bit type, they are refused)."""

    def __init__(self, hidden: int, post: Optional[str] = "rms", pre: Optional[str] = "rms",
                 bias: bool = False, layer_scale: Optional[float] = None, residual_scale: float = 1.0,
                 block_scale: float = 1.0, eps: float = 1e-5, device=None):
        super().__init__()
        _norm_kind(post, "post"), _norm_kind(pre, "pre")
        self.post, self.pre, self.eps = post, pre, float(eps)
        self.residual_scale, self.block_scale = float(residual_scale), float(block_scale)
        new = lambda v, w: torch.nn.Parameter(  # noqa: E731
            torch.full((hidden,), float(v), dtype=torch.float32, device=device)) if w else None
        self.post_weight = new(1, post is not None)
        self.post_bias = new(0, post is not None and bias)
        self.pre_weight = new(1, pre is not None)
        self.pre_bias = new(0, pre is not None and bias)
        self.layer_scale = new(layer_scale or 0.0, layer_scale is not None)

    def forward(self, f, x, gate=None):
        if gate is not None and self.layer_scale is not None:
            raise ValueError("a gate beside the module's own layer_scale")
        return block_norm_train(f, x, post=self.post, post_gamma=self.post_weight, post_beta=self.post_bias,
                                gate=self.layer_scale if gate is None else gate, pre=self.pre,
                                pre_gamma=self.pre_weight, pre_beta=self.pre_bias,
                                residual_scale=self.residual_scale, block_scale=self.block_scale, eps=self.eps)
