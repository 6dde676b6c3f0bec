"""Global gradient norm and clipping over many tensors.

Binding of ``include/addln_grad.h`` (argument marshalling only, like
``binding``):

    norm   = scale * sqrt(sum of all g^2)
    factor = scale * min(1, max_norm / (norm + 1e-6))
    out    = g * factor

as two kernels over all tensors, without waiting for the GPU.  Tensors are
CUDA tensors of one device, fp32, fp16 or bf16 (mixed freely), whose elements
fill their memory without gaps or repeats, in any order of dimensions.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import binding
from .binding import DTYPE_CODE
from .block import _check, changed, on_stream

# Every symbol include/addln_grad.h declares, with its ctypes signature.
_P, _I64, _F, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
SIGNATURES = {
    "grad_norm": (_I, [_P, _P, _P, _I64, _F, _P, _P, _I64, _P]),
    "grad_clip": (_I, [_P, _P, _P, _P, _P, _I64, _F, _F, _P, _P]),
    "grad_norm_clip": (_I, [_P, _P, _P, _P, _P, _I64, _F, _F, _P, _P, _I64, _P]),
    "grad_norm_workspace_size": (_I64, [_I64]),
}

_lib = None
_Tensor = torch.Tensor


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


def grad_norm_workspace_size(count: int) -> int:
    n = int(lib().grad_norm_workspace_size(int(count)))
    if n < 0:
        raise binding.AddLNError(n, "grad_norm_workspace_size")
    return n


# a number that the count alone decides
_workspace_size = functools.lru_cache(maxsize=256)(grad_norm_workspace_size)


def _dense(t) -> bool:
    """Whether t's elements fill their memory without gaps or repeats."""
    want = 1
    for n, st in sorted(((n, st) for n, st in zip(t.shape, t.stride()) if n != 1), key=lambda p: p[1]):
        if st != want:
            return False
        want *= n
    return True


def _lists(ts, name):
    """(pointers, sizes, dtypes) as ctypes arrays, and the device's index."""
    try:
        devices = set(map(_Tensor.get_device, ts))
    except TypeError:
        raise TypeError(f"{name} must hold torch.Tensors alone") from None
    if len(devices) != 1 or -1 in devices:
        raise ValueError(f"{name} must be CUDA tensors of one device")
    if not all(map(_Tensor.is_contiguous, ts)):
        for i, t in enumerate(ts):
            if t.numel() and not _dense(t):
                raise ValueError(f"{name}[{i}] has gaps or repeated elements; make it contiguous")
    n = len(ts)
    try:
        codes = [DTYPE_CODE[t.dtype] for t in ts]
    except KeyError as e:
        raise ValueError(f"unsupported dtype {e.args[0]} in {name}") from None
    return ((_P * n)(*map(_Tensor.data_ptr, ts)), (_I64 * n)(*map(_Tensor.numel, ts)), (_I * n)(*codes),
            devices.pop())


def _norm_tensor(norm, device):
    if not isinstance(norm, _Tensor) or norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != device:
        raise ValueError(f"norm must be one fp32 element on {device}")
    return norm.data_ptr()


def grad_norm(grads, scale: float = 1.0, stream=None):
    """scale * sqrt(sum of squares over all tensors), as a 0-dimensional fp32
    CUDA tensor (a CPU zero for an empty list).  The GPU is not waited for."""
    grads = list(grads)
    if not grads:
        return torch.zeros(())
    p, n, d, index = _lists(grads, "grads")
    device, count = torch.device("cuda", index), len(grads)
    out = []

    def call(s):
        norm = torch.empty((), dtype=torch.float32, device=device)
        size = _workspace_size(count)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        out.append(norm)
        return lib().grad_norm(p, n, d, count, scale, norm.data_ptr(), ws.data_ptr(), size, s)

    _check(on_stream(device, stream, call), "grad_norm")
    return out[0]


def clip_grads(grads, max_norm: float, out=None, scale: float = 1.0, norm=None, stream=None):
    """Scales the gradients so that their norm is at most max_norm, and
    returns that norm as it was (after `scale`), without waiting for the GPU.

    out: one tensor for each gradient, of its shape and strides, fp32 or the
    gradient's dtype (None: in place).  scale: 1 / loss scale.  norm: the norm
    where it is on the device already (one fp32 element, e.g. joined over
    several GPUs); otherwise it is computed here.  max_norm may be infinite:
    no limit, the factor is `scale` even where the norm is infinite too.
    """
    grads = list(grads)
    if not grads:
        if out is not None and len(list(out)):
            raise ValueError("out has tensors, grads has none")
        return torch.zeros(()) if norm is None else norm
    p, n, d, index = _lists(grads, "grads")
    device, count = torch.device("cuda", index), len(grads)
    op = od = None
    written = grads
    if out is not None:
        written = list(out)
        if len(written) != count:
            raise ValueError(f"out has {len(written)} tensors, grads has {count}")
        op, _, od, oindex = _lists(written, "out")
        if oindex != index:
            raise ValueError("out is on another device than grads")
        for i, (g, o) in enumerate(zip(grads, written)):
            if g.shape != o.shape or g.stride() != o.stride():
                if g.shape != o.shape or not (g.is_contiguous() and o.is_contiguous()):
                    raise ValueError(f"out[{i}] must have the gradient's shape and strides")
    ret = []

    def call(s):
        if norm is not None:
            ret.append(norm)
            return lib().grad_clip(p, op, n, d, od, count, scale, max_norm, _norm_tensor(norm, device), s)
        ret.append(torch.empty((), dtype=torch.float32, device=device))
        size = _workspace_size(count)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        return lib().grad_norm_clip(p, op, n, d, od, count, scale, max_norm, ret[0].data_ptr(), ws.data_ptr(), size,
                                    s)

    _check(on_stream(device, stream, call), "clip_grads")
    changed(written)
    return ret[0]


def clip_grad_norm_(parameters, max_norm: float, scale: float = 1.0, stream=None):
    """clip_grads in place on the .grad of every parameter that has one."""
    if isinstance(parameters, _Tensor):
        parameters = [parameters]
    return clip_grads([p.grad for p in parameters if p.grad is not None], max_norm, scale=scale, stream=stream)
