"""The dropout and 8-bit kernels through the bounds-checked debugging build:
every kernel shape (a warp, a CTA, a cluster a row; rows on borders, beside them
the same way, and anywhere), with values against 64 bits.  In that build an
access that would leave its buffer is skipped and reported."""
from __future__ import annotations

import ctypes

import pytest
import torch

import test_gpu_drop as td
import test_gpu_quant as tq
from test_gpu_block import at_offset

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")
from memory_bound_add_gb300 import drop, quant  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])


@pytest.fixture
def chk(monkeypatch):
    """The checked library in the wrappers' place; no violation at the end."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_add_gb300.build import CHECKED_LIB, build
    build()
    build(checked=True)
    lib = mba.binding.load(CHECKED_LIB)
    assert lib.addln_bounds_checked() == 1
    for m in (drop, quant):
        monkeypatch.setattr(m, "_lib", m.bind(lib))
        monkeypatch.setattr(m, "_fast", None)
    drop._workspace_size.cache_clear()  # its grids follow this build's occupancy
    yield lib
    drop._workspace_size.cache_clear()
    torch.cuda.synchronize()
    rc = lib.addln_get_device_error(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, f"{lib.addln_strerror(rc).decode()} (word {lib.addln_bounds_violation():#x})"


@DTYPES
@pytest.mark.parametrize("H", [1, 7, 8, 250, 264, 768, 1001, 4096, 4104, 5001, 8192, 16384])
def test_boundary(chk, dtype, H):
    for j, (norm, bias, beta) in enumerate([("layer", True, True), ("rms", False, False), (None, True, False)]):
        v = td.make((5, H), dtype, norm, bias, beta, seed=H)
        td.check_fwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}", with_x=j != 2, as_tensor=j == 0)
        td.check_bwd(v, 0.3, (3, 4), norm, what=f"{H} {norm}", as_tensor=j == 1)


@pytest.mark.parametrize("rows,H,dtype", [(1200, 64, F32), (700, 40, F16), (1000, 1001, BF16), (640, 4104, F16),
                                          (4097, 257, BF16)])
def test_many_rows(chk, rows, H, dtype):
    for norm, bias, beta in (("layer", True, True), ("rms", False, False)):
        v = td.make((rows, H), dtype, norm, bias, beta, seed=rows)
        td.check_fwd(v, 0.1, (11, 12), norm)
        if rows < 2000:  # the bounds of the column sums
            td.check_bwd(v, 0.1, (11, 12), norm)


@DTYPES
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 0)])
def test_dropout(chk, dtype, a, b):
    for n in (1, 9, 8191, 100003):
        x = td.randn((n,), dtype, n)
        y = at_offset(torch.zeros(n, dtype=dtype), b)[0]
        mba.dropout_fwd(at_offset(x, a)[0], y, 0.25, (1, 2))
        td.check_drop(x, 0.25, (1, 2), y)
    x = td.randn((1 << 20,), dtype, 1).cuda().repeat(6)  # four blocks a thread
    y = mba.dropout(x, 0.5, torch.tensor([5, 6], device="cuda"))
    td.check_drop(x[:4096].cpu(), 0.5, (5, 6), y[:4096])


@DTYPES
@pytest.mark.parametrize("H", [5, 520, 4099])
def test_boundary_off_the_borders(chk, dtype, H):
    td.test_off_the_borders_and_given_outputs(dtype, H)


@DTYPES
@pytest.mark.parametrize("H", [1, 7, 8, 31, 33, 250, 264, 768, 1001, 4096, 4104, 5001, 8192, 16384])
def test_quant(chk, dtype, H):
    for j, (scaling, group) in enumerate(tq.SCALINGS):
        norm, beta = tq.KINDS[j % len(tq.KINDS)]
        v = tq.make((5, H), dtype, norm, beta, residual=j != 1, seed=H)
        tq.check_fwd(v, norm, ["e4m3", "e5m2", "int8"][j % 3], scaling, group, major=j % 2 == 1, what=f"{H} {scaling} {group}")
    tq.check_fwd(v, norm, "int8", "tensor", given=0.02)


@DTYPES
@pytest.mark.parametrize("H", [5, 520, 4099])
@pytest.mark.parametrize("scaling,group", [("row", None), ("group", 64), ("pow2", 32)])
def test_quant_off_the_borders(chk, dtype, H, scaling, group):
    tq.test_off_the_borders(dtype, H, scaling, group)


@pytest.mark.parametrize("rows,H,dtype", [(1200, 64, F32), (4097, 257, BF16), (3000, 1001, F16), (640, 4104, BF16)])
def test_quant_many_rows(chk, rows, H, dtype):
    for scaling, group in (("row", None), ("group", 32)):
        v = tq.make((rows, H), dtype, "rms", seed=rows)
        tq.check_fwd(v, "rms", "e4m3", scaling, group)
