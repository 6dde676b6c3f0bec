"""The block boundary and the gradient kernels through the bounds-checked
debugging build: every kernel shape (a warp, a CTA, a cluster a row; 16-byte
and shifted rows; each kind of gate), with values against 64 bits.  In that
build an access that would leave its buffer is skipped and reported."""
from __future__ import annotations

import ctypes

import pytest
import torch

from _block_ref import assert_within, backward, forward
from test_gpu_block import at_offset, check_bwd, check_fwd, cuda, make
from test_gpu_grads import check as check_clip, draw

pytestmark = pytest.mark.gpu
mba = pytest.importorskip("memory_bound_add_gb300")
from memory_bound_add_gb300 import block, grads  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


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
    monkeypatch.setattr(block, "_lib", block.bind(lib))
    monkeypatch.setattr(grads, "_lib", grads.bind(lib))
    block._workspace_size.cache_clear()  # its grids follow this build's occupancy
    yield lib
    block._workspace_size.cache_clear()
    torch.cuda.synchronize()
    rc = lib.addln_get_device_error(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, f"{lib.addln_strerror(rc).decode()} (word {lib.addln_bounds_violation():#x})"


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("H", [1, 7, 8, 250, 264, 768, 1001, 4096, 4104, 5001, 8192, 16384])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer")])
def test_block(chk, dtype, H, post, pre):
    rows = 5
    for gate in (None, "channel", (rows, H), (1, H)):
        f, x, p = make((rows, H), dtype, post, pre, gate, beta=post == "layer", seed=H)
        check_fwd(f, x, p, post, pre, what=f"{H} gate {gate}")
        check_bwd(f, x, p, post, pre, what=f"{H} gate {gate}")


@pytest.mark.parametrize("B,S,H,dtype", [(300, 2, 96, BF16), (7, 100, 40, F16), (3, 333, 200, BF16),
                                         (2, 500, 1001, F16), (1, 5000, 16, F32)])
def test_gate_rows(chk, B, S, H, dtype):
    f, x, p = make((B, S, H), dtype, "rms", "layer", (B, 1, H), seed=B)
    check_fwd(f, x, p, "rms", "layer", what=f"{B}x{S}x{H}")
    check_bwd(f, x, p, "rms", "layer", what=f"{B}x{S}x{H}")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("H", [5, 520, 4099])
def test_off_the_borders(chk, dtype, H):
    # each tensor by a distance of its own, the gate a strided part
    f, x, p = make((6, H), dtype, "rms", "rms", None, seed=H)
    wide = torch.randn(6, 3 * H, generator=torch.Generator().manual_seed(1)).to(dtype)
    q = dict(p, gate=wide[:, H:2 * H])
    dq = dict(cuda(p), gate=wide.cuda()[:, H:2 * H])
    wh, wy, wst, eh, ey = forward(f, x, q, "rms", "rms", 1.0, 1.0, 1e-5)
    fc = at_offset(f, 1)[0]
    h, y = at_offset(f, 3)[0], at_offset(f, 4)[0]
    mba.block_norm_fwd(fc, at_offset(x, 2)[0], h, y, post="rms", pre="rms", **dq)
    assert_within(h, wh, eh, "h")
    assert_within(y, wy, ey, "y")
    dy = torch.randn(6, H, generator=torch.Generator().manual_seed(2)).to(dtype)
    hs, st = wh.to(dtype), [None if t is None else t.reshape(-1).float() for t in wst]
    want, err = backward(dy, None, f, hs, st, q, "rms", "rms", 1.0, 1.0)
    got = {k: at_offset(f, 5 + i)[0] for i, k in enumerate(("df", "dx", "dgate"))}
    mba.block_norm_bwd(at_offset(dy, 9)[0], None, fc, at_offset(hs, 10)[0],
                       tuple(None if t is None else t.cuda() for t in st), got["df"], got["dx"], post="rms", pre="rms",
                       dgate=got["dgate"], **dq)
    for k, v in got.items():
        assert_within(v, want[k].reshape(v.shape), err[k].reshape(v.shape), k)


@pytest.mark.parametrize("dtype", [F32, F16, BF16, "mixed"], ids=["fp32", "fp16", "bf16", "mixed"])
def test_clip(chk, dtype):
    for sizes in ([1], [255, 0, 9], [2047, 2048, 2049, 4096, 4097], [100000, 3, 65537, 0, 12, 1 << 20]):
        gs = draw(sizes, dtype, seed=len(sizes))
        for off in (0, 1):
            mine = [at_offset(g, off)[0] for g in gs]
            outs = [torch.empty_like(g, dtype=F32) for g in gs]
            norm = mba.clip_grads(mine, 0.5, out=outs)
            torch.cuda.synchronize()
            check_clip(gs, outs, norm, 0.5)
            norm = mba.clip_grads(mine, 0.5, scale=0.5)
            torch.cuda.synchronize()
            check_clip(gs, mine, norm, 0.5, 0.5)
            assert float(mba.grad_norm(gs)) > 0
