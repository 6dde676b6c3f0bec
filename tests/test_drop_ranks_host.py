"""FusedDropoutAddNorm in data-parallel training, as two gloo processes without a GPU."""
from __future__ import annotations

import os
import socket
import sys

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _worker(rank, world, port, q):
    sys.path.insert(0, ROOT)
    import memory_bound_add_gb300 as mba
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=world)
    try:
        torch.manual_seed(rank)
        m = mba.FusedDropoutAddNorm(8, p=0.5, input_bias=True)
        m.weight.data.fill_(rank + 1.0)
        before = m.rng.tolist()
        d = torch.nn.parallel.DistributedDataParallel(m)
        x = torch.zeros(2, 8)
        try:
            d(x, x)  # (what is broadcast before a forward is; then it wants a GPU)
        except ValueError as e:
            assert "CUDA" in str(e)
        q.put((rank, before, m.rng.tolist(), m.weight[0].item()))
    finally:
        dist.destroy_process_group()


def test_ranks_keep_their_seeds():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    ps = [ctx.Process(target=_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in ps:
        p.start()
    got = sorted(q.get(timeout=120) for _ in range(2))
    for p in ps:
        p.join(60)
        assert p.exitcode == 0
    for _, before, after, weight in got:
        assert after == before and weight == 1.0  # parameters are rank 0's
    assert got[0][2] != got[1][2]


def test_the_pair_moves_and_is_saved_with_the_module():
    import memory_bound_add_gb300 as mba
    m = torch.nn.Sequential(mba.FusedDropoutAddNorm(8, p=0.5), mba.FusedDropoutAddNorm(8, p=0.5, norm=None))
    state = m.state_dict()
    assert set(state) == {"0.weight", "0.bias", "0.rng", "1.rng"} and state["0.rng"].data_ptr() == m[0].rng.data_ptr()
    m[0].rng[1] = 7
    other = torch.nn.Sequential(mba.FusedDropoutAddNorm(8, p=0.5), mba.FusedDropoutAddNorm(8, p=0.5, norm=None))
    kept = other[0].rng
    assert str(other.load_state_dict(state)) == "<All keys matched successfully>"
    assert other[0].rng is kept and all(torch.equal(a.rng, b.rng) for a, b in zip(m, other))
    assert int(other[0].rng[1]) == 7
    # strict loading misses it and finds what is not its own, as any entry
    with pytest.raises(RuntimeError, match=r"Missing.*1\.rng"):
        other.load_state_dict({k: v for k, v in state.items() if k != "1.rng"})
    with pytest.raises(RuntimeError, match=r"Unexpected.*0\.seed"):
        other.load_state_dict({**state, "0.seed": state["0.rng"]})
    with pytest.raises(RuntimeError, match=r"size mismatch.*0\.rng"):
        other.load_state_dict({**state, "0.rng": torch.zeros(3, dtype=torch.int64)})
    assert "1.rng" in other.load_state_dict({"0.weight": state["0.weight"]}, strict=False).missing_keys
    given = {k: v.clone() for k, v in state.items()}
    other.load_state_dict(given, assign=True)
    assert other[0].rng is given["0.rng"]
    # it goes where the module goes, and stays whole numbers
    assert m.to("meta")[0].rng.is_meta
    assert other.double()[0].rng.dtype is torch.int64 and other[0].weight.dtype is torch.float64
    m.load_state_dict(given, assign=True)
    assert m[0].rng.tolist() == given["0.rng"].tolist()


def test_a_module_pickled_with_a_buffer():
    import pickle

    import memory_bound_add_gb300 as mba
    m = mba.FusedDropoutAddNorm(8, p=0.5)
    c = pickle.loads(pickle.dumps(m))
    assert torch.equal(c.rng, m.rng) and not list(c.buffers())
    m.register_buffer("rng", m.__dict__.pop("rng"))
    c = pickle.loads(pickle.dumps(m))
    assert torch.equal(c.rng, m.rng) and not list(c.buffers()) and set(c.state_dict()) == {"weight", "bias", "rng"}
