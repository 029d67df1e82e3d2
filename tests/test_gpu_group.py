"""ace_moe_group against a sort: every result is a whole number or a copy, so
all are equal."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu


def _check(idx, E, keep=None, gate=None):
    from token_dynamic_expert_b200 import ace
    T, k = idx.shape
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    so = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    st = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    sg = torch.full((T * k,), -7.0, device="cuda") if gate is not None else None
    ace.ace_moe_group(idx, E, off, so, keep=keep, gate=gate, slot_token=st, slot_gate=sg)
    torch.cuda.synchronize()
    roff, rso, slots = ora.group(idx.cpu().numpy(), None if keep is None else keep.cpu().numpy(), E)
    assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(so.cpu().numpy(), rso)
    n = len(slots)
    assert np.array_equal(st.cpu().numpy()[:n], slots // k) and (st[n:] == -7).all()
    if gate is not None:
        assert np.array_equal(sg.cpu().numpy()[:n], gate.cpu().numpy().reshape(-1)[slots])
        assert (sg[n:] == -7).all()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 5), (32, 8, 64), (255, 8, 256), (256, 8, 256),
                                   (257, 8, 256), (1003, 7, 128), (8192, 8, 512), (20000, 16, 300), (4000, 3, 1)])
@pytest.mark.parametrize("skip", [0.0, 0.6, 1.0])
def test_sizes(T, k, E, skip):
    g = torch.Generator(device="cuda").manual_seed(T + k + E)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    keep = (torch.rand(T, k, generator=g, device="cuda") >= skip).to(torch.uint8) if skip else None
    _check(idx, E, keep, torch.rand(T, k, generator=g, device="cuda"))


def test_one_expert_takes_all_and_some_take_none():
    _check(torch.full((3000, 4), 6, dtype=torch.int32, device="cuda"), 9)


def test_indices_outside_count_as_skipped():
    idx = torch.randint(-3, 13, (2000, 4), device="cuda", dtype=torch.int32)
    _check(idx, 10, None, torch.rand(2000, 4, device="cuda"))


def test_no_tokens():
    from token_dynamic_expert_b200 import ace
    off = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    ace.ace_moe_group(torch.empty(0, 3, dtype=torch.int32, device="cuda"), 4, off,
                      torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert off.tolist() == [0] * 5


def test_graph_replay_with_other_inputs():
    from token_dynamic_expert_b200 import ace
    idx = torch.randint(0, 32, (900, 4), device="cuda", dtype=torch.int32)
    off, so = torch.empty(33, dtype=torch.int32, device="cuda"), torch.empty(900, 4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ace.ace_moe_group(idx, 32, off, so)
    for seed in range(3):
        idx.copy_(torch.randint(0, 32, (900, 4), device="cuda", dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        roff, rso, _ = ora.group(idx.cpu().numpy(), None, 32)
        assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(so.cpu().numpy(), rso)
