"""Calls of one LayerI8 that share its buffers: from several streams and threads, none
of which waits for another by itself."""
import threading

import pytest
import torch

import i8_oracle as ora
from test_gpu_layer_i8 import GATES, _make

pytestmark = pytest.mark.gpu


def _inputs(T, d, n):
    g = torch.Generator(device="cuda").manual_seed(n + T)
    return [torch.randn(T - i, d, generator=g, device="cuda").bfloat16() for i in range(n)]


@pytest.mark.parametrize("T", [8, 700])
def test_calls_on_several_streams_keep_their_results(T):
    L, _, _ = _make(T, 512, 32, 256, 4, gate=GATES[1], bias=True)
    us = _inputs(T, 512, 4)
    want = [L.forward(u, torch.empty_like(u)) for u in us]
    got = [torch.zeros_like(u) for u in us]
    streams = [torch.cuda.Stream() for _ in us]
    torch.cuda.synchronize()
    for _ in range(20):
        for u, y, s in zip(us, got, streams):
            L.forward(u, y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert L.status()[0] == 0


def test_calls_from_several_threads_keep_their_results():
    L, _, _ = _make(300, 512, 32, 256, 4)
    us = _inputs(300, 512, 4)
    want = [L.forward(u, torch.empty_like(u)) for u in us]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(us))

    def work(u, w):
        s, ys = torch.cuda.Stream(), [torch.zeros_like(u) for _ in range(30)]
        torch.cuda.current_stream().synchronize()  # ys are zeros before s writes them
        start.wait()
        for y in ys:
            L.forward(u, y, stream=s)
        s.synchronize()
        bad.extend(i for i, y in enumerate(ys) if not torch.equal(y, w))

    threads = [threading.Thread(target=work, args=a) for a in zip(us, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_status_waits_for_a_call_on_another_stream():
    """The status words of a call that is still running are not read too early: a bad
    expert index cannot arise here, so the call before leaves a flag in them."""
    from token_dynamic_expert_b200 import ace
    L, u, _ = _make(700, 512, 32, 256, 4)
    s, y = torch.cuda.Stream(), torch.empty_like(u)
    for w in L.ws:
        w.view(torch.int32)[0] = ace.ACE_FLAG_BAD_INDEX
    torch.cuda.synchronize()
    for _ in range(10):
        L.forward(u, y, stream=s)
    assert L.status() == (ace.ACE_OK, 0)


def test_a_captured_call_between_others():
    L, _, _ = _make(96, 512, 32, 256, 4)
    us = _inputs(96, 512, 2)
    want = [L.forward(u, torch.empty_like(u)) for u in us]
    y, z = torch.zeros_like(us[0]), torch.zeros_like(us[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(us[0], y)
    for _ in range(3):
        g.replay()
        L.forward(us[1], z)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(z, want[1])


def test_an_input_on_another_device_is_refused():
    L, u, _ = _make(8, 128, 8, 64, 2)
    with pytest.raises(ValueError, match="device"):
        L.forward(u.cpu(), torch.empty(u.shape, dtype=u.dtype))


def test_rows_that_start_anywhere():
    """u and residual off 16-byte boundaries give the bits of aligned ones; y may be
    either of them; a y or sum of that kind, or one in the other, is refused before
    the first kernel."""
    L, u, res = _make(24, 256, 8, 64, 2)
    n = u.numel()

    def off(t, by):
        b = torch.zeros(n + 64, dtype=t.dtype, device="cuda")
        v = b[by:by + n].view(t.shape)
        return v.copy_(t)

    for by in (1, 2, 8):
        want, got = torch.empty_like(u), torch.empty_like(u)
        L.forward(u, want)
        L.forward(off(u, by), got)
        assert torch.equal(want, got)
        L.forward(u, want, res)
        L.forward(off(u, by), got, off(res, by + 1))
        assert torch.equal(want, got)
    for into in (0, 1):
        a, b = u.clone(), res.clone()
        L.forward(a, (a, b)[into], b)
        assert torch.equal((a, b)[into], want)
    both = torch.zeros(2 * n, dtype=u.dtype, device="cuda")
    kept = res.clone()
    for y, s in ((off(u, 1), None), (torch.empty_like(u), off(res, 1)), (both[8:8 + n].view(u.shape), both[:n].view(u.shape)),
                 (res, res)):
        with pytest.raises(ValueError, match="16-byte|overlap"):
            L.forward(u, y, res, sum=s)
    with pytest.raises(TypeError):
        L.forward(u, torch.empty_like(u), res, sum=res, tau=None)
    with pytest.raises(ValueError, match="must be"):
        L.forward(u[0], torch.empty_like(u[0]), res, sum=res)
    torch.cuda.synchronize()
    assert torch.equal(res, kept) and not both.any()
    y = torch.empty_like(u)
    L.forward(u, both[n:].view(u.shape), res, sum=both[:n].view(u.shape))  # neighbours
    assert torch.equal(both[n:].view(u.shape), want)


@pytest.mark.parametrize("T", [1, 8, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router_bias_is_part_of_the_logits(T, dtype):
    from token_dynamic_expert_b200 import layer_i8
    L, u, _ = _make(T, 256, 32, 64, 4, dtype=dtype)
    b = torch.randn(32, device="cuda")
    B = layer_i8.LayerI8(L.gamma, L.w_router, L.wq_gu, L.s_gu, L.wq_down, L.s_down, 4, T, router_bias=b)
    y = torch.empty_like(u)
    L.forward(u, y)
    B.forward(u, y)
    assert torch.equal(B.logits, L.logits + b)  # the sum of the products, then one addition
    idx, w = ora.gate(ora.f64(B.logits), 4)
    assert (B.idx.view(T, 4).cpu().numpy() == idx).all()
    spread = float(B.logits.max() - B.logits.min())
    assert ora.close(ora.f64(B.weight.view(T, 4)), w, (2 * spread + 20) * ora.U32, 1e-37) <= 1


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_a_layer_on_another_device_than_the_current_one():
    from token_dynamic_expert_b200 import layer_i8
    for T in (8, 96):
        L, u, _ = _make(T, 256, 16, 64, 4)
        want = L.forward(u, torch.empty_like(u))
        M = layer_i8.LayerI8(*(t.to("cuda:1") for t in (L.gamma, L.w_router, L.wq_gu, L.s_gu, L.wq_down, L.s_down)), 4, T)
        v = u.to("cuda:1")
        got = M.forward(v, torch.empty_like(v))
        assert M.status()[0] == 0 and torch.equal(got.cpu(), want.cpu())
