"""The 8-bit layer: the operators one after the other, as a program runs them.

Every stage's buffer is compared with 64-bit numpy on the buffer ahead of it,
with that operator's own tolerance (see its tests), so that a rounding does not
carry over; and the whole with the layer in 64 bits on the dequantised weights."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu


def _make(T, d, E, m, k, seed=0, gate=None, bias=False, factor=False, dtype=torch.bfloat16):
    from token_dynamic_expert_b200 import layer_i8
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, s=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * s

    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    wr = n(E, d, s=0.05).to(dtype)
    gu, sgu = layer_i8.quantise_rows(n(E, 2 * m, d, s=0.02))
    dn, sdn = layer_i8.quantise_rows(n(E, d, m, s=0.02))
    L = layer_i8.LayerI8(gamma, wr, gu, sgu, dn, sdn, k, T, bias=n(E, s=0.1) if bias else None,
                         factor=torch.rand(E, generator=g, device="cuda") + 0.5 if factor else None, gate=gate)
    return L, n(T, d).to(dtype), n(T, d).to(dtype)


def _stages(L, u, res, y, tau):
    """Checks every buffer of the last call against the one ahead of it."""
    T, k, E = u.shape[0], L.k, L.E
    dt = "bf16" if u.dtype == torch.bfloat16 else "f32"
    s = u if res is None else (u.float() + res.float()).to(u.dtype)
    _, q, scale = ora.norm(ora.f64(s), ora.f64(L.gamma), L.eps)
    assert np.array_equal(L.xq[:T].cpu().numpy(), q)
    assert ora.close(ora.f64(L.xs[:T]), scale, 24 * ora.U32) <= 1
    logits = ora.f64(L.logits[:T])
    xn = ora.f64(s) / np.sqrt((ora.f64(s) ** 2).mean(1, keepdims=True) + L.eps) * ora.f64(L.gamma)
    wr = ora.f64(L.w_router)
    # products of d terms summed in fp32, and a weight split into three bf16 terms
    assert (np.abs(logits - xn @ wr.T) <= (L.d + 32) * ora.U32 * (np.abs(xn) @ np.abs(wr).T)).all()
    idx, w = ora.gate(logits, k, None if L.bias is None else ora.f64(L.bias), **L.gate)
    assert np.array_equal(L.idx[:T * k].view(T, k).cpu().numpy(), idx)
    got_w = ora.f64(L.weight[:T * k].view(T, k))
    assert ora.close(got_w, w, (2 * (logits.max() - logits.min()) + 20) * ora.U32, 1e-37) <= 1
    keep = L.keep[:T * k].view(T, k).cpu().numpy()
    c = got_w * (1 if L.factor is None else ora.f64(L.factor)[idx])
    want = ~(c < tau)
    want[np.arange(T), got_w.argmax(1)] = True
    sure = np.abs(c - tau) > 4 * ora.U32 * np.abs(c)   # a product of fp32 on the border may fall either way
    assert np.array_equal(keep[sure] != 0, want[sure])
    off, slot_of, slots = ora.group(idx, keep, E)
    S = len(slots)
    assert np.array_equal(L.offsets.cpu().numpy(), off)
    assert np.array_equal(L.slot_of[:T * k].view(T, k).cpu().numpy(), slot_of)
    tok = L.slot_token[:S].cpu().numpy()
    assert np.array_equal(tok, slots // k)
    gu = ora.matmul(q, ora.f64(L.xs[:T]), ora.f64(L.wq_gu), ora.f64(L.s_gu), off, row_of=tok)
    assert ora.close(ora.f64(L.gu[:S]), gu, ora.HALF[dt] + 4 * ora.U32) <= 1
    _, hq, hs = ora.swiglu(ora.f64(L.gu[:S]))
    assert np.array_equal(L.hq[:S].cpu().numpy(), hq)
    assert ora.close(ora.f64(L.hs[:S]), hs, 13 * ora.U32) <= 1
    ys = ora.matmul(hq, ora.f64(L.hs[:S]), ora.f64(L.wq_down), ora.f64(L.s_down), off,
                    slot_scale=got_w.reshape(-1)[slots])
    got = ora.f64(L.yslot[:S])
    assert ora.close(got, ys, ora.HALF[dt] + 4 * ora.U32) <= 1
    ref, mag = np.zeros((T, L.d)), np.zeros((T, L.d))
    np.add.at(ref, tok, got)
    np.add.at(mag, tok, np.abs(got))
    # k fp32 additions and one rounding
    assert (np.abs(ora.f64(y) - ref) <= ora.HALF[dt] * np.abs(ref) + k * ora.U32 * mag + 1e-37).all()
    return ref


GATES = [dict(), dict(score="sigmoid", n_groups=4, topk_groups=2, group_score="top2", scale=2.5),
         dict(score="sigmoid", renorm=False), dict(n_groups=8, topk_groups=3)]


@pytest.mark.parametrize("T,d,E,m,k", [(1, 128, 8, 64, 2), (8, 512, 32, 128, 8), (61, 256, 16, 112, 4),
                                       (700, 384, 64, 96, 6)])
@pytest.mark.parametrize("gate", range(len(GATES)))
@pytest.mark.parametrize("residual,tau", [(False, 0.0), (True, 0.12)])
def test_every_stage(T, d, E, m, k, gate, residual, tau):
    L, u, res = _make(T, d, E, m, k, seed=T, gate=GATES[gate], bias=gate % 2 == 1, factor=tau > 0)
    res = res if residual else None
    y = torch.full_like(u, 7)
    s = torch.empty_like(u) if residual else None
    L.forward(u, y, residual=res, sum=s, tau=tau)
    from token_dynamic_expert_b200 import ace
    assert L.status() == (ace.ACE_OK, 0)
    if residual:
        assert torch.equal(s, (u.float() + res.float()).to(u.dtype))
    _stages(L, u, res, y, tau)


def test_fp32_activations():
    L, u, _ = _make(33, 128, 8, 48, 3, dtype=torch.float32)
    y = torch.empty_like(u)
    L.forward(u, y)
    _stages(L, u, None, y, 0.0)


def test_close_to_the_layer_in_64_bits():
    """8 bits hold a row to half a step of max / 127: relative to its root mean
    square an error of (max / rms) / (127 sqrt 12), 0.9% for normal rows (max / rms
    about 4) and 1.8% for h (a product, about 8).  The products carry x's to both
    halves of h and on to y, beside h's own: sqrt(2 x 0.9^2 + 1.8^2) = 2.2%; below
    4% for the matrix as a whole."""
    T, d, E, m, k = 300, 512, 16, 256, 4
    L, u, _ = _make(T, d, E, m, k, seed=9)
    y = torch.empty_like(u)
    L.forward(u, y)
    x = ora.f64(u)
    x = x / np.sqrt((x * x).mean(1, keepdims=True) + L.eps) * ora.f64(L.gamma)
    gu = ora.f64(L.wq_gu) * ora.f64(L.s_gu)[..., None]
    dn = ora.f64(L.wq_down) * ora.f64(L.s_down)[..., None]
    idx, w = ora.gate(ora.f64(L.logits), k)
    ref = np.zeros((T, d))
    for t in range(T):
        for i in range(k):
            p = gu[idx[t, i]] @ x[t]
            ref[t] += w[t, i] * (dn[idx[t, i]] @ (p[:m] / (1 + np.exp(-p[:m])) * p[m:]))
    assert np.linalg.norm(ora.f64(y) - ref) < 0.04 * np.linalg.norm(ref)


def test_fewer_tokens_in_place_sum_and_nothing_behind():
    L, u, res = _make(64, 256, 16, 64, 4)
    for T in (0, 1, 7, 64):
        s, r = u.clone(), res.clone()
        y = torch.full_like(u, 7)
        L.gu.fill_(3), L.yslot.fill_(3)
        L.forward(s[:T], y[:T], residual=r[:T], sum=r[:T])
        assert (y[T:] == 7).all() and torch.equal(s, u) and torch.equal(r[T:], res[T:])
        assert (L.gu[T * 4:] == 3).all() and (L.yslot[T * 4:] == 3).all()
        if T:
            assert torch.equal(r[:T], (u[:T].float() + res[:T].float()).to(u.dtype))
            _stages(L, u[:T], res[:T], y[:T], 0.0)


def test_skipping_everything_but_the_largest():
    L, u, _ = _make(100, 256, 16, 64, 4, factor=True)
    y = torch.empty_like(u)
    L.forward(u, y, tau=1e9)
    assert int(L.offsets[-1]) == 100
    _stages(L, u, None, y, 1e9)


def test_graph_with_new_inputs_and_another_stream():
    L, u, res = _make(96, 256, 16, 64, 4, gate=GATES[1], bias=True)
    y, y2 = torch.empty_like(u), torch.empty_like(u)
    L.forward(u, y, residual=res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(u, y2, residual=res)
    for _ in range(2):
        u.copy_(torch.randn_like(u))
        y2.zero_()
        g.replay()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        L.forward(u, y, residual=res, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)


def test_logits_are_the_forwards():
    import workloads
    from token_dynamic_expert_b200 import ace
    for dtype, T in (("bf16", 200), ("f32", 50)):
        w = workloads.Workload("g", T=T, d=256, E=48, m=128, k=6, dtype=dtype, bias=True, skip=0.5,
                               skip_of="slots")
        layer = workloads.make_layer(w, seed=3, device="cuda")
        u = workloads.make_tokens(w, token_seed=7, device="cuda")
        L = ace.make_layer(layer["gamma"], layer["wr"], layer["wg"], layer["wu"], layer["wd"], w.k,
                           router_bias=layer["bias"])
        dbg = ace.DebugOut(w.T, w.k, w.E)
        ace.ace_moe_forward(L, u, 0.0, torch.empty_like(u),
                            ace.alloc_workspace(ace.ace_workspace_size(L, w.T)), dbg=dbg.c)
        R = ace.make_router_layer(layer["gamma"], layer["wr"], layer["bias"])
        ws = ace.alloc_workspace(ace.ace_logits_workspace_size(R, T))
        ws.fill_(0xAB)
        logits = torch.empty(T, w.E, device="cuda")
        ace.ace_moe_logits(R, u, logits, ws)
        assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
        assert torch.equal(logits, dbg.logits)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,bias", [(1, 64, 1, False), (1, 2048, 128, True), (2, 192, 9, True), (5, 1088, 60, False),
                                        (7, 320, 256, True), (8, 2048, 512, False), (8, 4096, 33, True), (9, 2048, 33, True)])
def test_logits_of_few_tokens(dtype, T, d, E, bias):
    """fp32 products and sums: gamma w 1 rounding, at most d / 256 vectors of 8 in a
    thread, 5 across the warp, 8 across the CTA; the root's sum likewise, halved (9
    tokens take the prefill's way, sums of 64 columns and then d / 64 chunks)."""
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(d + E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    u = torch.randn(T, d, generator=g, device="cuda").to(dt)
    wr = (torch.randn(E, d, generator=g, device="cuda") * 0.05).to(dt)
    gamma, b = torch.rand(d, generator=g, device="cuda") + 0.5, torch.randn(E, generator=g, device="cuda") if bias else None
    R = ace.make_router_layer(gamma, wr, b)
    ws = ace.alloc_workspace(ace.ace_logits_workspace_size(R, T))
    ws.fill_(0xAB)
    logits = torch.full((T, E), 7.0, device="cuda")
    ace.ace_moe_logits(R, u, logits, ws, eps_rms=1e-5)
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
    x = ora.f64(u) / np.sqrt((ora.f64(u) ** 2).mean(1, keepdims=True) + 1e-5) * ora.f64(gamma)
    ref, mag = x @ ora.f64(wr).T, np.abs(x) @ np.abs(ora.f64(wr)).T
    if bias:
        ref, mag = ref + ora.f64(b), mag + np.abs(ora.f64(b))
    assert (np.abs(ora.f64(logits) - ref) <= (d / 32 + 40) * ora.U32 * mag).all()


def test_refusals():
    from token_dynamic_expert_b200 import layer_i8
    L, u, _ = _make(8, 128, 8, 64, 2)
    with pytest.raises(ValueError, match="u must be"):
        L.forward(torch.zeros(9, 128, dtype=torch.bfloat16, device="cuda"), u)
    with pytest.raises(ValueError, match="y must"):
        L.forward(u, u.float())
    with pytest.raises(ValueError, match="multiple"):
        layer_i8.LayerI8(L.gamma, L.w_router, L.wq_gu[:, :100].contiguous(), L.s_gu, L.wq_down[..., :50].contiguous(),
                         L.s_down, 2, 8)
    with pytest.raises(ValueError, match="match"):
        layer_i8.LayerI8(L.gamma, L.w_router[:4], L.wq_gu, L.s_gu, L.wq_down, L.s_down, 2, 8)


def test_rows_that_lie_apart():
    """Rows of u and residual within wider ones give the bits of contiguous rows;
    a y or sum of that kind is refused, and its neighbours stay as they were."""
    L, u, res = _make(24, 256, 8, 64, 2)
    wide = torch.randn(24, 768, device="cuda").bfloat16()
    wide[:, :256], wide[:, 256:512] = u, res
    for r, rw in ((None, None), (res, wide[:, 256:512])):
        want, got = torch.empty_like(u), torch.empty_like(u)
        L.forward(u, want, r)
        L.forward(wide[:, :256], got, rw)
        assert torch.equal(want, got) and L.status()[0] == 0
    before = wide.clone()
    with pytest.raises(ValueError, match="contiguous"):
        L.forward(u, wide[:, 512:])
    with pytest.raises(ValueError, match="contiguous"):
        L.forward(u, torch.empty_like(u), res, sum=wide[:, 512:])
    with pytest.raises(ValueError, match="device"):
        L.forward(u, torch.empty(24, 256, dtype=u.dtype))
    assert torch.equal(wide, before)
