"""Argument checks of the 8-bit layer's operators: refused on the host, before
any launch.  No GPU needed; addresses are never dereferenced."""
import ctypes

import pytest
import torch

P, Q, R = 0x1000000, 0x2000000, 0x3000000


@pytest.fixture(scope="module")
def ace():
    from token_dynamic_expert_b200 import build
    build.build()
    from token_dynamic_expert_b200 import ace as mod
    return mod


def _norm(ace, **kw):
    a = dict(x=P, ldx=64, res=None, ldr=0, T=4, d=64, dt=ace.ACE_BF16, gamma=Q, eps=1e-6, sum=None, lds=0, y=R, ldy=64,
             q=None, ldq=0, qs=None)
    a.update(kw)
    return ace.lib().ace_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(gamma=None), dict(y=None), dict(T=-1), dict(d=0), dict(dt=5),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(ldx=63), dict(ldy=63), dict(x=P + 1),
                                 dict(gamma=Q + 2), dict(q=R + 0x100000, ldq=64), dict(res=Q + 0x100000, ldr=60),
                                 dict(y=P + 2), dict(y=P, ldy=72), dict(q=P, ldq=64, qs=Q + 0x8000),
                                 dict(sum=R, lds=64), dict(y=Q), dict(q=R + 0x100000, ldq=64, qs=R)])
def test_norm_refuses(ace, bad):
    assert _norm(ace, **bad) == ace.ACE_ERR_INVALID_ARG


def test_norm_limits(ace):
    assert _norm(ace, d=16385, ldx=16385, ldy=16385) == ace.ACE_ERR_UNSUPPORTED
    assert _norm(ace, T=0, x=None, gamma=None) == ace.ACE_OK


def _swiglu(ace, **kw):
    a = dict(gu=P, ld=128, S=4, m=64, dt=ace.ACE_BF16, nv=None, y=R, ldy=64, q=None, ldq=0, qs=None)
    a.update(kw)
    return ace.lib().ace_swiglu(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(gu=None), dict(y=None), dict(S=-1), dict(m=0), dict(dt=2), dict(ld=127),
                                 dict(ldy=63), dict(gu=P + 1), dict(nv=Q + 2), dict(y=P + 16), dict(nv=R + 4),
                                 dict(q=R, ldq=64, qs=Q), dict(q=Q, ldq=64), dict(q=Q, ldq=60, qs=Q + 0x10000)])
def test_swiglu_refuses(ace, bad):
    assert _swiglu(ace, **bad) == ace.ACE_ERR_INVALID_ARG


def test_swiglu_limits(ace):
    assert _swiglu(ace, m=16385, ld=32770, ldy=16385) == ace.ACE_ERR_UNSUPPORTED
    assert _swiglu(ace, S=0, gu=None) == ace.ACE_OK


def _gate(ace, **kw):
    o = dict(score=0, n_groups=4, topk_groups=2, group_score=1, renorm_topk=1, scale=1.0, tau=0.0)
    a = dict(x=P, ld=64, dt=ace.ACE_F32, T=3, E=64, k=8, bias=None)
    b = dict(idx=Q, w=R, factor=None, keep=None)
    for k, v in kw.items():
        next(d for d in (o, a, b) if k in d)[k] = v
    return ace.lib().ace_gate_topk(*a.values(), ctypes.byref(ace.ace_gate_opts(**o)), *b.values(), None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(idx=None), dict(w=None), dict(T=-1), dict(E=0), dict(k=0), dict(k=17),
                                 dict(k=65), dict(dt=3), dict(score=2), dict(group_score=2), dict(n_groups=0),
                                 dict(n_groups=5), dict(topk_groups=0), dict(topk_groups=5), dict(ld=63),
                                 dict(n_groups=16, topk_groups=1), dict(scale=0.0), dict(scale=float("inf")),
                                 dict(scale=float("nan")), dict(x=P + 2), dict(bias=Q + 1), dict(idx=Q + 2),
                                 dict(idx=P), dict(w=P + 64), dict(w=Q + 32), dict(bias=Q), dict(keep=R + 4),
                                 dict(factor=R)])
def test_gate_refuses(ace, bad):
    assert _gate(ace, **bad) == ace.ACE_ERR_INVALID_ARG


def test_gate_limits(ace):
    assert _gate(ace, E=513, ld=513) == ace.ACE_ERR_UNSUPPORTED
    assert _gate(ace, n_groups=64, topk_groups=16) == ace.ACE_ERR_UNSUPPORTED
    assert _gate(ace, T=0, x=None, idx=None, w=None) == ace.ACE_OK
    lib = ace.lib()
    assert lib.ace_gate_topk(P, 64, 1, 3, 64, 8, None, None, Q, R, None, None, None) == ace.ACE_ERR_INVALID_ARG


def _group(ace, **kw):
    a = dict(idx=P, keep=None, gate=None, T=4, k=2, E=8, off=Q, so=R, st=None, sg=None)
    a.update(kw)
    return ace.lib().ace_moe_group(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(idx=None), dict(off=None), dict(so=None), dict(T=-1), dict(k=0), dict(k=17),
                                 dict(E=0), dict(sg=P + 0x10000), dict(idx=P + 1), dict(off=Q + 2), dict(so=R + 1),
                                 dict(so=P), dict(so=Q + 16), dict(st=R), dict(keep=Q), dict(gate=R, sg=P + 0x10000)])
def test_group_refuses(ace, bad):
    assert _group(ace, **bad) == ace.ACE_ERR_INVALID_ARG


def test_group_limits(ace):
    assert _group(ace, E=513) == ace.ACE_ERR_UNSUPPORTED
    assert _group(ace, T=2 ** 31 - 1) == ace.ACE_ERR_UNSUPPORTED


def _matmul(ace, S=8, out=0x9000000, ldo=96, dt=0, ws=0xA000000, ws_bytes=256, **kw):
    a = dict(xq=P, ldx=64, n_rows=8, x_scale=Q, wq=R, w_scale=0x4000000, E=1, N=96, K=64, offsets=None, row_of=None,
             slot_scale=None)
    a.update(kw)
    p = ace.ace_i8_product(**a)
    return ace.lib().ace_matmul_i8(ctypes.byref(p), S, out, ldo, dt, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(S=-1), dict(N=0), dict(K=0), dict(E=0), dict(n_rows=-1), dict(n_rows=7),
                                 dict(n_rows=0, row_of=Q), dict(dt=2), dict(E=4), dict(xq=None), dict(x_scale=None),
                                 dict(wq=None), dict(w_scale=None), dict(out=None), dict(xq=P + 8), dict(wq=R + 4),
                                 dict(ldx=48), dict(ldx=72), dict(ldo=95), dict(out=0x9000001), dict(x_scale=Q + 2),
                                 dict(out=P), dict(out=R + 128), dict(out=0xA000000), dict(slot_scale=Q + 1)])
def test_matmul_refuses(ace, bad):
    assert _matmul(ace, **bad) == ace.ACE_ERR_INVALID_ARG


def test_matmul_limits(ace):
    assert _matmul(ace, K=72, ldx=80) == ace.ACE_ERR_UNSUPPORTED
    assert _matmul(ace, K=65552, ldx=65552) == ace.ACE_ERR_UNSUPPORTED
    assert _matmul(ace, E=513, offsets=0x5000000) == ace.ACE_ERR_UNSUPPORTED
    assert _matmul(ace, ws=None) == ace.ACE_ERR_WORKSPACE
    assert _matmul(ace, ws=0xA000010) == ace.ACE_ERR_WORKSPACE
    assert _matmul(ace, ws_bytes=255) == ace.ACE_ERR_WORKSPACE


def test_binding_refuses_what_the_kernels_cannot_see(ace):
    """Types, shapes, strides and devices, before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        ace.ace_add_rmsnorm(x, torch.ones(64), y=torch.empty_like(x))
    with pytest.raises(TypeError, match="gamma"):
        ace.ace_add_rmsnorm(x, torch.ones(64, dtype=torch.bfloat16), y=torch.empty_like(x))
    with pytest.raises(TypeError, match="dtype"):
        ace.ace_add_rmsnorm(x.half(), torch.ones(64), y=x.half())
    with pytest.raises(ValueError, match="residual"):
        ace.ace_add_rmsnorm(x, torch.ones(64), residual=x[:3], y=torch.empty_like(x))
    with pytest.raises(ValueError, match="neighbouring"):
        ace.ace_add_rmsnorm(x.t().contiguous().t(), torch.ones(64), y=torch.empty_like(x))
    with pytest.raises(ValueError, match="neighbouring"):
        ace.ace_add_rmsnorm(x[:1].expand(4, 64), torch.ones(64), y=torch.empty_like(x))
    with pytest.raises(TypeError, match="idx"):
        ace.ace_gate_topk(torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2))
    with pytest.raises(KeyError):
        ace.ace_gate_topk(torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), score="tanh")
    with pytest.raises(ValueError, match="offsets"):
        ace.ace_matmul_i8(torch.zeros(3, 16, dtype=torch.int8), torch.ones(3), torch.zeros(2, 5, 16, dtype=torch.int8),
                          torch.ones(2, 5), torch.zeros(3, 5), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2 m"):
        ace.ace_swiglu(torch.zeros(3, 7))


def test_logits_refuses(ace):
    def call(T=4, u=P, eps=1e-6, logits=Q, ws=0xA000000, ws_bytes=1 << 30, **kw):
        a = dict(d=256, E=8, m=64, k=1, dtype=0, gamma=R, w_router=R)
        a.update(kw)
        return ace.lib().ace_moe_logits(ctypes.byref(ace.ace_layer(**a)), u, T, eps, logits, ws, ws_bytes, None)

    for bad in (dict(u=None), dict(logits=None), dict(T=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(gamma=None),
                dict(w_router=None), dict(u=P + 8), dict(logits=Q + 2), dict(E=0), dict(logits=P),
                dict(logits=0xA000000)):
        assert call(**bad) == ace.ACE_ERR_INVALID_ARG, bad
    assert call(d=100) == ace.ACE_ERR_UNSUPPORTED
    assert call(ws=None) == ace.ACE_ERR_WORKSPACE
    assert call(ws_bytes=1024) == ace.ACE_ERR_WORKSPACE
    bad = ace.ace_layer(d=256, E=8, m=64, k=1, dtype=0)
    assert ace.lib().ace_logits_workspace_size(ctypes.byref(bad), 4) == 0


def test_counts_near_two_to_the_31(ace):
    """Rounding such a count up to whole tiles would leave 32 bits."""
    n = 2 ** 31 - 255
    assert _norm(ace, T=n) == ace.ACE_ERR_UNSUPPORTED
    assert _swiglu(ace, S=n) == ace.ACE_ERR_UNSUPPORTED
    assert _gate(ace, T=n) == ace.ACE_ERR_UNSUPPORTED
    assert _group(ace, T=n, k=1) == ace.ACE_ERR_UNSUPPORTED
    assert _matmul(ace, S=n, n_rows=n) == ace.ACE_ERR_UNSUPPORTED
    assert _matmul(ace, n_rows=n) == ace.ACE_ERR_UNSUPPORTED


def test_router_layer_refuses(ace):
    """What the kernels would read past the end of."""
    g, w, b = torch.ones(64), torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8)
    assert ace.make_router_layer(g, w, b).E == 8
    for bad, err in (((g.bfloat16(), w), TypeError), ((g[:32], w), ValueError), ((g, w[0]), ValueError),
                     ((g, w.half()), TypeError), ((g, w[:, ::2]), ValueError), ((g, w, b[:7]), ValueError),
                     ((g, w, b.double()), TypeError), ((g, w[:, :32], b), ValueError)):
        with pytest.raises(err):
            ace.make_router_layer(*bad)
