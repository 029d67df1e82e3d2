"""Outputs and workspaces that lie on an input: refused on the host, before any
launch.  No GPU needed; addresses are never dereferenced."""
import ctypes

import pytest

U, G, W, B, OUT, WS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000


@pytest.fixture(scope="module")
def ace():
    from token_dynamic_expert_b200 import build
    build.build()
    from token_dynamic_expert_b200 import ace as mod
    return mod


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("dtype", [0, 1])
def test_logits(ace, T, dtype):
    d, E, es = 256, 8, (2, 4)[dtype]

    def call(logits=OUT, ws=WS, **kw):
        L = ace.ace_layer(**dict(dict(d=d, E=E, m=64, k=1, dtype=dtype, gamma=G, w_router=W, router_bias=B), **kw))
        return ace.lib().ace_moe_logits(ctypes.byref(L), U, T, 1e-6, logits, ws, 1 << 26, None)

    ends = {U: T * d * es, G: d * 4, W: E * d * es, B: E * 4}
    for at, n in ends.items():
        assert call(logits=at) == ace.ACE_ERR_INVALID_ARG
        assert call(logits=at + n - 4) == ace.ACE_ERR_INVALID_ARG
        assert call(logits=at - T * E * 4 + 4) == ace.ACE_ERR_INVALID_ARG
        assert call(ws=at) == ace.ACE_ERR_INVALID_ARG
        assert call(ws=(at + n - 4) & ~255) == ace.ACE_ERR_INVALID_ARG
        assert call(ws=at - 256) == ace.ACE_ERR_INVALID_ARG
    assert call(logits=WS + 256) == ace.ACE_ERR_INVALID_ARG


def test_matmul(ace):
    S, N, K, E = 8, 96, 64, 3
    at = dict(xq=0x1000000, x_scale=0x2000000, wq=0x3000000, w_scale=0x4000000, offsets=0x5000000, row_of=0x6000000,
              slot_scale=0x7000000)
    size = dict(xq=S * K, x_scale=S * 4, wq=E * N * K, w_scale=E * N * 4, offsets=(E + 1) * 4, row_of=S * 4, slot_scale=S * 4)

    def call(out=OUT, ws=WS):
        p = ace.ace_i8_product(ldx=K, n_rows=S, E=E, N=N, K=K, **at)
        return ace.lib().ace_matmul_i8(ctypes.byref(p), S, out, N, 1, ws, 256, None)

    for name, a in at.items():
        for out in (a, a + size[name] - 4, a - S * N * 4 + 4):
            assert call(out=out) == ace.ACE_ERR_INVALID_ARG, name
        for ws in (a, (a + size[name] - 4) & ~255):
            assert call(ws=ws) == ace.ACE_ERR_INVALID_ARG, name
    assert call(out=WS) == ace.ACE_ERR_INVALID_ARG
