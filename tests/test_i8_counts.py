"""Counts that do not fit the library's 32-bit arguments are refused by the binding,
where the conversion would have cut them to their low bits and served a part of
the rows.  Tensors without memory; no GPU needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def ace():
    from token_dynamic_expert_b200 import build
    build.build()
    from token_dynamic_expert_b200 import ace as mod
    return mod


def t(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


I32, I8, U8 = torch.int32, torch.int8, torch.uint8


@pytest.mark.parametrize("n", [2 ** 31 - 255, 2 ** 31 + 5, 2 ** 32 + 3])
def test_counts_beyond_32_bits(ace, n):
    ws = t(1 << 20, dtype=U8)
    R = ace.ace_layer(d=64, E=8, m=64, k=1, dtype=ace.ACE_F32)
    calls = [
        lambda: ace.ace_add_rmsnorm(t(n, 2), t(2), y=t(n, 2)),
        lambda: ace.ace_add_rmsnorm(t(1, n), t(n), y=t(1, n)),
        lambda: ace.ace_moe_logits(R, t(n, 64), t(n, 8), ws),
        lambda: ace.ace_gate_topk(t(n, 8), t(n, 2, dtype=I32), t(n, 2)),
        lambda: ace.ace_gate_topk(t(1, n), t(1, 2, dtype=I32), t(1, 2)),
        lambda: ace.ace_gate_topk(t(1, 8), t(1, n, dtype=I32), t(1, n)),
        lambda: ace.ace_moe_group(t(n, 1, dtype=I32), 8, t(9, dtype=I32), t(n, 1, dtype=I32)),
        lambda: ace.ace_moe_group(t(1, n, dtype=I32), 8, t(9, dtype=I32), t(1, n, dtype=I32)),
        lambda: ace.ace_moe_group(t(1, 1, dtype=I32), n, t(n + 1, dtype=I32), t(1, 1, dtype=I32)),
        lambda: ace.ace_matmul_i8(t(n, 16, dtype=I8), t(n), t(8, 16, dtype=I8), t(8), t(n, 8), ws),
        lambda: ace.ace_matmul_i8(t(n, 16, dtype=I8), t(n), t(8, 16, dtype=I8), t(8), t(4, 8), ws, row_of=t(4, dtype=I32)),
        lambda: ace.ace_matmul_i8(t(4, 16, dtype=I8), t(4), t(n, 16, dtype=I8), t(n), t(4, n), ws),
        lambda: ace.ace_matmul_i8(t(4, 16, dtype=I8), t(4), t(n, 8, 16, dtype=I8), t(n, 8), t(4, 8), ws,
                                  offsets=t(n + 1, dtype=I32)),
        lambda: ace.ace_swiglu(t(n, 2), y=t(n, 1)),
        lambda: ace.ace_swiglu(t(1, 2 * n), y=t(1, n)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ace.AceError) as e:
            call()
        assert e.value.code == ace.ACE_ERR_UNSUPPORTED, i


def test_logits_of_more_tokens_than_the_limit(ace):
    import ctypes
    L = ace.ace_layer(d=64, E=8, m=64, k=1, dtype=1, gamma=0x3000000, w_router=0x3000000)
    for n in (2 ** 31 - 255, 2 ** 31 - 1):
        assert ace.lib().ace_moe_logits(ctypes.byref(L), 0x1000000, n, 1e-6, 0x2000000, 0xA000000, 1 << 30,
                                        None) == ace.ACE_ERR_UNSUPPORTED
