"""What LayerI8 refuses, as it is built: a call finds nothing left to refuse after its
first kernel, which may have overwritten sum.  No GPU needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def mod():
    from token_dynamic_expert_b200 import build
    build.build()
    from token_dynamic_expert_b200 import layer_i8
    return layer_i8


def _args(E=8, d=128, m=64, k=2, dtype=torch.bfloat16):
    return dict(gamma=torch.ones(d), w_router=torch.zeros(E, d, dtype=dtype),
                wq_gu=torch.zeros(E, 2 * m, d, dtype=torch.int8), s_gu=torch.ones(E, 2 * m),
                wq_down=torch.zeros(E, d, m, dtype=torch.int8), s_down=torch.ones(E, d), k=k, max_tokens=4)


def _off(t, n=1):
    """The same values, n elements past a 16-byte boundary."""
    b = torch.zeros(t.numel() + 64, dtype=t.dtype)
    v = b[n:n + t.numel()].view(t.shape)
    return v.copy_(t)


def test_sound_arguments_end_at_the_device(mod):
    for kw in (dict(), dict(bias=torch.zeros(8), factor=torch.ones(8), gate=dict(score="sigmoid", n_groups=4, topk_groups=2,
                                                                                   group_score="top2", renorm=False, scale=2.5))):
        with pytest.raises(ValueError, match="CUDA device"):
            mod.LayerI8(**_args(), **kw)


@pytest.mark.parametrize("change,err,match", [
    (dict(k=17, E=32), ValueError, "k <= 16"), (dict(E=513), ValueError, "E <= 512"),
    (dict(d=16448), ValueError, "16384"), (dict(m=16400, d=64, E=1, k=1), ValueError, "16384"),
    (dict(max_tokens=2 ** 30), ValueError, "max_tokens"), (dict(eps=-1.0), ValueError, "eps"),
    (dict(eps=float("nan")), ValueError, "eps"),
    (dict(s_gu=torch.ones(8, 127)), ValueError, "s_gu"), (dict(s_down=torch.ones(8, 127)), ValueError, "s_down"),
    (dict(s_gu=torch.ones(8, 128, dtype=torch.float64)), TypeError, "s_gu"),
    (dict(s_down=torch.ones(8, 128).bfloat16()), TypeError, "s_down"),
    (dict(s_gu=torch.ones(128, 8).t()), ValueError, "s_gu"),
    (dict(wq_gu=torch.zeros(8, 128, 128, dtype=torch.uint8)), TypeError, "wq_gu"),
    (dict(wq_gu=torch.zeros(8, 128, 128, dtype=torch.int8).transpose(1, 2)), ValueError, "wq_gu"),
    (dict(wq_down=torch.zeros(8, 64, 128, dtype=torch.int8).transpose(1, 2)), ValueError, "wq_down"),
    (dict(w_router=torch.zeros(8, 128, dtype=torch.float16)), TypeError, "dtype"),
    (dict(gamma=torch.ones(64)), ValueError, "gamma"),
    (dict(s_gu=None), TypeError, "s_gu"), (dict(s_down=None), TypeError, "s_down"),
    (dict(bias=torch.zeros(7)), ValueError, "bias"), (dict(bias=torch.zeros(8, dtype=torch.float64)), TypeError, "bias"),
    (dict(router_bias=torch.zeros(9)), ValueError, "router_bias"),
    (dict(factor=torch.zeros(16)[::2]), ValueError, "factor"),
    (dict(wq_gu="off"), ValueError, "wq_gu must start"), (dict(wq_down="off"), ValueError, "wq_down must start"),
    (dict(w_router="off"), ValueError, "w_router must start"), (dict(gamma="off"), ValueError, "gamma must start"),
    (dict(gate=dict(n_groups=3)), RuntimeError, "ace_gate_topk"),
    (dict(gate=dict(n_groups=8, topk_groups=1)), RuntimeError, "ace_gate_topk"),
    (dict(gate=dict(scale=0.0)), RuntimeError, "ace_gate_topk"), (dict(gate=dict(score="tanh")), KeyError, "tanh"),
    (dict(gate=dict(tau=0.5)), TypeError, "tau"), (dict(gate=dict(k=3)), TypeError, "k"),
])
def test_refused_as_it_is_built(mod, change, err, match):
    sizes = {n: change[n] for n in ("E", "d", "m", "k") if n in change}
    a = _args(**sizes)
    a.update({n: (_off(a[n]) if isinstance(v, str) else v) for n, v in change.items() if n not in ("E", "d", "m")})
    with pytest.raises(err, match=match):
        mod.LayerI8(**a)
