"""ace_add_rmsnorm and ace_swiglu where fp32 intermediates leave their range while
inputs and results do not.  Tolerances as in test_gpu_i8_rows.py; a result below
the normal numbers of its type may be off by one of its steps."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149}  # the smallest numbers


def _norm(x, gamma, eps, res=None):
    from token_dynamic_expert_b200 import ace
    T, d = x.shape
    o = dict(y=torch.full_like(x, 7), q=torch.full((T, d), 99, dtype=torch.int8, device="cuda"),
             q_scale=torch.full((T,), 7.0, device="cuda"), sum=torch.full_like(x, 7))
    ace.ace_add_rmsnorm(x, gamma, residual=res, eps=eps, **o)
    torch.cuda.synchronize()
    return o


def _check_norm(x, gamma, dt, eps, res=None):
    o = _norm(x, gamma, eps, res)
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(o["sum"], s)
    y, q, scale = ora.norm(ora.f64(s), ora.f64(gamma), eps)
    # y is rounded to its type; s r to fp32 ahead of gamma
    assert ora.close(ora.f64(o["y"]), y, ora.HALF[dt] + 24 * ora.U32, 2 * STEP[dt]) <= 1
    assert np.array_equal(o["q"].cpu().numpy(), q)
    assert ora.close(ora.f64(o["q_scale"]), scale, 24 * ora.U32, 2 * STEP["f32"]) <= 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(3, 64), (5, 2048), (700, 512), (700, 2048), (2, 16384), (3, 1001)])
@pytest.mark.parametrize("size", [1e19, 1e20, 3e37])
def test_norm_of_rows_whose_squares_overflow(dt, T, d, size):
    g = torch.Generator(device="cuda").manual_seed(d + T)
    x = (torch.randn(T, d, generator=g, device="cuda").clamp(-3, 3) * size).to(DT[dt])
    x[1] = torch.randn(d, generator=g, device="cuda").to(DT[dt])  # an ordinary row among them
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    for eps in (1e-6, 0.0):
        _check_norm(x, gamma, dt, eps)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(3, 64), (5, 2048), (700, 512), (700, 2048), (2, 16384), (3, 1001)])
@pytest.mark.parametrize("size", [1e-15, 1e-19, 1e-22, 1e-25, 1e-35])
def test_norm_of_rows_whose_squares_underflow(dt, T, d, size):
    """Without eps, or with one as small, every row is of order 1 again."""
    g = torch.Generator(device="cuda").manual_seed(d + T)
    x = (torch.randn(T, d, generator=g, device="cuda") * size).to(DT[dt])
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    for eps in (0.0, 2.0 ** -120, 2.0 ** -90, 1e-6):
        _check_norm(x, gamma, dt, eps)


def test_norm_residual_and_in_place_beyond_the_range():
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(9)
    gamma = torch.rand(768, generator=g, device="cuda") + 0.5
    for T in (4, 700):
        x, res = ((torch.randn(T, 768, generator=g, device="cuda") * 1e21).bfloat16() for _ in range(2))
        _check_norm(x, gamma, "bf16", 1e-6, res)
        want = _norm(x, gamma, 1e-6, res)
        ace.ace_add_rmsnorm(x, gamma, residual=res, sum=res, y=x)
        assert torch.equal(x, want["y"]) and torch.equal(res, want["sum"])


def test_norm_of_zero_rows_without_eps():
    """0 / 0, as the formula has it, in y; the int8 row is zeros."""
    x = torch.zeros(3, 256, device="cuda")
    o = _norm(x, torch.ones(256, device="cuda"), 0.0)
    assert o["y"].isnan().all() and (o["q"] == 0).all() and (o["q_scale"] == 0).all()
