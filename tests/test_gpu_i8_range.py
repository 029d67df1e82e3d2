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


@pytest.mark.parametrize("T,d", [(3, 64), (700, 512), (700, 2048), (3, 1001)])
def test_norm_outputs_alone_beyond_the_range(T, d):
    """Every subset of the outputs has the bits of all of them together."""
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(d)
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    size = torch.tensor([1e21, 1.0, 1e-24], device="cuda")[torch.arange(T, device="cuda") % 3][:, None]
    for dt in (torch.bfloat16, torch.float32):
        x, res = ((torch.randn(T, d, generator=g, device="cuda") * size).to(dt) for _ in range(2))
        for r in (None, res):
            want = _norm(x, gamma, 0.0, r)
            for names in (("y",), ("sum", "y"), ("q", "q_scale"), ("y", "q", "q_scale"), ("sum", "q", "q_scale")):
                o = {n: torch.empty_like(want[n]) for n in names}
                ace.ace_add_rmsnorm(x, gamma, residual=r, eps=0.0, **o)
                assert all(torch.equal(o[n], want[n]) for n in names), names
            a, b = x.clone(), res.clone()  # y over either input, the sum not kept
            ace.ace_add_rmsnorm(a, gamma, residual=None if r is None else b, eps=0.0, y=a if r is None else b)
            assert torch.equal(a if r is None else b, want["y"])


def test_norm_of_zero_rows_without_eps():
    """0 / 0, as the formula has it, in y; the int8 row is zeros."""
    x = torch.zeros(3, 256, device="cuda")
    o = _norm(x, torch.ones(256, device="cuda"), 0.0)
    assert o["y"].isnan().all() and (o["q"] == 0).all() and (o["q_scale"] == 0).all()


def _swiglu(gu, dt):
    from token_dynamic_expert_b200 import ace
    S, m = gu.shape[0], gu.shape[1] // 2
    o = dict(y=torch.full((S, m), 7, dtype=gu.dtype, device="cuda"),
             q=torch.full((S, m), 99, dtype=torch.int8, device="cuda"), q_scale=torch.full((S,), 7.0, device="cuda"))
    ace.ace_swiglu(gu, **o)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("S,m", [(3, 64), (5, 768), (700, 512), (700, 2048), (2, 16384), (3, 1001)])
def test_swiglu_of_gates_far_below_zero(dt, S, m):
    """g from -100 to -80: SiLU(g) falls from 1e-33 to 4e-42, g e^g, past where its
    reciprocal leaves fp32 (-87.3); rows of them alone, and of one beside ordinary ones."""
    g = torch.Generator(device="cuda").manual_seed(S + m)
    gu = torch.randn(S, 2 * m, generator=g, device="cuda") * 2
    gu[:, :m] = torch.linspace(-100, -80, m, device="cuda")
    gu[:, m:] *= 2.0 ** torch.randint(-8, 60, (S, 1), generator=g, device="cuda")
    gu[1] = torch.randn(2 * m, generator=g, device="cuda")
    gu[1, m // 2] = -90.0
    gu = gu.to(DT[dt])
    o = _swiglu(gu, dt)
    h, q, scale = ora.swiglu(ora.f64(gu))
    # h in fp32 (half a step below the normal numbers), then y's rounding
    assert ora.close(ora.f64(o["y"]), h, ora.HALF[dt] + 11 * ora.U32, 2 * STEP[dt]) <= 1
    used = np.abs(h).max(1) >= 2.0 ** -126
    assert used.sum() >= min(S, 3) - 1 and used[1]
    assert np.array_equal(o["q"].cpu().numpy()[used], q[used])
    assert ora.close(ora.f64(o["q_scale"])[used], scale[used], 13 * ora.U32) <= 1
    assert not o["q"].cpu().numpy()[~used].any() and not o["q_scale"].cpu().numpy()[~used].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("S,m", [(2, 64), (700, 512), (3, 1001)])
def test_swiglu_of_gates_at_minus_infinity(dt, S, m):
    """SiLU's limit, 0: a channel that is masked out so leaves its row's others alone."""
    g = torch.Generator(device="cuda").manual_seed(m)
    gu = torch.randn(S, 2 * m, generator=g, device="cuda").to(DT[dt])
    masked = torch.rand(S, m, generator=g, device="cuda") < 0.3
    zeros = gu.clone()
    gu[:, :m][masked] = -float("inf")
    zeros[:, :m][masked] = 0.0
    # the row of zeros in 64 bits: such a row is formed by another path than one without
    # them, so y and scale agree within their tolerance, not bit for bit
    o = _swiglu(gu, dt)
    h, q, scale = ora.swiglu(ora.f64(zeros))
    assert ora.close(ora.f64(o["y"]), h, ora.HALF[dt] + 11 * ora.U32, 2 * STEP[dt]) <= 1
    assert np.array_equal(o["q"].cpu().numpy(), q) and (o["y"][masked] == 0).all()
    assert ora.close(ora.f64(o["q_scale"]), scale, 13 * ora.U32) <= 1


def test_swiglu_low_gates_in_each_output_alone_and_with_nan():
    from token_dynamic_expert_b200 import ace
    for S, m in ((4, 96), (700, 96), (700, 2048)):
        gu = torch.randn(S, 2 * m, device="cuda")
        gu[:, 3] = -88.0
        gu[1, 5], gu[2, m + 3] = float("nan"), float("inf")
        both = _swiglu(gu, "f32")
        y = torch.empty(S, m, device="cuda")
        q, qs = torch.empty(S, m, dtype=torch.int8, device="cuda"), torch.empty(S, device="cuda")
        ace.ace_swiglu(gu, y=y)
        ace.ace_swiglu(gu, q=q, q_scale=qs)
        assert torch.equal(y.view(torch.int32), both["y"].view(torch.int32))
        assert torch.equal(q, both["q"]) and torch.equal(qs.view(torch.int32), both["q_scale"].view(torch.int32))
        assert (q[1:3] == 0).all() and qs[1:3].isnan().all() and y[1].isnan().sum() == 1
        assert y[2, 3] == -float("inf") and not y[0].isnan().any()
        h, rq, rs = ora.swiglu(ora.f64(gu[3:]))
        assert ora.close(ora.f64(y[3:]), h, 12 * ora.U32, 2 * STEP["f32"]) <= 1
        assert np.array_equal(q[3:].cpu().numpy(), rq) and ora.close(ora.f64(qs[3:]), rs, 13 * ora.U32) <= 1
