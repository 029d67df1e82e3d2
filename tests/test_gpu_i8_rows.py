"""ace_add_rmsnorm and ace_swiglu against 64-bit numpy.

Tolerances: s is one fp32 addition and one rounding, compared bit for bit.  The
sum of squares of a row takes at most 16 additions in a thread and 10 across
the CTA (26 half steps, 13 for its root), the mean, eps, root and reciprocal 4,
the two products 2, and max, division by 127 2 more: 21, taken as 24.  h: the
base-2 exponential 2 ulp (4 half steps) with a correcting factor and its product
(2), 1 + e, the reciprocal 1 ulp (2), two products (2): 11.  Each result then
rounds once to its type, and the scale of h takes two products more (13).  q
has to be equal."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rand(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dt])


def _norm(x, gamma, res, eps=1e-6, want=("sum", "y", "q"), **bufs):
    from token_dynamic_expert_b200 import ace
    T, d = x.shape
    o = {}
    if "sum" in want:
        o["sum"] = torch.full((T, d), 7, dtype=x.dtype, device="cuda")
    if "y" in want:
        o["y"] = torch.full((T, d), 7, dtype=x.dtype, device="cuda")
    if "q" in want:
        o["q"] = torch.full((T, d), 99, dtype=torch.int8, device="cuda")
        o["q_scale"] = torch.full((T,), 7.0, device="cuda")
    o.update(bufs)
    ace.ace_add_rmsnorm(x, gamma, residual=res, eps=eps, **o)
    torch.cuda.synchronize()
    return o


def _check_norm(o, x, gamma, res, dt, eps=1e-6):
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    if "sum" in o:
        assert torch.equal(o["sum"], s)
    y, q, scale = ora.norm(ora.f64(s), ora.f64(gamma), eps)
    if "y" in o:
        assert ora.close(ora.f64(o["y"]), y, ora.HALF[dt] + 24 * ora.U32, 1e-38) <= 1
    if "q" in o:
        assert np.array_equal(o["q"].cpu().numpy(), q)
        assert ora.close(ora.f64(o["q_scale"]), scale, 24 * ora.U32) <= 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2048), (3, 7), (5, 64), (37, 1000), (130, 2050),
                                 (2, 8192), (3, 8191), (2, 16384), (1, 16383), (9, 16382)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_sizes(dt, T, d, residual):
    x, gamma = _rand((T, d), dt, d + T), torch.rand(d, device="cuda") + 0.5
    res = _rand((T, d), dt, d + T + 1, 3.0) if residual else None
    _check_norm(_norm(x, gamma, res), x, gamma, res, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 100, 264, 512, 520, 1000, 1024])
def test_many_short_rows(dt, d):
    """The forms that many rows take: a warp a row, several vectors a thread."""
    T = 700
    x, res, gamma = _rand((T, d), dt, d), _rand((T, d), dt, d + 1), torch.rand(d, device="cuda") + 0.5
    x[13], res[13] = 0, 0
    x[14, 0] = float("nan")
    o = _norm(x, gamma, res)
    ok = torch.arange(T, device="cuda") != 14
    _check_norm({k: v[ok] for k, v in o.items()}, x[ok], gamma, res[ok], dt)
    assert (o["q"][14] == 0).all() and o["q_scale"][14].isnan()
    gu = _rand((T, 2 * d), dt, d + 2, 2.0)
    _check_swiglu(_swiglu(gu), gu, dt)
    nv = torch.tensor([401], dtype=torch.int32, device="cuda")
    o = _swiglu(gu, n_valid=nv)
    _check_swiglu({k: v[:401] for k, v in o.items()}, gu[:401], dt)
    assert (o["y"][401:] == 7).all() and (o["q"][401:] == 99).all() and (o["q_scale"][401:] == 7).all()


@pytest.mark.parametrize("want", [("sum",), ("y",), ("q",), ("sum", "q"), ("y", "q"), ("sum", "y")])
def test_norm_each_output_alone(want):
    x, res, gamma = _rand((11, 768), "bf16", 1), _rand((11, 768), "bf16", 2), torch.rand(768, device="cuda")
    _check_norm(_norm(x, gamma, res, want=want), x, gamma, res, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_strided_rows_keep_their_gaps(dt):
    big = _rand((19, 300), dt, 3)
    x = big[:, 5:5 + 129]
    res = _rand((19, 131), dt, 4)[:, :129]
    gamma = torch.rand(129, device="cuda") + 0.1
    sums = torch.full((19, 200), 7, dtype=DT[dt], device="cuda")
    ys, qs = sums.clone(), torch.full((19, 200), 99, dtype=torch.int8, device="cuda")
    o = _norm(x, gamma, res, sum=sums[:, 3:132], y=ys[:, 1:130], q=qs[:, 2:131])
    _check_norm(o, x, gamma, res, dt)
    for t, lo in ((sums, 3), (ys, 1)):
        assert (t[:, :lo] == 7).all() and (t[:, lo + 129:] == 7).all()
    assert (qs[:, :2] == 99).all() and (qs[:, 131:] == 99).all()


def test_norm_in_place_on_either_input():
    gamma = torch.rand(512, device="cuda") + 0.5
    for into in ("x", "res"):
        x, res = _rand((6, 512), "bf16", 5), _rand((6, 512), "bf16", 6)
        x0, r0 = x.clone(), res.clone()
        o = _norm(x, gamma, res, sum=x if into == "x" else res, y=res if into == "x" else x)
        _check_norm(o, x0, gamma, r0, "bf16")


def test_norm_special_rows():
    """Zeros, one element alone, halves, tiny and huge rows, infinity, NaN."""
    d = 256
    x = torch.zeros(9, d, device="cuda")
    x[1, 17] = -3.0
    x[2] = torch.arange(d, device="cuda") % 128      # q = the value: no rounding
    x[3] = 1.0
    x[3, 1::2] = 0.5                                 # 63.5: to the even 64
    x[4] = torch.randn(d, device="cuda") * 1e-33     # 127 / M overflows
    x[5] = torch.randn(d, device="cuda") * 1e15
    x[6] = 1e-42                                     # below the normal numbers
    x[7, 3], x[8, 4] = float("inf"), float("nan")
    gamma = torch.ones(d, device="cuda")
    o = _norm(x, gamma, None)
    _check_norm({k: v[:6] for k, v in o.items()}, x[:6], gamma, None, "f32")
    assert (o["q"][3, 1::2] == 64).all() and (o["q"][2] == x[2].to(torch.int8)).all()
    assert (o["q"][6:] == 0).all() and o["q_scale"][6] == 0 and o["q_scale"][7:].isnan().all()


def test_norm_many_rows_next_to_halves():
    """Products s gamma / M that fall on or next to halves, in bf16 steps."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x = (torch.randint(-254, 255, (3000, 512), generator=g, device="cuda").float() / 2)
    x[:, 0] = 127.0
    gamma = torch.ones(512, device="cuda")
    gamma[1:256] += (torch.rand(255, generator=g, device="cuda") - 0.5) * 2.0 ** -21
    _check_norm(_norm(x, gamma, None), x, gamma, None, "f32")


def test_norm_no_rows():
    from token_dynamic_expert_b200 import ace
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ace.ace_add_rmsnorm(x, torch.ones(64, device="cuda"), y=torch.empty_like(x))


def _swiglu(gu, want=("y", "q"), n_valid=None):
    from token_dynamic_expert_b200 import ace
    S, m = gu.shape[0], gu.shape[1] // 2
    o = {}
    if "y" in want:
        o["y"] = torch.full((S, m), 7, dtype=gu.dtype, device="cuda")
    if "q" in want:
        o["q"] = torch.full((S, m), 99, dtype=torch.int8, device="cuda")
        o["q_scale"] = torch.full((S,), 7.0, device="cuda")
    ace.ace_swiglu(gu, n_valid=n_valid, **o)
    torch.cuda.synchronize()
    return o


def _check_swiglu(o, gu, dt):
    h, q, scale = ora.swiglu(ora.f64(gu))
    if "y" in o:
        assert ora.close(ora.f64(o["y"]), h, ora.HALF[dt] + 11 * ora.U32, 1e-37) <= 1
    if "q" in o:
        assert np.array_equal(o["q"].cpu().numpy(), q)
        assert ora.close(ora.f64(o["q_scale"]), scale, 13 * ora.U32) <= 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("S,m", [(1, 1), (1, 768), (5, 7), (64, 512), (300, 1000), (33, 1030),
                                 (2, 4096), (3, 8191), (1, 16384), (2, 16383)])
def test_swiglu_sizes(dt, S, m):
    gu = _rand((S, 2 * m), dt, S + m, 2.0)
    _check_swiglu(_swiglu(gu), gu, dt)


def test_swiglu_rows_in_use_and_strides():
    wide = _rand((50, 2 * 96 + 24), "bf16", 8)
    gu = wide[:, 8:8 + 192]
    for n in (-1, 0, 1, 37, 50, 60):
        nv = torch.tensor([n], dtype=torch.int32, device="cuda")
        o = _swiglu(gu, n_valid=nv)
        n = max(0, min(n, 50))
        _check_swiglu({k: v[:n] for k, v in o.items()}, gu[:n], "bf16") if n else None
        assert (o["y"][n:] == 7).all() and (o["q"][n:] == 99).all() and (o["q_scale"][n:] == 7).all()


def test_swiglu_special_rows():
    m = 64
    gu = torch.randn(6, 2 * m, device="cuda")
    gu[0, :m] = -200.0                # silu underflows to 0 for every element
    gu[1, :m] = 300.0
    gu[2] *= 1e-15                    # h near 1e-30: 127 / M is large
    gu[3, 5] = float("nan")
    gu[4, m + 2] = float("inf")
    gu[5, m:] = 0.0
    o = _swiglu(gu)
    _check_swiglu({k: v[1:3] for k, v in o.items()}, gu[1:3], "f32")
    assert (o["q"][[0, 3, 4, 5]] == 0).all()
    assert o["q_scale"][0] == 0 and o["q_scale"][5] == 0 and o["q_scale"][3:5].isnan().all()


@pytest.mark.parametrize("m,rows", [(64, 5), (512, 700), (2048, 700)])
def test_swiglu_from_the_smallest_to_the_largest_rows(m, rows):
    """Row maxima from 2^-120 to 2^127, each scale in several rows."""
    g = torch.Generator(device="cuda").manual_seed(m)
    gu = torch.randn(rows, 2 * m, generator=g, device="cuda")
    gu[:, m:] = torch.tanh(gu[:, m:])
    e = torch.linspace(-120, 124, rows, device="cuda").round()
    gu[:, m:] *= torch.ldexp(torch.ones(rows, device="cuda"), e.int())[:, None]
    gu[:, :m] = gu[:, :m].clamp(-3, 3)
    _check_swiglu(_swiglu(gu), gu, "f32")


def test_rows_replay_in_a_graph_and_on_another_stream():
    from token_dynamic_expert_b200 import ace
    x, res, gamma = _rand((40, 512), "bf16", 20), _rand((40, 512), "bf16", 21), torch.rand(512, device="cuda")
    bufs = [dict(sum=torch.empty_like(x), y=torch.empty_like(x), q=torch.empty(40, 512, dtype=torch.int8, device="cuda"),
                 q_scale=torch.empty(40, device="cuda")) for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ace.ace_add_rmsnorm(x, gamma, residual=res, stream=st, **bufs[0])
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ace.ace_add_rmsnorm(x, gamma, residual=res, **bufs[1])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k in bufs[0]:
        assert torch.equal(bufs[0][k], bufs[1][k])
    _check_norm(bufs[0], x, gamma, res, "bf16")
