"""ace_gate_topk against 64-bit sorting: the chosen experts are equal, also
where scores nearly or exactly tie.  Weights: the difference of two logits is
rounded to fp32 (|difference| half steps in the exponent), expf 2 ulp (4 half
steps), the sum of at most 16 terms over 5 shuffles 5, quotient and scale 2; for
numerator and sum both.  (2 D + 20) half steps for logits up to D apart."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _run(x, k, bias=None, **kw):
    from token_dynamic_expert_b200 import ace
    T = x.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    ace.ace_gate_topk(x, idx, w, bias=bias, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().double().numpy()


def _check(x, k, bias=None, **kw):
    idx, w = _run(x, k, bias, **kw)
    ridx, rw = ora.gate(ora.f64(x), k, None if bias is None else ora.f64(bias), **kw)
    assert np.array_equal(idx, ridx)
    v = ora.f64(x)
    v = v[np.isfinite(v)]
    D = float(v.max() - v.min()) if v.size else 0.0
    assert ora.close(w, rw, (2 * D + 20) * ora.U32, 1e-37) <= 1


def _logits(T, E, dt, seed, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(T, E, generator=g, device="cuda")).to(DT[dt])


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (31, 5), (32, 8), (33, 16), (60, 4), (128, 8),
                                 (256, 8), (300, 16), (512, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_sizes(E, k, score, biased):
    for dt in ("f32", "bf16"):
        x = _logits(67, E, dt, E + k)
        bias = 0.2 * torch.randn(E, device="cuda") if biased else None
        _check(x, k, bias, score=score)
        _check(x, k, bias, score=score, renorm=False, scale=2.5)


@pytest.mark.parametrize("E,G,tg,k", [(16, 2, 1, 8), (64, 8, 3, 8), (256, 8, 4, 8), (256, 32, 5, 16),
                                      (512, 16, 2, 16), (60, 6, 2, 5), (510, 17, 4, 16), (9, 9, 4, 4),
                                      (500, 5, 1, 16), (96, 3, 3, 7), (62, 31, 8, 16)])
@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, G, tg, k, rule, score):
    for dt, biased in (("f32", True), ("f32", False), ("bf16", True), ("bf16", False)):
        x = _logits(53, E, dt, E + G)
        bias = 0.3 * torch.randn(E, device="cuda") if biased else None
        _check(x, k, bias, score=score, n_groups=G, topk_groups=tg, group_score=rule)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 1000])
def test_token_counts(T):
    _check(_logits(T, 128, "f32", T), 8)


def test_many_tokens_with_bias_and_groups():
    _check(_logits(4096, 256, "f32", 99), 8, 0.1 * torch.randn(256, device="cuda"), score="sigmoid",
           n_groups=8, topk_groups=4, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rule", ["max", "top2"])
def test_ties_go_to_the_lower_index(score, rule):
    x = _logits(200, 64, "f32", 5)
    x = (x * 2).round() / 2                      # many equal logits
    for bias in (None, torch.zeros(64, device="cuda"), (torch.arange(64, device="cuda") % 2) * 0.125):
        _check(x, 8, bias, score=score)
        _check(x, 8, bias, score=score, n_groups=8, topk_groups=3, group_score=rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_fp32_can_tell(score):
    """Experts whose biased scores differ by 1e-12 to 1e-6: the bias undoes the
    difference of the scores up to its own rounding."""
    g = torch.Generator(device="cuda").manual_seed(3)
    E = 96
    x0 = torch.randn(E, generator=g, device="cuda")
    s = torch.softmax(x0.double(), 0) if score == "softmax" else torch.sigmoid(x0.double())
    bias = (0.5 - s).float()                     # every c within an fp32 step of 0.5
    x = x0 + torch.randn(300, E, generator=g, device="cuda") * 1e-6
    _check(x, 8, bias, score=score)
    for rule in ("max", "top2"):
        _check(x, 8, bias, score=score, n_groups=8, topk_groups=3, group_score=rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_chains_of_equal_and_nearly_equal_scores_across_the_border(score):
    """A few distinct values, an fp32 step or less apart in their choice value, each
    held by several experts: ties and near ties on both sides of rank k."""
    g = torch.Generator(device="cuda").manual_seed(21)
    E, T = 48, 400
    which = torch.randint(0, 6, (T, E), generator=g, device="cuda")
    x = torch.tensor([0.5, 0.5 + 2.0 ** -23, 0.5 + 2.0 ** -22, 0.5 - 2.0 ** -24, 0.25, -1.0], device="cuda")[which]
    x[:, 40:] -= 3
    for bias in (torch.zeros(E, device="cuda"), (torch.arange(E, device="cuda") % 3) * 2.0 ** -25):
        for k in (1, 2, 5, 8, 16):
            _check(x, k, bias, score=score)
            _check(x, min(k, 12), bias, score=score, n_groups=4, topk_groups=2, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("lowest", [-float("inf"), torch.finfo(torch.float32).min])
def test_masked_experts(score, biased, lowest):
    """Masked experts, down to fewer than k left and to none."""
    E, k = 64, 8
    x = _logits(70, E, "f32", 8)
    for t in range(65):
        x[t, torch.randperm(E)[:t]] = lowest
    x[65:] = lowest
    bias = 0.1 * torch.randn(E, device="cuda") if biased else None
    kw = dict(score=score, n_groups=4, topk_groups=2, group_score="top2")
    for args in (dict(score=score), dict(score=score, renorm=False), kw):
        idx, w = _run(x, k, bias, **args)
        ridx, rw = ora.gate(ora.f64(x), k, None if bias is None else ora.f64(bias), **args)
        assert np.array_equal(idx, ridx)
        if lowest == -float("inf"):
            assert ora.close(w, rw, 60 * ora.U32, 1e-37) <= 1
            if not biased:
                assert (w[65:] == 0).all()
        assert np.isfinite(w).all()


def test_sigmoid_far_from_zero_keeps_its_ratios():
    """All scores far below fp32's range: weights are still their ratios."""
    x = _logits(40, 32, "f32", 4) - 150.0
    _check(x, 4, score="sigmoid")
    _check(_logits(40, 32, "f32", 4) + 60.0, 4, score="sigmoid")


def test_nan_takes_the_token_only():
    x = _logits(6, 40, "f32", 6)
    ref, rw = _run(x, 4)
    x[2, 11] = float("nan")
    x[3, 7] = -float("nan")
    idx, w = _run(x, 4)
    others = [0, 1, 4, 5]
    assert np.array_equal(idx[others], ref[others]) and np.array_equal(w[others], rw[others])
    assert idx[2, 0] == 11 and idx[3, 0] == 7 and np.isnan(w[2]).all() and np.isnan(w[3]).all()
    assert ((idx >= 0) & (idx < 40)).all()


def test_keep_is_the_skip_rule_on_the_weights():
    from token_dynamic_expert_b200 import ace
    x = _logits(500, 64, "f32", 12)
    bias = torch.randn(64, device="cuda")        # the first slot need not hold the largest weight
    factor = torch.rand(64, device="cuda") + 0.5
    idx = torch.empty(500, 8, dtype=torch.int32, device="cuda")
    w, keep = torch.empty(500, 8, device="cuda"), torch.empty(500, 8, dtype=torch.uint8, device="cuda")
    ace.ace_gate_topk(x, idx, w, bias=bias, score="sigmoid", factor=factor, tau=0.12, keep=keep)
    c = w * factor[idx.long()]
    want = ~(c < 0.12)
    want[torch.arange(500), w.argmax(1)] = True  # argmax: the first of equals on these distinct weights
    assert torch.equal(keep != 0, want) and 0.2 < want.float().mean() < 0.9
    assert (w.argmax(1) != 0).any()


def test_strided_logits_and_graph_replay():
    from token_dynamic_expert_b200 import ace
    wide = _logits(33, 400, "f32", 13)
    for lo, E in ((0, 256), (3, 256), (4, 128)):
        _check(wide[:, lo:lo + E], 8, 0.1 * torch.randn(E, device="cuda"), score="sigmoid", n_groups=8,
               topk_groups=4, group_score="top2")
    x = wide[:, :256].contiguous()
    idx, w = torch.empty(33, 8, dtype=torch.int32, device="cuda"), torch.empty(33, 8, device="cuda")
    ace.ace_gate_topk(x, idx, w)
    i0, w0 = idx.clone(), w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ace.ace_gate_topk(x, idx, w)
    idx.zero_(), w.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, i0) and torch.equal(w, w0)


def test_agrees_with_the_layers_own_routing():
    """Softmax without bias or groups is ace_moe_route's choice and gates, from
    the logits of its own forward."""
    import workloads
    from token_dynamic_expert_b200 import ace
    w = workloads.Workload("g", T=200, d=256, E=64, m=128, k=6, dtype="bf16", bias=False, skip=0.5,
                           skip_of="slots")
    layer = workloads.make_layer(w, seed=3, device="cuda")
    u = workloads.make_tokens(w, token_seed=7, device="cuda")
    L = ace.make_layer(layer["gamma"], layer["wr"], layer["wg"], layer["wu"], layer["wd"], w.k)
    ws = ace.alloc_workspace(ace.ace_workspace_size(L, w.T))
    dbg = ace.DebugOut(w.T, w.k, w.E)
    ace.ace_moe_forward(L, u, 0.0, torch.empty_like(u), ws, dbg=dbg.c)
    idx, wt = _run(dbg.logits, w.k)
    assert np.array_equal(idx, dbg.topk_idx.cpu().numpy())
    assert np.allclose(wt, ora.f64(dbg.gate), rtol=1e-6, atol=0)
