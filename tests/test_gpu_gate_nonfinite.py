"""ace_gate_topk on tokens that hold NaN or infinite logits and biases: the
experts are those of a sort in 64 bits in which NaN stands above +infinity, none is
named twice, and a NaN logit (with softmax a +infinity too) makes the token's
weights NaN."""
import itertools

import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def _order(v):
    """Indices by value, largest first: NaN above +infinity, ties to the lower."""
    return sorted(range(len(v)), key=lambda i: (not np.isnan(v[i]), -v[i] if v[i] == v[i] else 0.0, i))


def _gate(x, k, bias, score, G, tg, rule, renorm, scale):
    T, E = x.shape
    n = E // G
    idx, w = np.zeros((T, k), np.int64), np.full((T, k), np.nan)
    for t in range(T):
        l = x[t]
        off = np.isnan(l) | ((l == INF) if score == "softmax" else False)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = np.exp(-np.logaddexp(0.0, -l))
            elif off.any():
                s = np.zeros(E)
            else:
                z = np.exp(l - (l.max() if l.max() > -INF else 0.0))
                s = z / (z.sum() if z.sum() > 0 else 1.0)
            s = np.where(off, NAN, s)
            c = s if bias is None else s + bias
            key = l if bias is None else c
            if rule == "max" or n == 1:  # a group of one counts as its expert
                gv = [max(key[g * n:(g + 1) * n], key=lambda v: (np.isnan(v), v)) for g in range(G)]
            else:
                gv = []
                for g in range(G):
                    part = c[g * n:(g + 1) * n]
                    a, b = _order(part)[:2]
                    gv.append(part[a] + part[b])
        allowed = set(_order(np.array(gv))[:tg])
        idx[t] = [e for e in _order(key) if e // n in allowed][:k]
        if not off.any():
            p = s[idx[t]]
            w[t] = scale * (p if not renorm else p / p.sum() if p.sum() > 0 else 0 * p)
    return idx, w


def _check(x, k, bias=None, score="softmax", G=1, tg=1, rule="max", renorm=True, scale=1.0):
    from token_dynamic_expert_b200 import ace
    T, E = x.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    keep = torch.full((T, k), 9, dtype=torch.uint8, device="cuda")
    factor = torch.rand(E, device="cuda") + 0.5
    ace.ace_gate_topk(x, idx, w, bias=bias, score=score, n_groups=G, topk_groups=tg, group_score=rule,
                      renorm=renorm, scale=scale, factor=factor, tau=0.05, keep=keep)
    got, gw = idx.cpu().numpy(), w.cpu().double().numpy()
    ri, rw = _gate(ora.f64(x), k, None if bias is None else ora.f64(bias), score, G, tg, rule, renorm, scale)
    assert np.array_equal(got, ri)
    assert np.array_equal(np.isnan(gw), np.isnan(rw))
    v = ora.f64(x)
    v = v[np.isfinite(v)]
    ok = ~np.isnan(rw)  # the bound of the finite tokens' tests
    assert ora.close(gw[ok], rw[ok], (2 * (v.max() - v.min()) + 20) * ora.U32, 1e-37) <= 1
    # the skip rule: NaN is not below tau, and the largest of the others is kept
    want = ~(w * factor[idx.long()] < 0.05).cpu().numpy()
    want[np.arange(T), np.where(np.isnan(gw), INF, gw).argmax(1)] = True  # numpy: the first of equals
    assert np.array_equal(keep.cpu().numpy() != 0, want)


def _tokens(E, G, value, dt, seed):
    """A token for each place of one value within the first, a middle and the last
    group, then pairs of places, then tokens without any."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = E // G
    at = [(gr * n + i,) for gr in sorted({0, G // 2, G - 1}) for i in range(n)]
    at += [(0, E - 1), (n - 1, E - n), (E // 2, E // 2 - 1), (), ()]
    x = (1.5 * torch.randn(len(at), E, generator=g, device="cuda")).to(dt)
    for t, es in enumerate(at):
        for e in es:
            x[t, e] = value
    return x


GROUPS = [(64, 8, 1, 8), (64, 8, 3, 8), (16, 2, 1, 8), (60, 6, 2, 16), (256, 8, 4, 8), (9, 9, 4, 4), (510, 17, 1, 16),
          (64, 2, 1, 8), (96, 1, 1, 16)]


@pytest.mark.parametrize("E,G,tg,k", GROUPS)
@pytest.mark.parametrize("value", [NAN, -NAN, INF, -INF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_logit_at_every_place_of_a_group(E, G, tg, k, value, score):
    for rule, biased, dt in itertools.product(("max", "top2"), (False, True), (torch.float32, torch.bfloat16)):
        x = _tokens(E, G, value, dt, E + G)
        bias = 0.3 * torch.randn(E, device="cuda") if biased else None
        _check(x, k, bias, score, G, tg, rule)
        _check(x, k, bias, score, G, tg, rule, renorm=False, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("rule", ["max", "top2"])
def test_many_nan_and_infinite_logits(score, rule):
    """Up to every logit of a token, of all four kinds."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(400, 64, generator=g, device="cuda")
    share = torch.linspace(0, 1, 400, device="cuda")[:, None]
    which = torch.randint(0, 4, x.shape, generator=g, device="cuda")
    odd = torch.tensor([NAN, -NAN, INF, -INF], device="cuda")[which]
    x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < share, odd, x)
    for bias in (None, 0.1 * torch.randn(64, device="cuda")):
        for tg in (1, 3):
            _check(x, 8, bias, score, 8, tg, rule)
            _check(x, 8, bias, score, 8, tg, rule, renorm=False)
        _check(x, 16, bias, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg", [(1, 1), (8, 1), (8, 3)])
def test_nan_beside_scores_closer_than_fp32_can_tell(score, G, tg):
    """The bias undoes the scores' differences, so that fp64 orders the experts: the
    NaN one among them keeps its place at the top."""
    g = torch.Generator(device="cuda").manual_seed(3)
    E = 96
    x0 = torch.randn(E, generator=g, device="cuda")
    s = torch.softmax(x0.double(), 0) if score == "softmax" else torch.sigmoid(x0.double())
    bias = (0.5 - s).float()
    x = x0 + torch.randn(200, E, generator=g, device="cuda") * 1e-6
    for t in range(150):
        x[t, (7 * t) % E] = (NAN, -NAN, INF)[t % 3]
    for k in (1, 8, 12):
        for rule in ("max", "top2"):
            _check(x, k, bias, score, G, tg, rule)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [NAN, INF, -INF, 3.4e38, -3.4e38])
def test_a_bias_that_is_not_finite_or_overflows_a_sum(score, value):
    """A NaN of the bias takes part in the choice alone: weights stay finite."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(60, 64, generator=g, device="cuda")
    for where in ((0,), (7, 8), (0, 1, 2), (63,), (8, 9, 16, 17, 40, 41)):
        bias = 0.1 * torch.randn(64, generator=g, device="cuda")
        bias[list(where)] = value
        for rule in ("max", "top2"):
            for tg in (1, 3):
                _check(x, 8, bias, score, 8, tg, rule)
        _check(x, 8, bias, score, renorm=False)


def test_the_experts_feed_the_grouping():
    """Every slot of a token with a NaN is an expert's: grouping loses none."""
    from token_dynamic_expert_b200 import ace
    x = _tokens(64, 8, NAN, torch.float32, 1)
    T = x.shape[0]
    idx, w = torch.empty(T, 8, dtype=torch.int32, device="cuda"), torch.empty(T, 8, device="cuda")
    ace.ace_gate_topk(x, idx, w, n_groups=8, topk_groups=1)
    off = torch.empty(65, dtype=torch.int32, device="cuda")
    ace.ace_moe_group(idx, 64, off, torch.empty_like(idx))
    assert int(off[-1]) == T * 8
    assert (torch.sort(idx, 1).values.diff(dim=1) > 0).all()
