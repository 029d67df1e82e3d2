"""ace_gate_topk on tokens that hold NaN or infinite logits and biases: the
experts are those of a sort in 64 bits in which NaN stands above +infinity, and none
is named twice."""
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
    got = idx.cpu().numpy()
    ri, _ = _gate(ora.f64(x), k, None if bias is None else ora.f64(bias), score, G, tg, rule, renorm, scale)
    assert np.array_equal(got, ri)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg", [(1, 1)])
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
