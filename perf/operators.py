"""The operators of the 8-bit MoE layer, each as a measured case: the residual + RMSNorm with int8 output, the gate
(softmax / sigmoid scores, balance bias, groups, top-k), the grouping of slots by expert, the int8 matrix product
(dense and grouped by expert) and the SwiGLU with int8 output.

A case's fields: op, and then
  norm    T, d, dtype, residual
  gate    T, E, k, score, bias, groups, topk_groups, rule, renorm, dtype, masked
  group   T, E, k, skip (share of slots that are not kept)
  matmul  S, N, K, out; E (0: dense), gather (rows through a map), slot_scale, skew (spread of the experts' popularity)
  swiglu  S, m, dtype, y (also the unquantised result)
int8 results are returned as the values they stand for (q * scale), beside their scales."""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decode step through the norm before the MoE layer
        dict(name="norm_decode", op="norm", T=1, d=2048, dtype="bf16", residual=True),
        # a prefill of eight thousand tokens less one
        dict(name="norm_prefill", op="norm", T=8191, d=2048, dtype="bf16", residual=True),
        # one token routed over 128 experts, plain softmax top-8
        dict(name="gate_decode", op="gate", T=1, E=128, k=8, score="softmax", bias=False, groups=1, topk_groups=1,
             rule="max", renorm=True, dtype="f32", masked=False),
        # a prefill's tokens routed over 256 experts in 8 groups, balanced by a bias
        dict(name="gate_prefill", op="gate", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             rule="top2", renorm=True, dtype="f32", masked=False),
        # the slots of an odd number of tokens, some skipped
        dict(name="group_ragged", op="group", T=1003, E=128, k=8, skip=0.6),
        dict(name="group_prefill", op="group", T=8192, E=256, k=8, skip=0.0),
        # a dense projection in decode and in prefill
        dict(name="matmul_decode", op="matmul", S=8, N=2048, K=2048, out="bf16", E=0, gather=False, slot_scale=False,
             skew=0.0),
        dict(name="matmul_prefill", op="matmul", S=8191, N=4096, K=2048, out="bf16", E=0, gather=False,
             slot_scale=False, skew=0.0),
        # the experts' gate and up projections: 8 decoded tokens, and a prefill, rows read through the slots' tokens
        dict(name="experts_decode", op="matmul", S=64, N=1536, K=2048, out="bf16", E=128, gather=True,
             slot_scale=False, skew=0.5),
        dict(name="experts_prefill", op="matmul", S=65536, N=1024, K=2048, out="bf16", E=256, gather=True,
             slot_scale=False, skew=0.5),
        # the activation between the two products, for 8 decoded tokens less a few slots, and for a prefill
        dict(name="swiglu_decode", op="swiglu", S=61, m=768, dtype="bf16", y=False),
        dict(name="swiglu_prefill", op="swiglu", S=65536, m=512, dtype="bf16", y=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gate", "group", "matmul", "matmul", "swiglu"])
    if op == "norm":
        d = rng.choice([8 * _log(rng, 8, 1024), _log(rng, 64, 8192)])
        return dict(op=op, T=max(1, min(_log(rng, 1, 16384), (1 << 24) // d)), d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7)
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8, 6])
        per = rng.randint(max(2, 8 // groups), 512 // groups)
        topk_groups = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384), E=groups * per, k=rng.randint(1, min(16, topk_groups * per)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                    topk_groups=topk_groups, rule=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.25)
    if op == "group":
        E = _log(rng, 2, 512)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(16, E)),
                    skip=rng.choice([0.0, 0.25, 0.6, 0.9]))
    if op == "swiglu":
        m = rng.choice([8 * _log(rng, 8, 512), _log(rng, 32, 4096)])
        return dict(op=op, S=max(1, min(_log(rng, 1, 65536), (1 << 25) // m)), m=m,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), y=rng.random() < 0.3)
    K = 16 * _log(rng, 8, 256)
    N = _log(rng, 64, 4096)
    E = rng.choice([0, 0, _log(rng, 4, 256)])
    S = max(1, min(_log(rng, 1, 65536 if E else 16384), int(6e10 / (N * K))))
    return dict(op=op, S=S, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]), E=E, gather=bool(E) and rng.random() < 0.6,
                slot_scale=bool(E) and rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))


def work(c):
    op, es = c["op"], 2 if c.get("dtype", c.get("out")) == "bf16" else 4
    if op == "norm":
        n = c["T"] * c["d"]
        return dict(bytes=n * ((3 if c["residual"] else 1) * es + es + 1) + 4 * (c["d"] + c["T"]), flops=8 * n)
    if op == "gate":
        return dict(bytes=c["T"] * (c["E"] * es + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0),
                    flops=c["T"] * c["E"] * 8)
    if op == "group":
        return dict(bytes=c["T"] * c["k"] * (9 + 4) + round(c["T"] * c["k"] * (1 - c["skip"])) * 8 + 4 * c["E"] + 4,
                    flops=2 * c["T"] * c["k"])
    if op == "swiglu":
        return dict(bytes=c["S"] * c["m"] * (2 * es + 1 + (es if c["y"] else 0)) + 4 * c["S"],
                    flops=6 * c["S"] * c["m"])
    S, N, K, E = c["S"], c["N"], c["K"], max(c["E"], 1)
    used = E * (1 - (1 - 1 / E) ** S)  # experts that some slot uses, for even popularity
    rows = (S + 7) // 8 if c["gather"] else S
    return dict(bytes=used * N * (K + 4) + rows * (K + 4) + S * (N * es + (4 if c["gather"] else 0)), flops=2 * S * N * K)


# ----------------------------------------------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, st = c["op"], dict(c)
    dev = dict(device="cuda")
    if op == "norm":
        T, d, dt = c["T"], c["d"], DTYPE[c["dtype"]]
        channel = torch.exp(0.5 * _normal(g, d))  # channels of unlike size, as a residual stream has
        st["x"] = (_normal(g, T, d) * channel).to(dt)
        st["res"] = (_normal(g, T, d) * channel * 2).to(dt) if c["residual"] else None
        st["gamma"] = torch.rand(d, generator=g, **dev) + 0.5
        st["sum"] = torch.empty(T, d, dtype=dt, **dev) if c["residual"] else None
        st["yb"] = torch.empty(T, d, dtype=dt, **dev)
        st["q"], st["qs"] = torch.empty(T, d, dtype=torch.int8, **dev), torch.empty(T, **dev)
    elif op == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        x = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, E)
        if c["masked"]:  # experts that are out of service for some tokens; the last token has none
            x = torch.where(torch.rand(T, E, generator=g, **dev) < 0.2, -math.inf, x)
            x[T - 1] = -math.inf
        st["x"] = x.to(DTYPE[c["dtype"]])
        st["b"] = 0.1 * _normal(g, E) if c["bias"] else None
        st["idx"] = torch.empty(T, k, dtype=torch.int32, **dev)
        st["w"] = torch.empty(T, k, **dev)
    elif op == "group":
        T, E, k = c["T"], c["E"], c["k"]
        pop = 0.5 * _normal(g, E) - torch.log(-torch.log(torch.rand(T, E, generator=g, **dev).clamp(1e-9, 1 - 1e-6)))
        st["idx"] = torch.topk(pop, k, 1).indices.to(torch.int32)
        st["gate"] = torch.rand(T, k, generator=g, **dev)
        low = torch.rand(T, k, generator=g, **dev)  # the slots of the lowest scores are skipped, never a token's first
        low[:, 0] = 2.0
        skipped = torch.topk(low.view(-1), min(round(T * k * c["skip"]), T * (k - 1)), largest=False).indices
        st["keep"] = torch.ones(T * k, dtype=torch.uint8, **dev).index_fill_(0, skipped, 0).view(T, k)
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, **dev)
        st["slot_of"] = torch.empty(T, k, dtype=torch.int32, **dev)
        st["n"] = T * k - len(skipped)
        st["slot_token"] = torch.empty(T * k, dtype=torch.int32, **dev)
        st["slot_gate"] = torch.empty(T * k, **dev)
    elif op == "matmul":
        S, N, K, E = c["S"], c["N"], c["K"], max(c["E"], 1)
        R = (S + 7) // 8 if c["gather"] else S
        st["xq"] = (_normal(g, R, K) * 36).round().clamp(-127, 127).to(torch.int8)
        st["xs"] = (torch.rand(R, generator=g, **dev) + 0.5) / 36
        st["wq"] = (_normal(g, E, N, K) * 36).round().clamp(-127, 127).to(torch.int8)
        st["ws"] = (torch.rand(E, N, generator=g, **dev) + 0.5) * (0.02 / 36)
        if not c["E"]:
            st["wq"], st["ws"] = st["wq"][0], st["ws"][0]
        e = torch.multinomial(torch.softmax(c["skew"] * _normal(g, E), 0), S, replacement=True, generator=g)
        count = torch.bincount(e, minlength=E)
        off = torch.zeros(E + 1, dtype=torch.int64, **dev)
        off[1:] = torch.cumsum(count, 0)
        st["offsets"], st["cap"] = off.to(torch.int32), int(count.max())
        st["row_of"] = torch.randint(0, R, (S,), generator=g, **dev).to(torch.int32) if c["gather"] else None
        st["ss"] = torch.rand(S, generator=g, **dev) if c["slot_scale"] else None
        st["y"] = torch.empty(S, N, dtype=DTYPE[c["out"]], **dev)
        st["scratch"] = torch.empty(4096, dtype=torch.uint8, **dev)
    else:
        S, m, dt = c["S"], c["m"], DTYPE[c["dtype"]]
        st["gu"] = (2 * _normal(g, S, 2 * m)).to(dt)
        st["yb"] = torch.empty(S, m, dtype=dt, **dev) if c["y"] else None
        st["q"], st["qs"] = torch.empty(S, m, dtype=torch.int8, **dev), torch.empty(S, **dev)
    return st


def _given(**outputs):
    return {name: v for name, v in outputs.items() if v is not None}


# ------------------------------------------------------------------------------------------------------ plain forms
def _quantise(p, unit):
    """int8 rows of p (64 bits: a quotient next to a half decides a whole step) as the values they stand for, and the
    scales; unit scales p to the true values."""
    top = p.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(p * 127 / top), 0.0)
    scale = (top * unit / 127).float()
    return q.float() * scale, scale[:, 0]


def _norm(st):
    s = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(st["x"].dtype)
    f = s.float()
    r = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-6)
    deq, scale = _quantise(f.double() * st["gamma"].double(), r.double())
    return _given(sum=s if st["sum"] is not None else None, y=(f * r * st["gamma"]).to(s.dtype), q=deq, scale=scale)


def _gate(st):
    x = st["x"].double()  # 64 bits: which of two nearly equal scores is the larger
    if st["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        z = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        total = z.sum(1, keepdim=True)
        s = torch.where(total > 0, z / total, 0.0)
    choice = s if st["b"] is None else s + st["b"].double()
    key = x if st["b"] is None else choice
    T, E, G = x.shape[0], x.shape[1], st["groups"]
    if st["rule"] == "max":
        group = key.view(T, G, -1).amax(2)
    else:
        group = choice.view(T, G, -1).topk(2, 2).values.sum(2)
    best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :st["topk_groups"]]
    allowed = torch.zeros_like(group).scatter_(1, best, 1.0).repeat_interleave(E // G, 1)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(allowed.gather(1, order), dim=1, descending=True, stable=True).indices)
    idx = order[:, :st["k"]]
    w = s.gather(1, idx)
    if st["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return dict(idx=idx.to(torch.int32), weight=w.float())


def _group(st):
    T, k = st["idx"].shape
    kept, expert = st["keep"].view(-1) != 0, st["idx"].view(-1).long()
    order = torch.sort(torch.where(kept, expert, st["E"]), stable=True).indices[:st["n"]]
    offsets = torch.zeros(st["E"] + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.zeros(st["E"] + 1, dtype=torch.int64, device="cuda").scatter_add_(
        0, torch.where(kept, expert, st["E"]), torch.ones_like(expert))[:-1], 0)
    slot_of = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    slot_of[order] = torch.arange(st["n"], dtype=torch.int32, device="cuda")
    return dict(offsets=offsets.to(torch.int32), slot_token=(order // k).to(torch.int32), slot_of=slot_of.view(T, k),
                slot_gate=st["gate"].view(-1)[order])


def _matmul(st):
    x = st["xq"].float()  # whole numbers below 2^24: their sums are exact in 32 bits
    xs = st["xs"]
    if st["row_of"] is not None:
        x, xs = x[st["row_of"].long()], xs[st["row_of"].long()]
    if not st["E"]:
        acc, ws = x @ st["wq"].float().t(), st["ws"]
    else:
        s = torch.arange(st["S"], device="cuda")
        expert = torch.searchsorted(st["offsets"][1:].contiguous(), s.to(torch.int32), right=True)
        ws = st["ws"][expert]
        if st["S"] <= 64:  # each slot with its expert's matrix
            acc = (st["wq"][expert].float() @ x[:, :, None])[:, :, 0]
        else:  # each expert with its slots, filled up to the largest expert's number
            at = s - st["offsets"][expert].long()
            xe = torch.zeros(st["E"], st["cap"], st["K"], device="cuda")
            xe[expert, at] = x
            acc = torch.bmm(xe, st["wq"].float().transpose(1, 2))[expert, at]
    if st["ss"] is not None:
        xs = xs * st["ss"]
    return (acc * (xs[:, None] * ws)).to(DTYPE[st["out"]])


def _swiglu(st):
    m = st["m"]
    v = st["gu"].double()  # 64 bits, as in _quantise
    h = v[:, :m] / (1 + torch.exp(-v[:, :m])) * v[:, m:]
    deq, scale = _quantise(h, 1.0)
    return _given(y=h.float().to(st["gu"].dtype) if st["y"] else None, q=deq, scale=scale)


def run(st):
    op = st["op"]
    if not own:
        return {"norm": _norm, "gate": _gate, "group": _group, "matmul": _matmul, "swiglu": _swiglu}[op](st)
    from token_dynamic_expert_b200 import ace
    if op == "norm":
        ace.ace_add_rmsnorm(st["x"], st["gamma"], residual=st["res"], sum=st["sum"], y=st["yb"], q=st["q"],
                            q_scale=st["qs"], eps=1e-6)
        return _given(sum=st["sum"], y=st["yb"], q=st["q"] * st["qs"][:, None], scale=st["qs"])
    if op == "gate":
        ace.ace_gate_topk(st["x"], st["idx"], st["w"], bias=st["b"], score=st["score"], n_groups=st["groups"],
                          topk_groups=st["topk_groups"], group_score=st["rule"], renorm=st["renorm"])
        return dict(idx=st["idx"], weight=st["w"])
    if op == "group":
        ace.ace_moe_group(st["idx"], st["E"], st["offsets"], st["slot_of"], keep=st["keep"], gate=st["gate"],
                          slot_token=st["slot_token"], slot_gate=st["slot_gate"])
        return dict(offsets=st["offsets"], slot_token=st["slot_token"][:st["n"]], slot_of=st["slot_of"],
                    slot_gate=st["slot_gate"][:st["n"]])
    if op == "matmul":
        return ace.ace_matmul_i8(st["xq"], st["xs"], st["wq"], st["ws"], st["y"], st["scratch"],
                                 offsets=st["offsets"] if st["E"] else None, row_of=st["row_of"],
                                 slot_scale=st["ss"])
    ace.ace_swiglu(st["gu"], y=st["yb"], q=st["q"], q_scale=st["qs"])
    return _given(y=st["yb"], q=st["q"] * st["qs"][:, None], scale=st["qs"])


# --------------------------------------------------------------------------------------- the definitions in 64 bits
def exact(c, seed):
    """The definitions once more: rows by their own arithmetic in 64 bits, tokens and slots one by one where order
    matters."""
    import numpy as np
    st = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        s = st["x"].cpu()
        if c["residual"]:
            s = torch.add(s.double(), st["res"].cpu().double()).to(s.dtype)
        v = s.double().numpy()
        gamma = st["gamma"].cpu().double().numpy()
        root = np.sqrt(np.einsum("ij,ij->i", v, v) / c["d"] + 1e-6)
        v *= gamma
        peak = np.maximum(v.max(1), -v.min(1))
        q = np.rint(v * 127.0 / np.where(peak > 0, peak, 1.0)[:, None])
        scale = peak / root / 127
        return _given(sum=torch.from_numpy(s.double().numpy()) if c["residual"] else None,
                    y=torch.from_numpy(v / root[:, None]), q=torch.from_numpy(q * scale[:, None]),
                    scale=torch.from_numpy(scale))
    if op == "swiglu":
        v = st["gu"].cpu().double().numpy()
        g, u = v[:, :c["m"]], v[:, c["m"]:]
        h = g * u
        h /= 1 + np.exp(-g)
        peak = np.maximum(h.max(1), -h.min(1))
        q = np.rint(h * 127.0 / np.where(peak > 0, peak, 1.0)[:, None])
        return _given(y=torch.from_numpy(h) if c["y"] else None, q=torch.from_numpy(q * (peak / 127)[:, None]),
                    scale=torch.from_numpy(peak / 127))
    if op == "matmul":
        w = st["wq"].reshape(max(c["E"], 1), c["N"], c["K"])
        wsc = st["ws"].reshape(max(c["E"], 1), c["N"]).double()
        rows = torch.arange(c["S"], device="cuda") if st["row_of"] is None else st["row_of"].long()
        out = torch.empty(c["S"], c["N"], dtype=torch.float64, device="cuda")
        off = st["offsets"].tolist() if c["E"] else [0, c["S"]]
        for e in range(len(off) - 1):
            r = rows[off[e]:off[e + 1]]
            if len(r):
                scaled = st["xq"][r].double() * st["xs"][r].double()[:, None]
                out[off[e]:off[e + 1]] = (scaled @ w[e].double().t()) * wsc[e]
        if st["ss"] is not None:
            out *= st["ss"].double()[:, None]
        return out
    if op == "gate":
        x = st["x"].cpu().double().numpy()
        b = None if st["b"] is None else st["b"].cpu().double().numpy()
        T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
        n = E // G
        with np.errstate(all="ignore"):
            if c["score"] == "sigmoid":
                s = np.exp(-np.logaddexp(0.0, -x))
            else:
                s = np.exp(x - np.where(np.isinf(x.max(1)), 0.0, x.max(1))[:, None])
                s /= np.where(s.sum(1) > 0, s.sum(1), 1.0)[:, None]
        weight = np.zeros((T, k))
        for t in range(T):
            key = x[t] if b is None else s[t] + b
            pick = s[t] if b is None else key
            if c["rule"] == "max":
                rank = key.reshape(G, n).max(1)
            else:
                rank = np.sort(pick.reshape(G, n), 1)[:, -2:].sum(1)
            first = np.lexsort((np.arange(G), -rank))[:c["topk_groups"]]
            members = np.sort((first[:, None] * n + np.arange(n)).reshape(-1))
            chosen = members[np.lexsort((members, -key[members]))[:k]]
            weight[t] = s[t][chosen]
            if c["renorm"]:
                weight[t] /= weight[t].sum() or 1.0
        return dict(idx=None, weight=torch.from_numpy(weight))
    expert = st["idx"].cpu().numpy().reshape(-1)
    at = np.flatnonzero(st["keep"].cpu().numpy().reshape(-1))
    at = at[np.lexsort((at, expert[at]))]
    return dict(offsets=None, slot_token=None, slot_of=None, slot_gate=st["gate"].cpu().double().view(-1)[torch.from_numpy(at)])
