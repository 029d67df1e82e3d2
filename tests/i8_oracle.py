"""The 8-bit layer's operators in 64-bit numpy, written from their formulas,
for the tests.  Inputs are tensors on any device; results are numpy arrays."""
import numpy as np

U32 = 2.0 ** -24                     # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "f32": U32}  # half a step of the storage type


def f64(t):
    return t.detach().cpu().double().numpy()


def quantise(p, unit):
    """int8 rows of p and their scales; unit [rows] turns p into true values."""
    top = np.abs(p).max(1)
    safe = np.where(top > 0, top, 1.0)
    q = np.rint(p * 127.0 / safe[:, None])
    return np.where(top[:, None] > 0, q, 0.0), top * unit / 127.0


def norm(s, gamma, eps):
    """y, q, scale of stored sums s (64-bit values of the storage type)."""
    r = 1.0 / np.sqrt((s * s).mean(1) + eps)
    q, scale = quantise(s * gamma, r)
    return s * r[:, None] * gamma, q, scale


def swiglu(gu):
    m = gu.shape[1] // 2
    with np.errstate(over="ignore"):
        h = gu[:, :m] / (1.0 + np.exp(-gu[:, :m])) * gu[:, m:]
    return (h,) + quantise(h, np.ones(len(h)))


def gate(x, k, bias=None, score="softmax", n_groups=1, topk_groups=1, group_score="max",
         renorm=True, scale=1.0):
    """idx, weight by sorting, one token at a time."""
    T, E = x.shape
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = np.exp(-np.logaddexp(0.0, -x))
        else:
            top = x.max(1, keepdims=True)
            z = np.exp(x - np.where(np.isinf(top), 0.0, top))
            tot = z.sum(1, keepdims=True)
            s = z / np.where(tot > 0, tot, 1.0)
    n = E // n_groups
    idx, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        choice = s[t] if bias is None else s[t] + bias
        key = x[t] if bias is None else choice
        if group_score == "max":
            gv = key.reshape(n_groups, n).max(1)
        else:
            gv = np.sort(choice.reshape(n_groups, n), 1)[:, -2:].sum(1)
        first = sorted(range(n_groups), key=lambda g: (-gv[g], g))[:topk_groups]
        pool = [e for e in range(E) if e // n in first]
        idx[t] = sorted(pool, key=lambda e: (-key[e], e))[:k]
        w[t] = s[t][idx[t]]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, w * scale


def group(idx, keep, E):
    """offsets, slot_of, slot list (flat slots in position order)."""
    flat = idx.reshape(-1)
    on = (flat >= 0) & (flat < E)
    if keep is not None:
        on &= keep.reshape(-1) != 0
    slots = np.flatnonzero(on)
    slots = slots[np.lexsort((slots, flat[slots]))]
    offsets = np.zeros(E + 1, np.int64)
    offsets[1:] = np.cumsum(np.bincount(flat[slots], minlength=E))
    slot_of = np.full(flat.shape, -1, np.int64)
    slot_of[slots] = np.arange(len(slots))
    return offsets, slot_of.reshape(idx.shape), slots


def matmul(xq, xs, wq, ws, offsets=None, row_of=None, slot_scale=None, S=None):
    """[S][N] products; rows of slots beyond offsets[-1] are NaN."""
    w, wsc = (wq[None], ws[None]) if wq.ndim == 2 else (wq, ws)
    S = len(row_of) if row_of is not None else (S or len(xq))
    rows = np.arange(S) if row_of is None else row_of
    off = [0, S] if offsets is None else list(offsets)
    out = np.full((S, w.shape[1]), np.nan)
    for e in range(len(off) - 1):
        r = rows[off[e]:off[e + 1]]
        ok = (r >= 0) & (r < len(xq))
        rr = np.where(ok, r, 0)
        a = (xq[rr] @ w[e].T) * (np.where(ok, xs[rr], 0.0)[:, None] * wsc[e])
        out[off[e]:off[e + 1]] = a
    return out if slot_scale is None else out * slot_scale[:, None]


def close(got, ref, rel, tiny=0.0):
    """Largest |got - ref| in units of its allowance rel |ref| + tiny."""
    d = np.abs(got - ref)
    return float((d / (rel * np.abs(ref) + tiny + 1e-300)).max()) if d.size else 0.0
