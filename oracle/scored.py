"""Plain fp64 statements of scored gates and of experts in 8-bit integers -- TEST INFRASTRUCTURE ONLY."""
import numpy as np

from .moe import as_f64, silu


def gate_scores(l, score):
    """softmax over all experts or sigmoid, row by row; a NaN logit counts as -inf."""
    l = np.asarray(l, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        z = np.where(l == m, 1.0, np.exp(l - m))
    return z / z.sum(1, keepdims=True)


def gate_select(l, k, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, balance=None):
    """(idx [T, k], w [T, k]) of the gate: one token and one expert after another, in Python."""
    s = gate_scores(l, score)
    T, E = s.shape
    with np.errstate(invalid="ignore"):
        c = s + (0.0 if balance is None else as_f64(balance)[None, :])
    c = np.where(np.isnan(c), -np.inf, c)
    per = E // n_group
    idx = np.empty((T, k), np.int64)
    w = np.empty((T, k))
    for t in range(T):
        ranks = []
        for g in range(n_group):
            best = sorted((c[t, e] for e in range(g * per, (g + 1) * per)), reverse=True)
            with np.errstate(invalid="ignore"):
                r = best[0] + best[1] if group_top == 2 and per > 1 else best[0]
            ranks.append(-np.inf if np.isnan(r) else r)
        kept = sorted(range(n_group), key=lambda g: (-ranks[g], g))[:topk_group]
        pool = [e for e in range(E) if e // per in kept]
        idx[t] = sorted(pool, key=lambda e: (-c[t, e], e))[:k]
        w[t] = s[t, idx[t]]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, w * np.float64(np.float32(scale))


def quantise_rows(a):
    """(codes, scale) of the rows of a [M, K]: codes rne(127 v / max|v|) exactly, scale max|v| / 127."""
    a = as_f64(a)
    m = np.abs(a).max(1)
    safe = np.where(m > 0, m, 1.0)
    # 127 v is exact for fp32 values, and a quotient of two values of 24 bits that is not a half is at least
    # 2^-33 from one, so rounding the fp64 quotient decides as the exact one would
    return np.rint(a * 127.0 / safe[:, None]), m / 127.0


def int8_expert(X, q1, q3, q2, s1, s3, s2):
    """dict of an int8 expert's values on rows X: h, its codes hq and scale sh, and y."""
    xq, sx = quantise_rows(X)
    q1, q3, q2 = as_f64(q1), as_f64(q3), as_f64(q2)
    g = (xq @ q1) * sx[:, None] * as_f64(s1)[None, :]
    u = (xq @ q3) * sx[:, None] * as_f64(s3)[None, :]
    h = silu(g) * u
    hq, sh = quantise_rows(h)
    return dict(h=h, hq=hq, sh=sh, y=(hq @ q2) * sh[:, None] * as_f64(s2)[None, :])
