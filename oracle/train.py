"""Plain fp64 statements of the operators that train through the layer -- TEST INFRASTRUCTURE ONLY."""
import numpy as np

from .moe import as_f64


def group(idx, E):
    """(counts, offsets, pos [T, k], src) of given choices; entries outside [0, E) are dropped (pos -1)."""
    idx = np.asarray(idx)
    pos = np.full(idx.shape, -1, np.int64)
    rows = [[] for _ in range(E)]
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            if 0 <= idx[t, j] < E:
                rows[idx[t, j]].append((t, j))
    counts = np.array([len(r) for r in rows], np.int64)
    order = [tj for r in rows for tj in r]
    for p, (t, j) in enumerate(order):
        pos[t, j] = p
    return counts, np.concatenate([[0], np.cumsum(counts)]), pos, np.array([t for t, _ in order], np.int64)


def collect(rows, pos, w=None):
    """out[t] = sum_j w[t, j] rows[pos[t, j]]; entries outside the rows have none."""
    rows = as_f64(rows)
    out = np.zeros((pos.shape[0], rows.shape[1]))
    for t, j in np.argwhere((pos >= 0) & (pos < len(rows))):
        out[t] += (1.0 if w is None else float(w[t, j])) * rows[pos[t, j]]
    return out


def collect_backward(dout, rows, pos, w=None):
    """(drows, dw) of collect; drows is 0 where no entry names the row."""
    dout, rows = as_f64(dout), as_f64(rows)
    drows, dw = np.zeros_like(rows), np.zeros(pos.shape)
    for t, j in np.argwhere((pos >= 0) & (pos < len(rows))):
        drows[pos[t, j]] = (1.0 if w is None else float(w[t, j])) * dout[t]
        dw[t, j] = dout[t] @ rows[pos[t, j]]
    return drows, dw


def keep(v, group=128):
    """(codes, scales) of rows [R, I], `group` columns to a scale: 127 v / max|v| to nearest even, max|v| / 127 in fp32;
    a scale of NaN where an infinity or NaN is among them."""
    v = as_f64(v)
    n = -(-v.shape[1] // group)
    codes, scales = np.zeros(v.shape), np.zeros((v.shape[0], n), np.float32)
    for b in range(n):
        c = slice(b * group, min((b + 1) * group, v.shape[1]))
        m = np.abs(v[:, c]).max(1)
        ok = np.isfinite(m)
        safe = np.where(ok & (m > 0), m, 1.0)[:, None]
        codes[:, c] = np.rint(127.0 * np.where(ok[:, None], v[:, c], 0.0) / safe)
        scales[:, b] = np.where(ok, np.where(ok, m, 0).astype(np.float32) / np.float32(127), np.nan)
    return codes, scales


def kept(codes, scales, group=128):
    """The values that codes and scales stand for."""
    return np.asarray(codes, np.float64) * np.repeat(as_f64(scales), group, 1)[:, :np.shape(codes)[1]]


def sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_backward(g, u, dh):
    """(dg, du) of swiglu."""
    s = sigmoid(g)
    return dh * u * (s + g * s * sigmoid(-g)), dh * g * s


def matmul(a, w, counts, offsets, transposed=False):
    """Rows of the groups times their expert's weights; rows of no group are 0."""
    a, w = as_f64(a), as_f64(w)
    c = np.zeros((len(a), w.shape[1] if transposed else w.shape[2]))
    for e, (o, n) in enumerate(zip(offsets, counts)):
        c[o:o + n] = a[o:o + n] @ (w[e].T if transposed else w[e])
    return c


def matmul_dw(a, dc, counts, offsets):
    a, dc = as_f64(a), as_f64(dc)
    return np.stack([a[o:o + n].T @ dc[o:o + n] for o, n in zip(offsets, counts)])
