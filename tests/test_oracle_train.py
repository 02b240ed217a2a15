"""The 64-bit statements of the training operators, each gradient against central differences and the identities that
tie the operators together."""
import numpy as np
import pytest

import oracle
from oracle import train as tr


def difference(f, x, step=1e-5):
    """Gradient of the scalar f at x by central differences (the error is step^2 f''' / 6 and 1e-16 |f| / step)."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = f()
        x[i] = keep - step
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


@pytest.mark.parametrize("T,E,k", [(1, 5, 1), (9, 4, 3), (40, 16, 6)])
def test_group_is_the_layers_grouping(T, E, k):
    r = np.random.default_rng(T)
    idx = np.argsort(r.random((T, E)), 1)[:, :min(k, E)]
    counts, offsets, pos, src = tr.group(idx, E)
    c, o, p, s = oracle.permute(idx, E)
    assert np.array_equal(counts, c) and np.array_equal(offsets, o) and np.array_equal(pos, p) and np.array_equal(src, s)


def test_group_drops_and_repeats():
    idx = np.array([[1, -1, 1], [7, 0, 4], [1, 3, -9]])
    counts, offsets, pos, src = tr.group(idx, 4)
    assert counts.tolist() == [1, 3, 0, 1] and offsets.tolist() == [0, 1, 4, 4, 5]
    assert pos.tolist() == [[1, -1, 2], [-1, 0, -1], [3, 4, -1]] and src.tolist() == [1, 0, 0, 2, 2]


@pytest.mark.parametrize("weights", [True, False])
def test_collect_gradient(weights):
    r = np.random.default_rng(3)
    T, k, H, E = 5, 3, 4, 4
    idx = r.integers(-1, E, (T, k))
    _, offsets, pos, _ = tr.group(idx, E)
    rows, d = r.standard_normal((offsets[-1], H)), r.standard_normal((T, H))
    w = r.random((T, k)) if weights else None
    drows, dw = tr.collect_backward(d, rows, pos, w)
    f = lambda: float((tr.collect(rows, pos, w) * d).sum())  # noqa: E731
    np.testing.assert_allclose(drows, difference(f, rows), atol=1e-8)
    if weights:
        np.testing.assert_allclose(dw, difference(f, w), atol=1e-8)
    assert np.all(dw[pos < 0] == 0)


def test_kept_values():
    r = np.random.default_rng(4)
    v = r.standard_normal((6, 300))
    v[1, :128], v[2, 130], v[3, 299], v[4, 5] = 0, np.inf, np.nan, -500
    codes, scales = tr.keep(v)
    assert scales.shape == (6, 3) and np.abs(codes).max() == 127 and scales[1, 0] == 0 and not codes[1, :128].any()
    assert np.isnan(scales[2, 1]) and np.isnan(scales[3, 2]) and np.isnan(scales).sum() == 2 and codes[4, 5] == -127
    back = tr.kept(codes, scales)
    ok = np.isfinite(back) & np.isfinite(v)
    # half a code, and the fp32 rounding of the scale on up to 127 of them
    step = np.repeat(scales, 128, 1)[:, :300]
    assert np.all(np.abs(back - v)[ok] <= (step * (0.5 + 127 * 2.0 ** -24))[ok] * (1 + 1e-12))


def test_swiglu_gradient():
    r = np.random.default_rng(5)
    g, u, d = r.standard_normal((3, 7)) * 3, r.standard_normal((3, 7)), r.standard_normal((3, 7))
    g[0, :3] = [0.0, -30.0, 30.0]
    dg, du = tr.swiglu_backward(g, u, d)
    f = lambda: float((tr.swiglu(g, u) * d).sum())  # noqa: E731
    np.testing.assert_allclose(dg, difference(f, g), atol=1e-7)
    np.testing.assert_allclose(du, difference(f, u), atol=1e-7)
    big = np.array([[800.0, -800.0]])
    assert np.all(np.isfinite(tr.swiglu_backward(big, big, big)))


def test_matmul_gradients():
    r = np.random.default_rng(6)
    counts, offsets = np.array([2, 0, 3, 1]), np.array([0, 2, 2, 5, 6])
    a, w, d = r.standard_normal((6, 3)), r.standard_normal((4, 3, 2)), r.standard_normal((6, 2))
    f = lambda: float((tr.matmul(a, w, counts, offsets) * d).sum())  # noqa: E731
    np.testing.assert_allclose(tr.matmul(d, w, counts, offsets, True), difference(f, a), atol=1e-8)
    np.testing.assert_allclose(tr.matmul_dw(a, d, counts, offsets), difference(f, w), atol=1e-8)
