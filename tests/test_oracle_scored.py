"""Pins of the oracle's scored gates and int8 experts, independent of its own code path."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle


def test_scores_closed_forms():
    l = np.array([[0.3, -1.2, 2.0], [0.0, 0.0, 0.0]])
    s = oracle.gate_scores(l, "sigmoid")
    for t in range(2):
        for e in range(3):
            assert abs(s[t, e] - 1 / (1 + math.exp(-l[t, e]))) < 1e-15
    s = oracle.gate_scores(l, "softmax")
    den = math.fsum(math.exp(v) for v in l[0])
    assert all(abs(s[0, e] - math.exp(l[0, e]) / den) < 1e-15 for e in range(3))
    assert np.allclose(s[1], 1 / 3, rtol=1e-15)
    inf = np.inf
    assert oracle.gate_scores(np.array([[inf, 0.0, inf]]), "softmax").tolist() == [[0.5, 0.0, 0.5]]
    assert oracle.gate_scores(np.array([[-inf, -inf]]), "softmax").tolist() == [[0.5, 0.5]]
    assert oracle.gate_scores(np.array([[np.nan, 1.0]]), "softmax").tolist() == [[0.0, 1.0]]
    assert oracle.gate_scores(np.array([[-inf, inf, np.nan]]), "sigmoid").tolist() == [[0.0, 1.0, 0.0]]


def test_plain_gate_is_softmax_over_the_chosen():
    r = np.random.default_rng(0)
    l = r.standard_normal((40, 12))
    for k in (1, 3, 12):
        idx, w = oracle.gate_select(l, k)
        assert np.array_equal(idx, oracle.topk_select(l, k))
        assert np.allclose(w, oracle.topk_weights(l, idx), rtol=1e-13, atol=0)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_by_brute_force(group_top):
    """The kept set beats every other set of groups, the chosen set every other set of its experts."""
    r = np.random.default_rng(1)
    E, G, keep, k = 12, 4, 2, 3
    l = np.round(r.standard_normal((60, E)) * 2) / 2
    b = np.round(r.standard_normal(E)) / 4
    idx, w = oracle.gate_select(l, k, "sigmoid", G, keep, group_top, False, 2.5, b)
    s = 1 / (1 + np.exp(-l))
    c = s + b
    for t in range(60):
        rank = [sum(sorted(c[t, 3 * g:3 * g + 3])[-group_top:]) for g in range(G)]
        beats = lambda v, a, o: v[a] > v[o] or (v[a] == v[o] and a < o)  # noqa: E731
        kept = [set(S) for S in itertools.combinations(range(G), keep)
                if all(beats(rank, a, o) for a in S for o in range(G) if o not in S)]
        assert len(kept) == 1
        pool = [e for e in range(E) if e // 3 in kept[0]]
        best = [set(S) for S in itertools.combinations(pool, k)
                if all(beats(c[t], a, o) for a in S for o in pool if o not in S)]
        assert len(best) == 1 and set(idx[t].tolist()) == best[0]
        assert all(beats(c[t], idx[t, j], idx[t, j + 1]) for j in range(k - 1))
        assert np.allclose(w[t], 2.5 * s[t, idx[t]], rtol=1e-15)


def test_balance_moves_the_choice_not_the_weights():
    l = np.array([[1.0, 0.0, -1.0]])
    idx, w = oracle.gate_select(l, 1, "sigmoid", renorm=False, balance=np.array([0.0, 0.0, 9.0]))
    assert idx.tolist() == [[2]] and abs(w[0, 0] - 1 / (1 + math.e)) < 1e-15


def test_quantise_rows_exactly():
    r = np.random.default_rng(2)
    a = r.standard_normal((6, 40)).astype(np.float32)
    a[1] = 0
    a[2, :4] = [1.0, 0.5, -0.5, 0.25]
    a[2, 4:] = 0
    q, s = oracle.quantise_rows(a)
    for i in range(6):
        m = max(Fraction(abs(float(v))) for v in a[i])
        assert s[i] == float(m) / 127.0
        for j in range(40):
            want = round(Fraction(float(a[i, j])) * 127 / m) if m else 0  # Fraction rounds halves to even
            assert q[i, j] == want
    assert q[2, :4].tolist() == [127, 64, -64, 32]


def test_int8_expert_by_hand():
    X = np.array([[2.0, -1.0]])
    q1, q3, q2 = np.array([[3], [1]]), np.array([[1], [2]]), np.array([[5, -7]])
    r = oracle.int8_expert(X, q1, q3, q2, np.array([0.01]), np.array([0.02]), np.array([0.5, 0.25]))
    xq, sx = [127, -64], 2.0 / 127  # -63.5 is halfway: to even
    g, u = (3 * xq[0] + xq[1]) * sx * 0.01, (xq[0] + 2 * xq[1]) * sx * 0.02
    h = g / (1 + math.exp(-g)) * u
    assert abs(r["h"][0, 0] - h) < 1e-15 and abs(r["hq"][0, 0]) == 127
    assert np.allclose(r["y"], [[h * 5 * 0.5, h * -7 * 0.25]], rtol=1e-14)
