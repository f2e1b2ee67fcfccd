"""Pins of the router-choice and MXFP4 oracles (CPU): brute force, finite differences, the
formats' tables."""
import itertools

import numpy as np
import pytest

from oracle import mxfp4, topk
from oracle import route as rt


def test_choice_equals_the_plain_router():
    rng = np.random.default_rng(0)
    l = np.round(rng.standard_normal((50, 8)) * 4) / 4      # with ties
    idx = topk.choose(l, 3)
    ref, p = rt.route(l, 3)
    np.testing.assert_array_equal(idx, ref)
    np.testing.assert_allclose(topk.weights(l, idx), p, rtol=1e-14)


def test_groups_by_brute_force():
    rng = np.random.default_rng(1)
    E, G, tg, k = 12, 4, 2, 3
    l, b = rng.standard_normal((40, E)), 0.3 * rng.standard_normal(E)
    idx = topk.choose(l, k, "sigmoid", b, G, tg, 2)
    for t in range(40):
        key = 1 / (1 + np.exp(-l[t])) + b
        best = max(itertools.combinations(range(G), tg),
                   key=lambda gs: sum(np.sort(key[g * 3:g * 3 + 3])[-2:].sum() for g in gs))
        pool = [e for g in best for e in range(g * 3, g * 3 + 3)]
        assert list(idx[t]) == sorted(pool, key=lambda e: -key[e])[:k]


def test_masked_rows():
    l = np.full((2, 6), -np.inf)
    l[1, 4] = 0.5
    idx = topk.choose(l, 2, "sigmoid", np.linspace(0, 1, 6))
    np.testing.assert_array_equal(idx, [[0, 1], [4, 0]])
    np.testing.assert_array_equal(topk.weights(l, idx, "sigmoid"), [[0, 0], [1, 0]])
    np.testing.assert_array_equal(topk.weights(l, idx, "softmax", False), [[0, 0], [1, 0]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_by_differences(score, renorm):
    rng = np.random.default_rng(2)
    T, E, k, h = 6, 7, 3, 1e-6
    l, d = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    idx = topk.choose(l, k, score)
    g = topk.bwd(l, idx, d, score, renorm, 1.7)
    for e in range(E):
        up, dn = l.copy(), l.copy()
        up[:, e] += h
        dn[:, e] -= h
        f = lambda z: (topk.weights(z, idx, score, renorm, 1.7) * d).sum(1)   # noqa: E731
        # central difference: h^2 times the third derivative (order 1) plus 1e-16 / h
        np.testing.assert_allclose(g[:, e], (f(up) - f(dn)) / (2 * h), atol=1e-8)


def test_e2m1_table_and_ties():
    np.testing.assert_array_equal(mxfp4.encode(mxfp4.VALUES), np.arange(8))
    np.testing.assert_array_equal(mxfp4.encode(-mxfp4.VALUES), np.arange(8) + 8)   # -0 keeps its sign
    mids = (mxfp4.VALUES[1:] + mxfp4.VALUES[:-1]) / 2
    np.testing.assert_array_equal(mxfp4.encode(mids), [0, 2, 2, 4, 4, 6, 6])
    np.testing.assert_array_equal(mxfp4.encode(np.nextafter(mids, 9)), np.arange(1, 8))
    np.testing.assert_array_equal(mxfp4.encode([6.5, 100.0]), [7, 7])


def test_quantize_round_trip():
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 256, (5, 32), dtype=np.uint8)
    codes[:, 0], codes[:, 16] = 0x77, 0x66                # every block's largest is 6 or 4: its own scale again
    scales = rng.integers(1, 250, (5, 2), dtype=np.uint8)
    v = mxfp4.decode(codes, scales)
    c2, s2 = mxfp4.quantize_rows(v)
    np.testing.assert_array_equal(s2, scales)
    np.testing.assert_array_equal(c2, codes)
    z, s = mxfp4.quantize_rows(np.zeros((1, 32)))
    assert not z.any() and not s.any()
    cc, cs = mxfp4.quantize_cols(v[:3])
    assert cc.shape == (64, 16) and cs.shape == (64, 1)
