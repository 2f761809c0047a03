"""Pins of the grouped-head oracle: scalar brute force, properties of the
rotation, and mistakes that the comparison has to catch."""

import math

import numpy as np
import pytest

from oracle import gqa_oracle


def _brute(q, k, v, scale):
    n, Hq, d = q.shape
    L, Hk, _ = k.shape
    out = np.zeros(q.shape)
    for i in range(n):
        for h in range(Hq):
            g = h // (Hq // Hk)
            keys = L - n + i + 1
            if keys <= 0:
                continue
            w = [math.exp(scale * sum(q[i, h, e] * k[j, g, e] for e in range(d))) for j in range(keys)]
            for e in range(d):
                out[i, h, e] = sum(w[j] * v[j, g, e] for j in range(keys)) / sum(w)
    return out


@pytest.mark.parametrize("n,L,Hq,Hk", [(1, 1, 2, 1), (1, 5, 4, 2), (3, 7, 3, 3), (4, 4, 6, 2), (3, 2, 2, 1), (2, 0, 2, 1)])
def test_attention_against_scalar_sums(n, L, Hq, Hk):
    rng = np.random.default_rng(n * 100 + L)
    q, k, v = rng.normal(size=(n, Hq, 4)), rng.normal(size=(L, Hk, 4)), rng.normal(size=(L, Hk, 4))
    out, mean, size = gqa_oracle.attend(q, k, v, 0.5)
    assert np.allclose(out, _brute(q, k, v, 0.5), atol=1e-12)
    assert (mean >= np.abs(out) - 1e-12).all() and (size >= 0).all()
    if L > 1 and L > n:   # a mask that is off by one is seen
        assert not np.allclose(gqa_oracle.attend(q, k[:-1], v[:-1], 0.5)[0], out, atol=1e-3)


def _table(n, D):
    a = np.arange(n)[:, None] * 100.0 ** (-np.arange(0, D, 2) / D)[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1)


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rotated_products_depend_on_distance_alone(style):
    rng = np.random.default_rng(1)
    table, x, y = _table(50, 8), rng.normal(size=(1, 1, 12)), rng.normal(size=(1, 1, 12))

    def dot(p, s):
        a, b = gqa_oracle.rotate(x, table, np.array([p]), style)[0], gqa_oracle.rotate(y, table, np.array([s]), style)[0]
        assert np.isclose((a * a).sum(), (x * x).sum()) and (a[..., 8:] == x[..., 8:]).all()
        return float((a * b).sum())

    assert np.isclose(dot(3, 10), dot(20, 27)) and np.isclose(dot(0, 0), float((x * y).sum()))
    assert not np.isclose(dot(3, 10), dot(10, 3))   # the sign of the rotation matters


def test_styles_are_one_rotation_in_two_orders():
    rng = np.random.default_rng(2)
    table, x = _table(9, 8), rng.normal(size=(4, 2, 8))
    order = np.array([0, 4, 1, 5, 2, 6, 3, 7])      # place 2i, 2i + 1 of the interleaved order <- i, i + 4
    pos = np.array([0, 3, 5, 8])
    a = gqa_oracle.rotate(x, table, pos, "half")[0]
    b = gqa_oracle.rotate(x[..., order], table, pos, "interleaved")[0]
    assert np.allclose(a[..., order], b)
