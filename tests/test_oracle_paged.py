"""Pins of the oracle for rotary positions and the paged cache (float64, CPU), independent of it:
closed forms, matrices, dense attention and brute force."""

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from oracle import rope as orope


def test_frequencies_by_hand():
    w, m = orope.frequencies(4, 100.0)
    assert np.allclose(w, [1.0, 0.1]) and m == 1.0
    assert np.allclose(orope.frequencies(4, 100.0, "linear", 4.0)[0], [0.25, 0.025])
    # the larger base interpolates the slowest pair by the factor and the fastest not at all
    w, _ = orope.frequencies(128, 10000.0, "ntk", 8.0)
    w0, _ = orope.frequencies(128, 10000.0)
    assert w[0] == w0[0] and np.isclose(w[-1], w0[-1] / 8.0)
    w, m = orope.frequencies(128, 10000.0, "parts", 4.0, orig=4096)
    turns = 4096 * w0 / (2 * np.pi)
    assert np.array_equal(w[turns > 32], w0[turns > 32])
    assert np.allclose(w[turns < 1], w0[turns < 1] / 4.0) and (turns < 1).any()
    assert np.isclose(m, 1 + 0.1 * np.log(4.0))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_the_matrix_and_keeps_relative_positions(layout):
    rng = np.random.default_rng(0)
    R, hd = 6, 10
    w, _ = orope.frequencies(R, 50.0)
    x = rng.normal(size=(3, 2, hd))
    pos = [0, 5, -7]
    y = orope.rotate(x, pos, R, layout, w, 1.5)
    for t, n in enumerate(pos):
        M = orope.rotation_matrix(R, hd, layout, n * w, 1.5)
        assert np.allclose(y[t], x[t] @ M.T)
        # the gradient is the transpose
        assert np.allclose(orope.rotate(x[t:t + 1], [n], R, layout, w, 1.5, inverse=True)[0],
                           x[t] @ M)
    # q at n against k at m depends on n - m alone
    q, k = rng.normal(size=(1, 1, hd)), rng.normal(size=(1, 1, hd))
    dot = lambda n, m: float((orope.rotate(q, [n], R, layout, w) * orope.rotate(k, [m], R, layout, w)).sum())
    assert np.isclose(dot(11, 4), dot(107, 100))
    assert np.allclose(orope.rotate(x, [0, 0, 0], R, layout, w), x)


def test_rotation_gradient_by_differences():
    rng = np.random.default_rng(1)
    w, m = orope.frequencies(8, 100.0, "parts", 2.0, orig=64)
    x, dy = rng.normal(size=(2, 1, 8)), rng.normal(size=(2, 1, 8))
    dx = orope.rotate(dy, [3, 40], 8, "interleaved", w, m, inverse=True)
    f = lambda z: float((orope.rotate(z, [3, 40], 8, "interleaved", w, m) * dy).sum())
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = 1e-4
        assert np.isclose((f(x + e) - f(x - e)) / 2e-4, dx[idx], rtol=1e-7, atol=1e-8)


def test_decode_equals_dense_attention():
    rng = np.random.default_rng(2)
    b, n_q, n_kv, hd, page, n_pages = 3, 6, 2, 8, 4, 12
    kp, vp = rng.normal(size=(n_pages, n_kv, page, hd)), rng.normal(size=(n_pages, n_kv, page, hd))
    tables = rng.permutation(n_pages).reshape(b, 4)
    lens = [16, 0, 7]
    q = rng.normal(size=(b, n_q, hd))
    o, lse, w = opaged.decode(q, kp, vp, tables, lens)
    assert np.array_equal(o[1], np.zeros((n_q, hd))) and np.isneginf(lse[1]).all()
    for i in (0, 2):
        n = lens[i]
        k = np.concatenate([kp[p] for p in tables[i]], axis=1)[:, :n]
        v = np.concatenate([vp[p] for p in tables[i]], axis=1)[:, :n]
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a))
        kk, vv = (t(np.repeat(a, 3, axis=0)) for a in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(t(q[i])[:, None], kk, vv)[:, 0]
        assert np.allclose(o[i], ref.numpy())
        z = (t(q[i])[:, None] @ kk.transpose(1, 2))[:, 0] / np.sqrt(hd)
        assert np.allclose(lse[i], torch.logsumexp(z, 1).numpy())
        assert np.allclose(w[i].sum(), n_q)   # every query head gives one in all
        assert np.allclose(w[i], torch.softmax(z, 1).numpy().reshape(n_kv, 3, n).sum(1))
    # a page outside the pool leaves its keys out
    bad = tables.copy()
    bad[0][1] = n_pages
    o2, _, w2 = opaged.decode(q, kp, vp, bad, lens)
    assert not w2[0][:, 4:8].any() and np.allclose(w2[0].sum(), n_q)
    assert np.array_equal(o2[2], o[2])


def test_keep_slots_by_hand():
    s = np.array([5.0, 1.0, 5.0, np.nan, 2.0, -0.0, 0.0, 9.0])
    assert opaged.keep_slots(s, 8, 3, 1) == [0, 2, 7]       # ties: the lower slots; 7 is recent
    assert opaged.keep_slots(s, 8, 2, 0) == [0, 7]
    assert opaged.keep_slots(s, 8, 2, 2) == [6, 7]
    assert opaged.keep_slots(s, 8, 6, 1) == [0, 1, 2, 4, 5, 7]   # -0 ties with 0
    assert opaged.keep_slots(s, 8, 8, 0) == list(range(8))
    assert opaged.keep_slots(s, 5, 4, 0) == [0, 1, 2, 4]    # NaN goes first


def test_evict_moves_rows_and_scores():
    rng = np.random.default_rng(3)
    kp, vp = rng.normal(size=(5, 2, 2, 4)), rng.normal(size=(5, 2, 2, 4))
    tables = np.array([[4, 0, 2], [1, 3, 0]])
    score = rng.random((2, 2, 6))
    score[0, 0] = [3, 1, 2, 0, 5, 0]
    keeps, s2, k2, v2, nl = opaged.evict(score, kp, vp, tables, [6, 3], 3, 1)
    assert nl == [3, 3] and keeps[0][0] == [0, 4, 5] and keeps[1] == [[0, 1, 2]] * 2
    assert np.array_equal(k2[4, 0], [kp[4, 0, 0], kp[2, 0, 0]])     # slots 0 and 4
    assert np.array_equal(v2[0, 0], [vp[2, 0, 1], vp[0, 0, 1]])     # slot 5; slot 3 stays
    assert np.array_equal(s2[0, 0], [3, 5, 0, 0, 5, 0])
    assert np.array_equal(s2[1], score[1]) and np.array_equal(k2[1], kp[1])
