"""Decode attention over the paged cache where values are infinite, NaN or near the type's largest.

The output is sum_n w_n v_n in IEEE arithmetic with the softmax's weights: an infinite value gives
the infinity of its sign wherever its weight is not zero, infinities of both signs give NaN, and
finite values give a finite mean, however large they are.  Every path has to say the same: groups of
1, 4, 8 and 16 heads, rows with a block of their own and rows cut into runs.  All keys here have
weights far above the smallest fp32 number, so the oracle's non-finite outputs are the kernel's.
Finite elements: the bound of tests/test_gpu_paged.py.
"""

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from tests.helpers import dev, f64
from tests.test_gpu_paged import HALF_STEP, U, Cache

pytestmark = pytest.mark.gpu
INF = float("inf")
# near the largest number (3.4028e38), and for fp32 above 3.3962e38, where numbers round to an infinite
# bf16; below bf16's largest (3.3895e38) for bf16.  A mean of equal ones does not round to infinity.
HUGE = {"f32": 3.398e38, "bf16": 3.35e38}

GROUPS = [(1, "bf16"), (4, "bf16"), (8, "bf16"), (16, "bf16"), (1, "f32"), (4, "f32"), (8, "f32"),
          (16, "f32")]
# whole rows; rows cut into runs; with head sizes that are padded
SHAPES = [(64, 0), (64, 4000), (40, 0), (128, 2000), (256, 4000)]


def put(c, pool, seq, g, slot, dim, value):
    pool[int(c.tables[seq, slot // c.page]), g, slot % c.page, dim] = value


def check(c, o, lse):
    """o and lse against the oracle, non-finite elements exactly."""
    kp, vp, tables = c.host()
    q, scale, group = f64(c.q), c.hd ** -0.5, c.n_q // c.n_kv
    o, lse = f64(o), f64(lse)
    with np.errstate(invalid="ignore", over="ignore"):
        ro, rl, _ = opaged.decode(q, kp, vp, tables, c.lens_l)
        for i, n in enumerate(c.lens_l):
            _, pg, at = opaged.slots_of(tables, i, n, c.page, kp.shape[0])
            for g in range(c.n_kv):
                hs = slice(g * group, (g + 1) * group)
                k, v = kp[pg, g, at], vp[pg, g, at]
                z = scale * q[i, hs] @ k.T
                w = np.exp(z - rl[i, hs, None])
                assert w.min() > 1e-30
                dz = (scale * (np.abs(q[i, hs]) @ np.abs(k).T) * (2 * c.hd + 4) * U
                      + 4 * U * np.abs(z)).max(1, keepdims=True)
                rel = 2 * dz + (4 * n + 16) * U + (2.0 ** -16 if c.dtype == "bf16" else 0)
                tol = (w @ np.abs(v)) * rel
                tol += HALF_STEP[c.dtype] * (np.abs(ro[i, hs]) + tol)
                want, got = ro[i, hs], o[i, hs]
                fin = np.isfinite(want)
                assert np.array_equal(got[~fin], want[~fin], equal_nan=True), (i, g)
                assert (np.abs(got - want)[fin] <= tol[fin]).all(), (i, g)
                # (a sequence that was taken again counts its maximum from log sum + 9.7)
                tl = dz[:, 0] + (n + 64) * U + 4 * U * np.abs(rl[i, hs])
                assert (np.abs(lse[i, hs] - rl[i, hs]) <= tl).all(), (i, g)


def cache(lib, group, dtype, hd, width, lens=(700, 33, 1)):
    c = Cache(lib, list(lens), 2 * group, 2, hd, 16, dtype, width=width, seed=group)
    c.q.mul_(0.5)
    return c


@pytest.mark.parametrize("hd,width", SHAPES)
@pytest.mark.parametrize("group,dtype", GROUPS)
def test_infinite_values(lib, group, dtype, hd, width):
    c = cache(lib, group, dtype, hd, width)
    put(c, c.vp, 0, 0, 3, 1, INF)
    put(c, c.vp, 0, 0, 650, 2, -INF)
    put(c, c.vp, 0, 0, 5, 7, INF)            # both signs, far apart: other warps, other parts
    put(c, c.vp, 0, 0, 690, 7, -INF)
    put(c, c.vp, 0, 1, 100, hd - 1, float("nan"))
    put(c, c.vp, 1, 0, 32, 0, -INF)          # the last key of a unit of one
    put(c, c.vp, 2, 1, 0, 4, INF)            # a weight of exactly 1
    before = c.score.clone()
    o, lse = c.decode()
    assert torch.isposinf(o[0, :group, 1]).all() and torch.isneginf(o[0, :group, 2]).all()
    assert torch.isnan(o[0, :group, 7]).all() and torch.isposinf(o[2, group:, 4]).all()
    check(c, o, lse)
    # the weights do not depend on the values
    assert torch.isfinite(c.score).all() and not torch.equal(c.score, before)
    again, _ = c.decode(with_score=False)
    assert torch.equal(o.nan_to_num(7.0), again.nan_to_num(7.0))
    lib.tp_check_device_error()


@pytest.mark.parametrize("kind", ["one", "all of one sign", "all of both signs", "large"])
@pytest.mark.parametrize("hd,width", SHAPES)
@pytest.mark.parametrize("group,dtype", GROUPS)
def test_largest_values(lib, group, dtype, hd, width, kind):
    c = cache(lib, group, dtype, hd, width)
    big = HUGE[dtype]
    if kind == "one":
        put(c, c.vp, 0, 0, 3, 1, big)
        put(c, c.vp, 0, 1, 699, 0, -big)
        put(c, c.vp, 2, 0, 0, hd - 1, big)
    elif kind == "all of one sign":
        c.vp.fill_(big)
    else:
        # (2^114: a sum of 700 of them stays below the largest number, with weights up to e^5.5 it may not)
        g = torch.Generator().manual_seed(8)
        s = torch.where(torch.rand(c.vp.shape, generator=g) < 0.5, -1.0, 1.0).to(dev())
        c.vp.copy_(s * (big if kind == "all of both signs" else 2.0 ** 114))
    o, lse = c.decode(with_score=False)
    assert torch.isfinite(o).all()
    check(c, o, lse)
    lib.tp_check_device_error()


def test_pages_outside_the_pool_with_infinite_values(lib):
    # a sequence that is taken again leaves the same keys out
    c = cache(lib, 8, "bf16", 64, 0, lens=(100, 60))
    lib.tp_check_device_error()
    put(c, c.vp, 0, 0, 90, 1, INF)
    c.tables[0, 2] = c.kp.shape[0]
    c.tables[1, 1] = -1
    o, lse = c.decode(with_score=False)
    check(c, o, lse)
    with pytest.raises(lib.TpError) as e:
        lib.tp_check_device_error()
    assert e.value.status == lib.TP_ERR_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [1, 8])
def test_many_rows_in_runs(lib, group, dtype):
    # more rows than runs, so that a run ends one row and begins others: infinities and the largest
    # values in rows of every position of a run, and the weights of rows that were taken again
    lens = [(37 * i) % 101 + 1 for i in range(100)] + [2500, 33]
    c = cache(lib, group, dtype, 64, 2000, lens=lens)
    for i in range(0, len(lens), 3):
        put(c, c.vp, i, i & 1, lens[i] // 2, i % 64, INF if i % 2 else -INF)
        put(c, c.vp, i, 1 - (i & 1), lens[i] - 1, 63 - i % 64, HUGE[dtype])
    before = f64(c.score)
    o, lse = c.decode()
    check(c, o, lse)
    kp, _, tables = c.host()
    q, got = f64(c.q), f64(c.score)
    for i, n in enumerate(lens):
        _, pg, at = opaged.slots_of(tables, i, n, c.page, kp.shape[0])
        for g in range(c.n_kv):
            hs = slice(g * group, (g + 1) * group)
            k = kp[pg, g, at]
            z = c.hd ** -0.5 * q[i, hs] @ k.T
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            dz = (c.hd ** -0.5 * (np.abs(q[i, hs]) @ np.abs(k).T) * (2 * c.hd + 4) * U
                  + 4 * U * np.abs(z)).max(1, keepdims=True)
            # (its score, and the log-sum's error of check())
            want = before[i, g, :n] + w.sum(0)
            tol = (w * (2 * dz + (2 * n + 96) * U)).sum(0) + U * np.abs(want)
            assert (np.abs(got[i, g, :n] - want) <= tol).all(), (i, g)
            assert np.array_equal(got[i, g, n:], before[i, g, n:])
    lib.tp_check_device_error()
