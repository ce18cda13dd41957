"""The arithmetic behind fp32 products on bf16 matrix instructions, on the CPU: a number cut into three
bf16 parts (each the rounding of what is left), and the six largest of the nine products of two cuts.

Bounds, for 2^e <= |x| < 2^(e+1): a bf16 has 8 significant bits, so the first part leaves at most
2^(e-8), the second, of a number below 2^(e-8) (or that power itself, which leaves nothing), at most
2^(e-17), and the third has room for the last 7 bits.  The products left out, a1 b2 + a2 b1 + a2 b2, are
then at most 2 * 2^-25 + 2^-34 of 2^(e+e')."""

import numpy as np
import pytest


def bf16(x):
    """Rounds fp32 to bf16, ties to even."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def cut(x):
    parts = []
    r = np.asarray(x, dtype=np.float32)
    for _ in range(3):
        parts.append(bf16(r))
        r = (r - parts[-1]).astype(np.float32)
    return parts, r


def numbers():
    g = np.random.default_rng(0)
    x = g.uniform(1, 2, 200000).astype(np.float32)
    edge = np.float32(1) + g.integers(0, 1 << 7, 20000).astype(np.float32) * np.float32(2.0 ** -7)
    # halfway between two bf16 numbers, and a few last places off
    half = (edge.astype(np.float64) + 2.0 ** -8 + g.integers(-300, 300, 20000) * 2.0 ** -23).astype(np.float32)
    worst = np.float32([1 + 2 ** -8 - 2 ** -16 + 2 ** -17, 1 + 2 ** -8, 2 - 2 ** -23, 1 + 2 ** -8 - 2 ** -17 + 2 ** -23])
    x = np.concatenate([x, edge, half, worst])
    return x[(x >= 1) & (x < 2)]


@pytest.mark.parametrize("e", [0, 40, -40, 126, -100])
def test_three_parts_are_exact(e):
    x = numbers() * np.float32(2.0 ** e)
    (a0, a1, a2), rest = cut(x)
    assert not rest.any()
    assert (a0.astype(np.float64) + a1 + a2 == x).all()
    assert (np.abs(a1) <= np.float64(2.0) ** (e - 8)).all() and np.abs(a1).max() == np.float64(2.0) ** (e - 8)
    assert (np.abs(a2) <= np.float64(2.0) ** (e - 17)).all()


def test_products_left_out():
    x = numbers().astype(np.float64)
    y = np.random.default_rng(1).permutation(x)
    for u, v in ((x, y), (x, x)):
        (a, _), (b, _) = cut(u.astype(np.float32)), cut(v.astype(np.float32))
        a, b = [p.astype(np.float64) for p in a], [p.astype(np.float64) for p in b]
        six = a[0] * b[0] + a[0] * b[1] + a[1] * b[0] + a[1] * b[1] + a[0] * b[2] + a[2] * b[0]
        left = np.abs(u * v - six)
        assert (left <= 2.0 ** -24 + 2.0 ** -34).all()
        assert left.max() > 2.0 ** -25          # (the bound is not one bit smaller)


def test_small_numbers_have_coarser_parts():
    # bf16's smallest number is 2^-133: below about 2^-109 the last part cannot hold every bit
    x = numbers() * np.float32(2.0 ** -120)
    parts, _ = cut(x)
    off = np.abs(sum(p.astype(np.float64) for p in parts) - x)
    assert off.max() <= 2.0 ** -134
    assert off.max() > 0


def test_numbers_without_parts():
    # the largest bf16 is 2^128 - 2^120; numbers halfway to 2^128, 2^128 - 2^119 (3.3962e38), and above
    # round to infinity, those below it (3.39e38 among them) do not
    half = np.float32(2.0 ** 127 * (2 - 2.0 ** -8))
    below = np.nextafter(half, np.float32(0))
    with np.errstate(invalid="ignore", over="ignore"):
        parts, rest = cut(np.float32([half, 3.4e38]))
        assert np.isinf(parts[0]).all() and not np.isfinite(rest).any()
        parts, rest = cut(np.float32([below, 3.39e38]))
    assert np.isfinite(parts).all() and not rest.any()
