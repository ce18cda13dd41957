"""Oracle for rotary positions (float64, CPU).

Test infrastructure only (see the package docstring).

Pair i of a row at position n turns by the angle n * w_i, w_i = base^(-2i/R) for R rotated dims;
the pair is dims (i, i + R/2) in the half layout and (2i, 2i + 1) in the interleaved one, the
other dims pass through.  Longer contexts: linear interpolation (w / s), a larger base
(base * s^(R/(R-2))), or by parts: with r = orig * w / 2 pi turns over the original context, pairs
of more than beta_fast turns keep w, pairs of fewer than beta_slow take w / s, linear between, and
the rotated dims are scaled by 1 + 0.1 ln s.
"""

import numpy as np


def frequencies(R, base=10000.0, scaling="none", factor=1.0, orig=0, beta_fast=32.0,
                beta_slow=1.0):
    """(w (R/2,), magnitude)."""
    w = np.array([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=np.float64)
    if scaling == "none":
        return w, 1.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "ntk":
        big = base * factor ** (R / (R - 2.0)) if R > 2 else base
        return np.array([big ** (-2.0 * i / R) for i in range(R // 2)]), 1.0
    turns = orig * w / (2 * np.pi)
    keep = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
    return keep * w + (1 - keep) * w / factor, 1.0 + 0.1 * np.log(factor)


def rotation_matrix(R, hd, layout, angles, magnitude):
    """The (hd, hd) matrix of one position: row vector x -> x @ M.T is the rotated row."""
    M = np.eye(hd)
    for i, a in enumerate(angles):
        p, q = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        M[p, p] = M[q, q] = magnitude * np.cos(a)
        M[p, q] = -magnitude * np.sin(a)
        M[q, p] = magnitude * np.sin(a)
    return M


def rotate(x, positions, R, layout, w, magnitude=1.0, inverse=False):
    """x (T, H, hd) -> rotated (the gradient's transpose with ``inverse``)."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    for t, n in enumerate(np.asarray(positions).tolist()):
        a = float(n) * np.asarray(w, dtype=np.float64)
        c, s = magnitude * np.cos(a), magnitude * np.sin(a)
        if inverse:
            s = -s
        i = np.arange(R // 2)
        p, q = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        y[t][:, p] = x[t][:, p] * c - x[t][:, q] * s
        y[t][:, q] = x[t][:, p] * s + x[t][:, q] * c
    return y
