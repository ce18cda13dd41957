"""Rotary positions on the GPU against the float64 oracle.

Error bound per element, from the arithmetic: the angle is reduced in 64 bits (relative 2^-50
with the frequency's own rounding, so |position| 2^-50 rad), rounded once to fp32 as at most one
half turn (pi 2^-25), sine and cosine are CUDA's to 2 ulp (2^-23), the magnitude 2^-24; then two
products and a sum of fp32, 3 * 2^-24 of |x1| + |x2|.  Together m (|x1| + |x2|) (5e-7 +
|position| 2^-50), and half a step of the output type.
"""

import numpy as np
import pytest
import torch

from oracle import rope as orope
from tests.helpers import dev, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def check(y, x, positions, R, layout, w, m, dtype, inverse=False):
    x, y, pos = f64(x), f64(y), positions.cpu().numpy()
    ref = orope.rotate(x, pos, R, layout, w, m, inverse=inverse)
    a = np.abs(x)
    pair = np.zeros_like(a)
    i = np.arange(R // 2)
    p, q = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    pair[..., p] = pair[..., q] = a[..., p] + a[..., q]
    tol = m * pair * (5e-7 + np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -50)
    tol += HALF_STEP[dtype] * (np.abs(ref) + tol)
    assert (np.abs(y - ref) <= tol).all(), float((np.abs(y - ref) - tol).max())
    assert np.array_equal(y[..., R:], x[..., R:])     # the other dims pass through exactly


def table(lib, desc):
    f = torch.empty(desc.rot_dim // 2, dtype=torch.float64, device=dev())
    lib.tp_rope_freqs(desc, f)
    return f


def rows(seed, *shape, dtype="bf16"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype]).to(dev())


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("parts", 4.0)])
@pytest.mark.parametrize("R", [2, 64, 130])
def test_frequencies(lib, R, scaling, factor):
    desc = lib.rope_desc(R, "half", 500000.0, scaling, factor, 8192)
    w, _ = orope.frequencies(R, 500000.0, scaling, factor, orig=8192)
    got = table(lib, desc).cpu().numpy() * 2 * np.pi
    assert np.allclose(got, w, rtol=1e-14, atol=0)    # a few roundings of 64-bit pow


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,hd,R", [(1, 1, 2, 2), (5, 3, 128, 128), (257, 9, 128, 64),
                                      (33, 2, 80, 80), (19, 7, 96, 48), (7, 72, 256, 256),
                                      (3, 5, 50, 34), (130, 1, 1024, 1024), (700, 40, 64, 32),
                                      (65, 9, 80, 40), (9, 2, 1024, 8)])
def test_rotation(lib, T, H, hd, R, layout, dtype):
    x = rows(T + hd, T, H, hd, dtype=dtype)
    pos = torch.arange(T, dtype=torch.int32, device=dev()) * 37 - 11
    out = torch.full_like(x, float("nan"))
    for scaling, inverse in (("none", False), ("parts", True)):
        factor = 1.0 if scaling == "none" else 8.0
        desc = lib.rope_desc(R, layout, 10000.0, scaling, factor, 2048)
        w, m = orope.frequencies(R, 10000.0, scaling, factor, orig=2048)
        f = table(lib, desc)
        lib.tp_rope(desc, x, pos, f, out, inverse=inverse)
        check(out, x, pos, R, layout, w, m, dtype, inverse)
        again = x.clone()
        lib.tp_rope(desc, again, pos, f, again, inverse=inverse)      # in place
        assert torch.equal(again, out)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_alignment(lib, layout):
    T, H, hd, R = 37, 5, 64, 64
    desc = lib.rope_desc(R, layout, magnitude=0.5)
    w, _ = orope.frequencies(R)
    f = table(lib, desc)
    pos = torch.randint(0, 4096, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).to(dev())
    base = rows(9, T, 3 * H, hd + 8)
    for name, x in (("slice", base[:, H:2 * H, :hd]), ("odd start", base[:, H:2 * H, 3:hd + 3]),
                    ("heads first", base[:, :H, :hd].transpose(0, 1).contiguous().transpose(0, 1)),
                    ("one row for all heads", base[:, :1, :hd].expand(T, H, hd))):
        out = torch.zeros(T, H, hd + 1, dtype=torch.bfloat16, device=dev())
        for o in (out[:, :, :hd], out[:, :, 1:], torch.empty(T, H, hd, dtype=torch.bfloat16, device=dev())):
            lib.tp_rope(desc, x, pos, f, o)
            check(o, x, pos, R, layout, w, 0.5, "bf16")
    before = base.clone()
    lib.tp_rope(desc, base[:, H:2 * H, :hd], pos, f, base[:, H:2 * H, :hd])
    assert torch.equal(base[:, :H], before[:, :H]) and torch.equal(base[:, 2 * H:], before[:, 2 * H:])
    assert torch.equal(base[..., hd:], before[..., hd:])


def test_far_positions(lib):
    # at 10^9 tokens an angle in fp32 would be off by tens of radians
    desc = lib.rope_desc(64)
    w, _ = orope.frequencies(64)
    x = rows(4, 6, 2, 64, dtype="f32")
    pos = torch.tensor([0, 1, 1_000_003, -999_983, 1_000_000_007, 2**31 - 1], dtype=torch.int32, device=dev())
    out = torch.empty_like(x)
    lib.tp_rope(desc, x, pos, table(lib, desc), out)
    check(out, x, pos, 64, "half", w, 1.0, "f32")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_by_differences(lib, layout):
    # the rotation is linear: sum(dy * rope(x)) and sum(dx * x) are equal, and a central difference
    # over one input gives its dx; fp32 sums of 32 terms of size 1 stay within 1e-4
    desc = lib.rope_desc(16, layout, 100.0, "parts", 2.0, 64)
    f = table(lib, desc)
    x, dy = rows(5, 2, 1, 16, dtype="f32"), rows(6, 2, 1, 16, dtype="f32")
    pos = torch.tensor([3, 40], dtype=torch.int32, device=dev())
    dx, y = torch.empty_like(x), torch.empty_like(x)
    lib.tp_rope(desc, dy, pos, f, dx, inverse=True)

    def loss(z):
        lib.tp_rope(desc, z, pos, f, y)
        return float((y.double() * dy.double()).sum())
    for idx in np.ndindex(*x.shape):
        e = torch.zeros_like(x)
        e[idx] = 0.5
        assert abs((loss(x + e) - loss(x - e)) - float(dx[idx])) <= 1e-4


def test_streams_and_capture(lib):
    desc = lib.rope_desc(128)
    f = table(lib, desc)
    x, y = rows(7, 64, 8, 128), torch.empty(64, 8, 128, dtype=torch.bfloat16, device=dev())
    pos = torch.arange(64, dtype=torch.int32, device=dev())
    lib.tp_rope(desc, x, pos, f, y)
    want = y.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y.zero_()
    s.wait_stream(torch.cuda.current_stream())
    lib.tp_rope(desc, x, pos, f, y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.tp_rope(desc, x, pos, f, y)
    pos += 1000
    g.replay()
    w, m = orope.frequencies(128)
    check(y, x, pos, 128, "half", w, m, "bf16")


def test_refusals(lib):
    desc = lib.rope_desc(64)
    f = table(lib, desc)
    x = rows(8, 4, 2, 64)
    pos = torch.arange(4, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError):
        lib.tp_rope(desc, x.cpu(), pos, f, x)
    with pytest.raises(TypeError):
        lib.tp_rope(desc, x, pos.long(), f, x)
    with pytest.raises(TypeError):
        lib.tp_rope(desc, x, pos, f.float(), x)
    with pytest.raises(TypeError):
        lib.tp_rope(desc, x, pos, f, x.float())
    with pytest.raises(ValueError):
        lib.tp_rope(desc, x, pos, f, x[:3])
    with pytest.raises(lib.TpError):
        lib.tp_rope(desc, x[:, :, :32], pos, f, x[:, :, :32])      # head_dim < rot_dim
