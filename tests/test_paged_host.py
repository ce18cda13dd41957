"""Rotary positions and the paged cache without a GPU: the calls check their arguments before
anything is enqueued, and the workspace queries answer.  No kernel is launched here."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


def _paged(lib, b=2, n_pages=8, max_pages=4, strides=(0, 0, 0), page=16, n_q=8, n_kv=2, hd=64,
           dtype=1, flags=0, scale=0.0):
    return lib.tp_paged_desc(b, n_pages, max_pages, *strides, page, n_q, n_kv, hd, dtype, flags,
                             scale, 0)


def _rows(lib, data=0x1000, ts=512, hs=64):
    return ctypes.byref(lib.tp_head_rows(data, ts, hs))


def _decode(lib, desc, q=None, kp=FAKE, vp=FAKE, tables=FAKE, lens=FAKE, o=None, lse=None,
            score=None, ws=FAKE, n=1 << 40):
    return lib.load().tp_attn_decode_paged(
        ctypes.byref(desc) if desc is not None else None, q or _rows(lib), kp, vp, tables, lens,
        o or _rows(lib, 0x9000), lse, score, ws, n, None)


def _append(lib, desc, T=2, seq_ids=FAKE, slots=FAKE, tables=FAKE, k=None, v=None, rope=None,
            freqs=None, positions=None, q=None, q_out=None, kp=FAKE, vp=ctypes.c_void_p(0x2000)):
    return lib.load().tp_kv_append_paged(
        ctypes.byref(desc), T, seq_ids, slots, tables, k or _rows(lib, ts=128), v or _rows(lib, ts=128),
        rope, freqs, positions, q, q_out, kp, vp, None)


def _evict(lib, desc, score=FAKE, lens=FAKE, budget=8, recent=2, kp=FAKE,
           vp=ctypes.c_void_p(0x2000), tables=FAKE, new_lens=FAKE, keep=None, ws=FAKE, n=1 << 40):
    return lib.load().tp_kv_evict_paged(ctypes.byref(desc), score, lens, budget, recent, kp, vp,
                                        tables, new_lens, keep, ws, n, None)


def _rope(lib, desc, dtype=1, T=2, heads=2, hd=64, x=None, positions=FAKE, freqs=FAKE, out=None):
    return lib.load().tp_rope(ctypes.byref(desc) if desc is not None else None, dtype, T, heads,
                              hd, x or _rows(lib, ts=128), positions, freqs, 0,
                              out or _rows(lib, 0x9000, ts=128), None)


def test_status_string(lib):
    assert lib.load().tp_status_string(lib.TP_ERR_INDEX) == b"TP_ERR_INDEX"


@pytest.mark.parametrize("bad", [
    dict(b=-1), dict(b=65536), dict(n_q=0), dict(n_kv=0), dict(n_q=7), dict(hd=4), dict(hd=12),
    dict(hd=264), dict(page=0), dict(n_pages=0), dict(max_pages=0),
    dict(n_pages=1 << 31), dict(max_pages=1 << 28, page=16), dict(max_pages=(1 << 26) + 1, page=16),
])
def test_paged_shapes(lib, bad):
    d = _paged(lib, **bad)
    assert _decode(lib, d) == lib.TP_ERR_SHAPE
    assert _append(lib, d) == lib.TP_ERR_SHAPE
    assert _evict(lib, d) == lib.TP_ERR_SHAPE
    assert lib.tp_attn_decode_paged_workspace(d, True) == 0
    assert lib.tp_kv_evict_paged_workspace(d, 8) == 0
    assert lib.tp_last_error() != ""


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(flags=1), dict(scale=-1.0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(strides=(4096, 1024, 60)), dict(strides=(-4096, 1024, 64)),
    dict(strides=(2048, 512, 64)),          # heads of a page overlap
    dict(strides=(1024, 1024, 64)),         # pages overlap
])
def test_paged_arguments(lib, bad):
    d = _paged(lib, **bad)
    assert _decode(lib, d) == lib.TP_ERR_INVALID_ARG
    assert _append(lib, d) == lib.TP_ERR_INVALID_ARG
    assert _evict(lib, d) == lib.TP_ERR_INVALID_ARG


def test_decode_arguments(lib):
    d = _paged(lib)
    A, W = lib.TP_ERR_INVALID_ARG, lib.TP_ERR_WORKSPACE
    assert _decode(lib, None) == A
    for name in ("kp", "vp", "tables", "lens", "ws"):
        assert _decode(lib, d, **{name: None}) == A, name
        assert _decode(lib, d, **{name: ODD}) == A, name
    assert _decode(lib, d, lse=ODD) == A and _decode(lib, d, score=ODD) == A
    for rows in ((0, 512, 64), (0x1008, 512, 64), (0x1000, 511, 64), (0x1000, 512, 60),
                 (0x1000, -512, 64)):
        assert _decode(lib, d, q=_rows(lib, *rows)) == A
        assert _decode(lib, d, o=_rows(lib, *rows)) == A
    assert _decode(lib, d, o=_rows(lib, 0x9000, 512, 56)) == A      # rows of o overlap
    for score in (None, FAKE):
        need = lib.tp_attn_decode_paged_workspace(d, score is not None)
        assert need > 0
        assert _decode(lib, d, score=score, n=need - 1) == W
    assert _decode(lib, _paged(lib, b=0)) == lib.TP_OK


def test_append_arguments(lib):
    d = _paged(lib)
    A, S = lib.TP_ERR_INVALID_ARG, lib.TP_ERR_SHAPE
    assert _append(lib, d, T=-1) == S
    assert _append(lib, d, T=1 << 31) == S
    assert _append(lib, d, T=3, seq_ids=None) == S
    for name in ("kp", "vp", "tables", "slots"):
        assert _append(lib, d, **{name: None}) == A, name
        assert _append(lib, d, **{name: ODD}) == A, name
    assert _append(lib, d, seq_ids=ctypes.c_void_p(0x1001)) == A
    assert _append(lib, d, kp=FAKE, vp=FAKE) == A                    # one pool for both
    rope = ctypes.byref(lib.rope_desc(64))
    q, qo = _rows(lib), _rows(lib, 0x9000)
    assert _append(lib, d, q=q, q_out=qo) == A                       # q without a rotation
    assert _append(lib, d, rope=rope, freqs=FAKE, q=q) == A
    assert _append(lib, d, rope=rope, freqs=FAKE, q_out=qo) == A
    assert _append(lib, d, rope=rope) == A                           # no table
    assert _append(lib, d, rope=rope, freqs=ctypes.c_void_p(0x1004)) == A
    assert _append(lib, d, rope=rope, freqs=FAKE, positions=ODD) == A
    assert _append(lib, d, rope=ctypes.byref(lib.rope_desc(66)), freqs=FAKE) == S
    assert _append(lib, d, rope=rope, freqs=FAKE, q=q, q_out=_rows(lib, 0x1000, 1024, 64)) == A
    assert _append(lib, d, T=0) == lib.TP_OK


def test_evict_arguments(lib):
    d = _paged(lib)
    A, S, W = lib.TP_ERR_INVALID_ARG, lib.TP_ERR_SHAPE, lib.TP_ERR_WORKSPACE
    for budget, recent in ((0, 0), (-1, 0), (65, 0), (8, -1), (8, 9)):
        assert _evict(lib, d, budget=budget, recent=recent) == S
    assert lib.tp_kv_evict_paged_workspace(d, 65) == 0
    assert lib.tp_kv_evict_paged_workspace(d, 0) == 0
    for name in ("kp", "vp", "tables", "score", "lens", "new_lens", "ws"):
        assert _evict(lib, d, **{name: None}) == A, name
        assert _evict(lib, d, **{name: ODD}) == A, name
    assert _evict(lib, d, keep=ODD) == A
    assert _evict(lib, d, kp=FAKE, vp=FAKE) == A
    need = lib.tp_kv_evict_paged_workspace(d, 8)
    assert need > 0 and _evict(lib, d, n=need - 1) == W
    assert _evict(lib, _paged(lib, b=0)) == lib.TP_OK


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), "TP_ERR_SHAPE"), (dict(rot_dim=7), "TP_ERR_SHAPE"),
    (dict(rot_dim=1026), "TP_ERR_SHAPE"), (dict(rot_dim=128), "TP_ERR_SHAPE"),
    (dict(rot_dim=64, layout=2), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling=4), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, base=0.0), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, base=float("nan")), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="linear", factor=0.0), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="ntk", factor=float("inf")), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="parts", factor=2.0, orig_len=0), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="parts", factor=2.0, orig_len=9, beta_fast=1.0), "TP_ERR_INVALID_ARG"),
    (dict(rot_dim=64, magnitude=-1.0), "TP_ERR_INVALID_ARG"),
])
def test_rope_descriptors(lib, kw, status):
    st = _rope(lib, lib.rope_desc(**kw))
    assert lib.load().tp_status_string(st).decode() == status
    if kw["rot_dim"] != 128:
        st = lib.load().tp_rope_freqs(ctypes.byref(lib.rope_desc(**kw)), FAKE, None)
        assert lib.load().tp_status_string(st).decode() == status


def test_rope_arguments(lib):
    d = lib.rope_desc(64)
    A, S = lib.TP_ERR_INVALID_ARG, lib.TP_ERR_SHAPE
    assert _rope(lib, None) == A
    assert _rope(lib, d, dtype=2) == A
    for bad in (dict(T=-1), dict(heads=-1), dict(heads=65536), dict(hd=1032), dict(hd=63), dict(T=1 << 31)):
        assert _rope(lib, d, **bad) == S
    assert _rope(lib, d, positions=None) == A and _rope(lib, d, positions=ODD) == A
    assert _rope(lib, d, freqs=None) == A and _rope(lib, d, freqs=ctypes.c_void_p(0x1004)) == A
    assert _rope(lib, d, x=_rows(lib, 0)) == A and _rope(lib, d, x=_rows(lib, 0x1001)) == A
    assert _rope(lib, d, x=_rows(lib, ts=-128)) == A
    assert _rope(lib, d, out=_rows(lib, 0x9000, 64, 64)) == A       # rows of out overlap
    assert _rope(lib, d, out=_rows(lib, 0x1000, 256, 64)) == A      # in place, other strides
    assert _rope(lib, d, T=0) == lib.TP_OK and _rope(lib, d, heads=0) == lib.TP_OK
    assert lib.load().tp_rope_freqs(ctypes.byref(d), None, None) == A


def test_python_checks(lib):
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    tables = torch.zeros(2, 2, dtype=torch.int32)
    d = lib.paged_desc(8, kp, tables)
    assert (d.b, d.n_pages, d.max_pages, d.page_size, d.n_kv) == (2, 4, 2, 16, 2)
    assert (d.page_stride, d.head_stride, d.slot_stride) == (2048, 1024, 64)
    slot_major = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)
    d2 = lib.paged_desc(8, slot_major, tables)
    assert (d2.page_stride, d2.head_stride, d2.slot_stride) == (2048, 64, 128)
    with pytest.raises(TypeError):
        lib.paged_desc(8, kp.half(), tables)
    with pytest.raises(ValueError):
        lib.paged_desc(8, kp.transpose(2, 3), tables)
    with pytest.raises(ValueError):
        lib._pages(d, -1, kp, slot_major, tables)       # the pools' strides differ
    with pytest.raises(TypeError):
        lib._pages(d, -1, kp, kp, tables.long())
    with pytest.raises(ValueError):
        lib._pages(d, -1, kp, kp, tables[:1])
    with pytest.raises(ValueError):
        lib._rows("q", torch.zeros(2, 64, 8).transpose(1, 2), -1, torch.float32, (2, 8, 64))
    with pytest.raises(ValueError):
        lib._rows("q", torch.zeros(2, 8, 64), 0, torch.float32, (2, 8, 64))     # not on the device
