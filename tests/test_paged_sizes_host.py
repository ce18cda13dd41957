"""Sizes of the paged cache's workspaces at the far end of the documented range: a size is either at
least what its arrays hold, computed here without a width, or refused.  No kernel is launched."""

import ctypes

import pytest

FAKE = ctypes.c_void_p(0x1000)
OTHER = ctypes.c_void_p(0x2000)


def _desc(lib, b, cap, n_q, n_kv):
    return lib.tp_paged_desc(b, 8, cap, 0, 0, 0, 1, n_q, n_kv, 64, 1, 0, 0.0, 0)


SIZES = [  # b, slots of a table row, n_q, n_kv
    (2, 64, 8, 2), (65535, 1 << 30, 1, 1), (65535, 1 << 20, 64, 8), (1, 1 << 30, 65535, 65535),
    (16384, 1 << 30, 65532, 16383), (65535, 1 << 29, 65535, 65535), (65535, 1 << 30, 65535, 65535),
    (65535, 1 << 30, 65535, 1), (65535, 1 << 30, 65534, 32767),
]


@pytest.mark.parametrize("b,cap,n_q,n_kv", SIZES)
def test_workspace_sizes_do_not_wrap(lib, b, cap, n_q, n_kv):
    d = _desc(lib, b, cap, n_q, n_kv)
    rows = lib._pack_rows(0x1000, 64 * n_q, 64)
    columns = -(-(n_q // n_kv) // 4) * 4
    need = b * n_kv * cap * columns * 4
    n = lib.tp_attn_decode_paged_workspace(d, True)
    if need <= 1 << 56:
        assert n >= need
    else:
        assert n == 0 and "too many" in lib.tp_last_error()
        # the call itself refuses before any launch, whatever workspace it is offered
        assert lib.load().tp_attn_decode_paged(
            ctypes.byref(d), rows, FAKE, OTHER, FAKE, FAKE, rows, None, FAKE, FAKE, (1 << 64) - 1,
            None) == lib.TP_ERR_SHAPE
    assert lib.tp_attn_decode_paged_workspace(d, False) > 0      # (no scores: no such array)
    need = b * n_kv * cap * 4
    n = lib.tp_kv_evict_paged_workspace(d, cap)
    if need <= 1 << 56:
        assert n >= need
    else:
        assert n == 0 and "too many" in lib.tp_last_error()
        assert lib.load().tp_kv_evict_paged(
            ctypes.byref(d), FAKE, FAKE, cap, 0, FAKE, OTHER, FAKE, FAKE, None, FAKE, (1 << 64) - 1,
            None) == lib.TP_ERR_SHAPE
