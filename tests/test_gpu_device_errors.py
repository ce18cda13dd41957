"""The device error word: every kind of error reaches the host once, also where two kinds happened
since the last check.  No kernel here traps, faults or hangs: a wait runs out within its limit, and a
sequence outside the tables is left out by the kernel that meets it."""
import pytest
import torch

from tests.helpers import dev

pytestmark = pytest.mark.gpu


def index_error(lib):
    i32 = dict(dtype=torch.int32, device=dev())
    kp = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device=dev())
    tables = torch.zeros(1, 2, **i32)
    k = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=dev())
    lib.tp_kv_append_paged(lib.paged_desc(1, kp, tables), k, k, torch.zeros(1, **i32), tables, kp,
                           torch.zeros_like(kp), seq_ids=torch.full((1,), 5, **i32))


def status_of(lib):
    try:
        lib.tp_check_device_error()
    except lib.TpError as e:
        return e.status, str(e)
    return lib.TP_OK, ""


@pytest.mark.parametrize("order", ["index, wait", "wait, index"])
def test_both_kinds_are_reported(lib, order):
    status_of(lib)
    status_of(lib)
    for what in order.split(", "):
        index_error(lib) if what == "index" else lib.tp_selftest_wait_timeout(2000)
    status, message = status_of(lib)
    assert status == lib.TP_ERR_TIMEOUT and "site bits 33" in message
    assert status_of(lib)[0] == lib.TP_ERR_INDEX
    assert status_of(lib)[0] == lib.TP_OK
