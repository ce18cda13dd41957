"""Eviction with indices out of range, and over a pool wider than 2^31 elements.

A length outside 0 .. slots is cut to that range; a kept row whose page or whose new place's page is
outside the pool stays where it is, its score and its entry in ``keep`` move all the same; nothing else
is written, and the error word names the index once."""

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from tests.helpers import dev, f64
from tests.test_gpu_paged import Cache

pytestmark = pytest.mark.gpu


def expected(c, lens, budget, recent):
    """(keep, score, kp, vp, new lens) of the contract, from float64 copies."""
    kp, vp, tables = c.host()
    score = c.score.cpu().numpy()
    old_score, old = score.copy(), (kp.copy(), vp.copy())
    n_pages, page = kp.shape[0], c.page
    keep = np.full((len(lens), c.n_kv, budget), -1, dtype=np.int32)
    new = []
    for i, n in enumerate(min(max(n, 0), c.cap) for n in lens):
        new.append(min(n, budget))
        for g in range(c.n_kv):
            kept = opaged.keep_slots(old_score[i, g], n, budget, recent)
            keep[i, g, :len(kept)] = kept
            score[i, g, :len(kept)] = old_score[i, g, kept]
            for j, s in enumerate(kept):
                frm, to = tables[i][s // page], tables[i][j // page]
                if 0 <= frm < n_pages and 0 <= to < n_pages:
                    for arr, was in ((kp, old[0]), (vp, old[1])):
                        arr[to, g, j % page] = was[frm, g, s % page]
    return keep, score, kp, vp, new


def run(lib, c, lens, budget, recent):
    keep_w, score, kp, vp, new = expected(c, lens, budget, recent)
    lens_d = torch.tensor(lens, dtype=torch.int32, device=dev())
    keep = torch.full((len(lens), c.n_kv, budget), 77, dtype=torch.int32, device=dev())
    ws = torch.full((lib.tp_kv_evict_paged_workspace(c.desc, budget),), 0xff, dtype=torch.uint8,
                    device=dev())
    lib.tp_kv_evict_paged(c.desc, c.score, lens_d, budget, recent, c.kp, c.vp, c.tables, lens_d,
                          keep=keep, workspace=ws)
    assert lens_d.tolist() == new
    assert np.array_equal(keep.cpu().numpy(), keep_w)
    assert np.array_equal(c.score.cpu().numpy(), score)
    assert np.array_equal(f64(c.kp), kp, equal_nan=True) and np.array_equal(f64(c.vp), vp, equal_nan=True)


def reported_once(lib):
    with pytest.raises(lib.TpError) as e:
        lib.tp_check_device_error()
    assert e.value.status == lib.TP_ERR_INDEX
    lib.tp_check_device_error()


@pytest.mark.parametrize("slot_major", [False, True])
@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 80)])
@pytest.mark.parametrize("bad", ["source", "destination", "both, of either side"])
def test_pages_outside_the_pool(lib, bad, dtype, hd, slot_major):
    c = Cache(lib, [600, 500, 40], 2, 2, hd, 16, dtype, slot_major=slot_major, seed=6)
    lib.tp_check_device_error()
    if bad == "source":
        c.tables[0, 30] = c.kp.shape[0]          # slots 480 .. 495: behind the budget
    elif bad == "destination":
        c.tables[1, 3] = -7                      # slots 48 .. 63: before it
    else:
        c.tables[0, 30] = 1 << 30
        c.tables[0, 35] = -1
        c.tables[0, 2] = c.kp.shape[0] + 5
        c.tables[1, :6] = -(1 << 31)
    run(lib, c, [600, 500, 40], 300, 20)
    reported_once(lib)


def test_lengths_out_of_range(lib):
    c = Cache(lib, [600, 500, 40, 90], 2, 2, 64, 16, seed=7)
    lib.tp_check_device_error()
    # (sequence 3 then ends with its table, whose last entries name no page)
    run(lib, c, [-3, 500, -(1 << 31), (1 << 31) - 1], 300, 20)
    reported_once(lib)


def test_offsets_past_31_bits(lib):
    # the pool's last page starts more than 2^32 bytes behind its first
    n_pages, page, hd, stride = 5, 16, 64, (1 << 29) + 64
    g = torch.Generator(device=dev()).manual_seed(1)
    c = Cache(lib, [57], 1, 1, hd, page)
    pools = []
    for _ in range(2):
        flat = torch.empty(stride * (n_pages - 1) + page * hd, dtype=torch.bfloat16, device=dev())
        p = flat.as_strided((n_pages, 1, page, hd), (stride, page * hd, hd, 1))
        p.normal_(generator=g)
        pools.append(p)
    c.kp, c.vp = pools
    c.tables = torch.tensor([[4, 0, 3, 1]], dtype=torch.int32, device=dev())
    c.desc, c.cap = lib.paged_desc(1, c.kp, c.tables), 64
    c.score = torch.rand(1, 1, 64, generator=g, device=dev())
    run(lib, c, [57], 20, 4)
    # and the append into the pages at both ends
    kp, vp = f64(c.kp), f64(c.vp)
    k, v = (torch.randn(2, 1, hd, generator=g, device=dev()).bfloat16() for _ in range(2))
    i32 = dict(dtype=torch.int32, device=dev())
    lib.tp_kv_append_paged(c.desc, k, v, torch.tensor([3, 20], **i32), c.tables, c.kp, c.vp,
                           seq_ids=torch.zeros(2, **i32))
    for t, (p, s) in enumerate(((4, 3), (0, 4))):
        kp[p, 0, s], vp[p, 0, s] = f64(k)[t, 0], f64(v)[t, 0]
    assert np.array_equal(f64(c.kp), kp) and np.array_equal(f64(c.vp), vp)
    lib.tp_check_device_error()
