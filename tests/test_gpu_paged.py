"""The paged key/value cache on the GPU: append, decode attention, eviction, and a run of them
together, against the float64 oracle.

Bounds of the decode attention, per element, from the arithmetic (u = 2^-24; the tensor cores'
fp32 accumulation is taken as 2u a step).  A score's error is dz = scale |q|.|k| (2 hd + 4) u +
4 u |z| (the largest over the keys); a weight's relative error is then at most 2 dz + (2 n + 16) u
(its own score, the common maximum and sum over n keys), so
  |o - ref|     <= sum_n w_n |v_n| (2 dz + (4 n + 16) u [+ 2^-16: bf16 weights in two parts]) + half a step
  |lse - ref|   <= dz + (n + 8) u + 4 u |lse|
  |score - ref| <= ref's increment (2 dz + (2 n + 16) u) + u |score|
A pass over the keys in split parts has fewer sums in a row, never more.
"""

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from oracle import rope as orope
from tests.helpers import dev, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


class Cache:
    """A pool whose pages are handed out in a shuffled order; what no sequence uses is NaN."""

    def __init__(self, lib, lens, n_q, n_kv, hd, page, dtype="bf16", seed=0, slot_major=False,
                 extra=0, pad=0, width=0):
        g = torch.Generator().manual_seed(seed)
        self.lib, self.n_q, self.n_kv, self.hd, self.page = lib, n_q, n_kv, hd, page
        self.dtype, self.lens_l, b = dtype, list(lens), len(lens)
        used = [-(-(n + extra) // page) for n in lens]
        width, n_pages = max(max(used) + 1, 2, width), sum(used) + 3
        order = torch.randperm(n_pages, generator=g).tolist()
        t = torch.full((b, width), -1, dtype=torch.int32)     # entries not in use: never read
        for i, u in enumerate(used):
            for c in range(u):
                t[i, c] = order.pop()
        shape = (n_pages, page, n_kv, hd + pad) if slot_major else (n_pages, n_kv, page, hd + pad)
        pools = []
        for _ in range(2):
            p = torch.full(shape, float("nan"), dtype=DT[dtype])
            v = (p.transpose(1, 2) if slot_major else p)[..., :hd]
            for i, n in enumerate(lens):
                s = torch.arange(n)
                v[t[i, s // page].long(), :, s % page] = torch.randn(n, n_kv, hd, generator=g).to(DT[dtype])
            p = p.to(dev())
            pools.append((p.transpose(1, 2) if slot_major else p)[..., :hd])
        self.kp, self.vp = pools
        self.tables = t.to(dev())
        self.lens = torch.tensor(self.lens_l, dtype=torch.int32, device=dev())
        self.desc = lib.paged_desc(n_q, self.kp, self.tables)
        self.cap = width * page
        self.q = (2 * torch.randn(b, n_q, hd, generator=g)).to(DT[dtype]).to(dev())
        self.score = torch.rand(b, n_kv, self.cap, generator=g).to(dev())

    def host(self):
        return f64(self.kp), f64(self.vp), self.tables.cpu().numpy()

    def decode(self, with_score=True, q=None, o=None, lens=None, ws=None, stream=None):
        q = self.q if q is None else q
        o = torch.full_like(q, float("nan")) if o is None else o
        lse = torch.full(q.shape[:2], float("nan"), device=dev())
        if ws is None:
            n = self.lib.tp_attn_decode_paged_workspace(self.desc, with_score)
            # what an earlier call may have left: NaN
            ws = torch.full((n,), 0xff, dtype=torch.uint8, device=dev())
        self.lib.tp_attn_decode_paged(self.desc, q, self.kp, self.vp, self.tables,
                                      self.lens if lens is None else lens, o, lse=lse,
                                      score=self.score if with_score else None, workspace=ws,
                                      stream=stream)
        return o, lse

    def check(self, o, lse, before, q=None, lens=None):
        """o, lse and (``before`` not None) the score's increments against the oracle."""
        kp, vp, tables = self.host()
        q = f64(self.q if q is None else q)
        lens = self.lens_l if lens is None else lens
        ro, rl, rw = opaged.decode(q, kp, vp, tables, lens, self.desc.scale or None)
        scale = self.desc.scale or self.hd ** -0.5
        group = self.n_q // self.n_kv
        o, lse = f64(o), f64(lse)
        if before is not None:
            got, was = f64(self.score), f64(before)
        for i, n in enumerate(lens):
            slots, pg, at = opaged.slots_of(tables, i, min(n, self.cap), self.page, kp.shape[0])
            if not len(slots):
                assert not o[i].any() and np.isneginf(lse[i]).all()
            for g in range(self.n_kv):
                if not len(slots):
                    continue
                hs = slice(g * group, (g + 1) * group)
                k, v = kp[pg, g, at], vp[pg, g, at]
                z = scale * q[i, hs] @ k.T
                w = np.exp(z - rl[i, hs, None])
                dz = (scale * (np.abs(q[i, hs]) @ np.abs(k).T) * (2 * self.hd + 4) * U
                      + 4 * U * np.abs(z)).max(1, keepdims=True)
                rel = 2 * dz + (4 * n + 16) * U + (2.0 ** -16 if self.dtype == "bf16" else 0)
                tol = (w @ np.abs(v)) * rel
                tol += HALF_STEP[self.dtype] * (np.abs(ro[i, hs]) + tol)
                assert (np.abs(o[i, hs] - ro[i, hs]) <= tol).all(), (i, g)
                tl = dz[:, 0] + (n + 8) * U + 4 * U * np.abs(rl[i, hs])
                assert (np.abs(lse[i, hs] - rl[i, hs]) <= tl).all(), (i, g)
                if before is not None:
                    want = was[i, g].copy()
                    want[:rw[i].shape[1]] += rw[i][g]
                    tol = np.zeros(self.cap)
                    tol[slots] = (w * (2 * dz + (2 * n + 16) * U)).sum(0) + U * np.abs(want[slots])
                    assert (np.abs(got[i, g] - want) <= tol).all(), (i, g)
        if before is not None:      # empty sequences and what lies behind a sequence
            for i, n in enumerate(lens):
                assert torch.equal(self.score[i, :, n:], before[i, :, n:])


DECODE = [
    # lens, n_q, n_kv, hd, page, dtype
    ([1], 1, 1, 8, 1, "bf16"),
    ([0, 1, 333], 8, 1, 128, 16, "bf16"),
    ([15, 16, 17, 31, 32, 33, 63, 64, 65], 8, 2, 128, 16, "bf16"),
    ([1111, 5, 64, 0], 8, 8, 64, 24, "f32"),
    ([100, 8, 7, 0], 10, 2, 80, 7, "bf16"),
    ([100, 8, 7, 0], 10, 2, 80, 7, "f32"),
    ([700, 127], 32, 2, 256, 64, "bf16"),
    ([300, 127], 32, 2, 256, 64, "f32"),
    ([50, 129], 40, 2, 96, 1, "bf16"),
    ([50, 129], 66, 2, 96, 3, "f32"),
    ([130, 2], 66, 2, 72, 32, "bf16"),
    ([128, 129], 3, 3, 8, 128, "bf16"),
    ([40, 3], 70, 1, 16, 8, "bf16"),
    ([40, 700, 1, 90], 8, 2, 40, 16, "f32"),
    ([40, 2100, 1, 90], 8, 1, 256, 16, "f32"),
    ([40, 2100, 1, 90], 32, 2, 128, 16, "f32"),
    ([40, 700, 1, 90], 4, 4, 32, 16, "bf16"),
    ([2049, 512, 513, 90, 1025], 16, 2, 128, 32, "bf16"),
    ([2049, 512, 513, 90, 1025], 4, 2, 128, 32, "f32"),
    ([3, 0, 9] * 70, 4, 2, 64, 8, "bf16"),
]


@pytest.mark.parametrize("lens,n_q,n_kv,hd,page,dtype", DECODE)
@pytest.mark.parametrize("slot_major", [False, True])
def test_decode(lib, lens, n_q, n_kv, hd, page, dtype, slot_major):
    c = Cache(lib, lens, n_q, n_kv, hd, page, dtype, slot_major=slot_major, pad=8 if slot_major else 0)
    before = c.score.clone()
    o, lse = c.decode()
    c.check(o, lse, before)
    first = c.score.clone()
    c.score.copy_(before)
    o2, lse2 = c.decode()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(first, c.score)
    o3, lse3 = c.decode(with_score=False)
    c.check(o3, lse3, None)
    lib.tp_check_device_error()


@pytest.mark.parametrize("lens,n_q,n_kv,hd,page,dtype", DECODE)
def test_decode_wide_tables(lib, lens, n_q, n_kv, hd, page, dtype):
    # tables with room for rows far longer than the sequences: the work is cut into runs, which end
    # anywhere in a sequence, hold several short ones, and meet empty ones
    c = Cache(lib, lens, n_q, n_kv, hd, page, dtype, width=60000 // page)
    few = len(lens) * n_kv <= 40
    before = c.score.clone() if few else None
    o, lse = c.decode(with_score=few)
    c.check(o, lse, before)
    o2, lse2 = c.decode(with_score=False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    lib.tp_check_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_many_rows_in_runs(lib, dtype):
    # more rows than runs, lengths around a unit's
    lens = [(37 * i) % 101 for i in range(100)] + [1, 2500, 33]
    c = Cache(lib, lens, 8, 4, 64, 16, dtype, width=2000)
    c.check(*c.decode(with_score=False), None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_long(lib, dtype):
    # one sequence over every SM, and lengths that end anywhere in the split
    c = Cache(lib, [30011, 9000], 8, 2, 64, 40, dtype)
    before = c.score.clone()
    c.check(*c.decode(), before)
    for n in (29952, 20001, 4097):
        lens = torch.tensor([n, 1], dtype=torch.int32, device=dev())
        c.check(*c.decode(with_score=False, lens=lens), None, lens=[n, 1])


def test_decode_strided_rows_and_scale(lib):
    c = Cache(lib, [77, 300, 12], 8, 2, 64, 16)
    qkv = torch.randn(3, 12, 72, generator=torch.Generator().manual_seed(3)).bfloat16().to(dev())
    q = qkv[:, :8, :64]
    out = torch.full((8, 3, 64), 7.0, dtype=torch.bfloat16, device=dev())
    c.desc.scale = 0.4
    before = c.score.clone()
    o, lse = c.decode(q=q, o=out.transpose(0, 1))
    c.check(o, lse, before, q=q)


def test_decode_extreme_values(lib):
    # large scores: one key takes all the weight; equal scores: the mean; a common score that a
    # softmax without its maximum would overflow on
    c = Cache(lib, [400, 400], 8, 2, 64, 16)
    c.q.mul_(50)
    before = c.score.clone()
    c.check(*c.decode(), before)
    c.q.zero_()
    before = c.score.clone()
    c.check(*c.decode(), before)


@pytest.mark.parametrize("width", [0, 4000])     # whole rows; runs, some of them without a weight
@pytest.mark.parametrize("n_q,dtype", [(4, "bf16"), (4, "f32"), (1, "f32"), (16, "f32")])
def test_decode_infinite_keys(lib, n_q, dtype, width):
    # a key with a score of -infinity has weight 0; all of them: no softmax (NaN), lse -infinity
    a, b = (1000, 400) if width else (100, 40)
    c = Cache(lib, [a, b], n_q, 1, 64, 16, dtype, width=width)
    c.q[..., 0] = 1.0
    tables = c.tables.cpu().numpy()
    hit = [s for s in range(a) if s % 3 == 0 or s < b]
    for i, at in ((0, torch.tensor(hit)), (1, torch.arange(b))):
        c.kp[c.tables[i, (at // 16).to(dev())].long(), 0, (at % 16).to(dev()), 0] = -float("inf")
    before = c.score.clone()
    o, lse = c.decode()
    assert torch.isnan(o[1]).all() and torch.isneginf(lse[1]).all()
    assert torch.isnan(c.score[1, 0, :b]).all()
    kp, vp = f64(c.kp), f64(c.vp)
    s = np.arange(a)
    k, v = kp[tables[0][s // 16], 0, s % 16], vp[tables[0][s // 16], 0, s % 16]
    for j in range(n_q):
        z = k @ f64(c.q)[0, j] / 8.0
        e = np.exp(z - z.max())
        assert np.allclose(f64(o)[0, j], (e / e.sum()) @ v, rtol=2e-2, atol=2e-2)
    assert torch.equal(c.score[0, 0, hit], before[0, 0, hit])
    # NaN in a key: its sequence and KV head give NaN, others do not
    c2 = Cache(lib, [100, 40], 2 * n_q, 2, 64, 16, dtype)
    c2.kp[int(c2.tables[0, 0]), 1, 3, 5] = float("nan")
    o, lse = c2.decode(with_score=False)
    assert torch.isnan(o[0, n_q:]).all() and torch.isnan(lse[0, n_q:]).all()
    assert torch.isfinite(o[0, :n_q].float()).all() and torch.isfinite(o[1].float()).all()


def test_decode_indices_out_of_range(lib):
    # checked on the device: pages outside the pool are left out, lengths are cut to the table
    c = Cache(lib, [100, 40, 64], 8, 2, 64, 16)
    c.tables[0, 2] = c.kp.shape[0]
    c.tables[1, :3] = -5
    lib.tp_check_device_error()
    before = c.score.clone()
    o, lse = c.decode()
    c.check(o, lse, before)
    assert torch.equal(c.score[1], before[1]) and torch.equal(c.score[0, :, 32:48], before[0, :, 32:48])
    with pytest.raises(lib.TpError) as e:
        lib.tp_check_device_error()
    assert e.value.status == lib.TP_ERR_INDEX
    lib.tp_check_device_error()
    # (sequence 1 ends with its page; the entries behind it name no page)
    c = Cache(lib, [100, 48, 64], 8, 2, 64, 16)
    lens = torch.tensor([-3, 1 << 30, 64], dtype=torch.int32, device=dev())
    c.check(*c.decode(with_score=False, lens=lens), None, lens=[0, 48, 64])
    with pytest.raises(lib.TpError):
        lib.tp_check_device_error()


def test_decode_offsets_past_31_bits(lib):
    # the pool's last pages lie more than 2^31 elements behind its first
    n_pages, page, hd = 5, 16, 64
    stride = (1 << 29) + 64
    pools = []
    g = torch.Generator(device=dev()).manual_seed(0)
    for _ in range(2):
        flat = torch.empty(stride * (n_pages - 1) + page * hd, dtype=torch.bfloat16, device=dev())
        p = flat.as_strided((n_pages, 1, page, hd), (stride, page * hd, hd, 1))
        p.normal_(generator=g)
        pools.append(p)
    tables = torch.tensor([[4, 0, 3, 4]], dtype=torch.int32, device=dev())
    desc = lib.paged_desc(4, pools[0], tables)
    q = torch.randn(1, 4, hd, generator=g, device=dev()).bfloat16()
    c = Cache(lib, [1], 4, 1, hd, page)
    c.kp, c.vp, c.tables, c.desc, c.cap = pools[0], pools[1], tables, desc, 64
    n = torch.tensor([57], dtype=torch.int32, device=dev())
    o, lse = c.decode(with_score=False, q=q, lens=n)
    c.check(o, lse, None, q=q, lens=[57])


def test_two_graphs_share_a_workspace_and_streams(lib):
    a, b = Cache(lib, [500, 3000], 8, 2, 64, 16, seed=1), Cache(lib, [64, 1999], 8, 2, 64, 16, seed=2)
    need = max(lib.tp_attn_decode_paged_workspace(c.desc, True) for c in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    graphs, outs = [], []
    for c in (a, b):
        c.decode(ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.decode(ws=ws))
        graphs.append(g)
    for _ in range(2):
        before = [c.score.clone() for c in (a, b)]
        graphs[0].replay()
        graphs[1].replay()
        a.lens.copy_(torch.tensor([20, 2900]))
        a.lens_l = [20, 2900]
        mid = a.score.clone()
        graphs[0].replay()
        a.check(*outs[0], mid)
        b.check(*outs[1], before[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    res = [a.decode(with_score=False, stream=s) for _ in range(2)]
    torch.cuda.current_stream().wait_stream(s)
    a.check(*res[1], None)


# ------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n_q,n_kv,hd,R,page,slot_major", [
    (8, 2, 128, 128, 16, False), (10, 2, 80, 40, 7, True), (3, 3, 8, 2, 1, False),
    (4, 1, 256, 256, 64, True), (8, 8, 64, 50, 24, False)])
def test_append(lib, n_q, n_kv, hd, R, page, slot_major, layout, dtype):
    lens = [40, 0, 9, 130]
    c = Cache(lib, lens, n_q, n_kv, hd, page, dtype, slot_major=slot_major, extra=70)
    g = torch.Generator().manual_seed(5)
    new = [70, 3, 0, 17]
    seq = [i for i, n in enumerate(new) for _ in range(n)]
    slot = [lens[i] + k for i, n in enumerate(new) for k in range(n)]
    pad = [5, 30]
    T = len(seq)
    slots = torch.tensor(slot, dtype=torch.int32)
    slots[pad] = -1
    seqs = torch.tensor(seq, dtype=torch.int32, device=dev())
    pos = torch.randint(-50, 100000, (T,), generator=g).to(torch.int32)
    qkv = torch.randn(T, n_q + 2 * n_kv, hd, generator=g).to(DT[dtype]).to(dev())
    q, k, v = qkv.split([n_q, n_kv, n_kv], dim=1)
    rope = lib.rope_desc(R, layout, 10000.0, "linear", 2.0)
    freqs = torch.empty(R // 2, dtype=torch.float64, device=dev())
    lib.tp_rope_freqs(rope, freqs)
    w, m = orope.frequencies(R, 10000.0, "linear", 2.0)
    kp0, vp0, tables = c.host()
    q_out = torch.full_like(q, float("nan"))
    from tests.test_gpu_rope import check as rope_check
    slots_d, pos_d = slots.to(dev()), pos.to(dev())
    lib.tp_kv_append_paged(c.desc, k, v, slots_d, c.tables, c.kp, c.vp, seq_ids=seqs, q=q,
                           q_out=q_out, rope=rope, freqs=freqs, positions=pos_d)
    lib.tp_check_device_error()
    rope_check(q_out, q, pos_d, R, layout, w, m, dtype)
    rot = torch.empty_like(k)
    lib.tp_rope(rope, k, pos_d, freqs, rot)
    rope_check(rot, k, pos_d, R, layout, w, m, dtype)
    for t in range(T):
        if t not in pad:
            p, s = tables[seq[t]][slot[t] // page], slot[t] % page
            kp0[p, :, s], vp0[p, :, s] = f64(rot)[t], f64(v)[t]
    # every slot that no token named is as it was
    assert np.array_equal(f64(c.kp), kp0, equal_nan=True) and np.array_equal(f64(c.vp), vp0, equal_nan=True)
    # q in place, positions of the slots
    want = torch.empty_like(q)
    lib.tp_rope(rope, q, slots_d, freqs, want)
    lib.tp_kv_append_paged(c.desc, k, v, slots_d, c.tables, c.kp, c.vp, seq_ids=seqs, q=q, q_out=q,
                           rope=rope, freqs=freqs)
    assert torch.equal(q, want)


def test_append_one_token_each_without_rotation(lib):
    c = Cache(lib, [40, 0, 9], 4, 2, 64, 16, extra=1)
    k, v = (torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(i)).bfloat16().to(dev())
            for i in (1, 2))
    lib.tp_kv_append_paged(c.desc, k, v, c.lens, c.tables, c.kp, c.vp)
    for i, n in enumerate(c.lens_l):
        p = int(c.tables[i, n // 16])
        assert torch.equal(c.kp[p, :, n % 16], k[i]) and torch.equal(c.vp[p, :, n % 16], v[i])


def test_append_indices_out_of_range(lib):
    c = Cache(lib, [40, 20], 4, 2, 64, 16, extra=8)
    kp, vp = c.kp.clone(), c.vp.clone()
    k = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=dev())
    i32 = dict(dtype=torch.int32, device=dev())
    lib.tp_check_device_error()
    for seq, slot in (([2, -1, 0, 0, 1], [40, 3, 1 << 20, c.cap, 31]), ([7] * 5, [0] * 5)):
        c.tables[1, 1] = 1000
        lib.tp_kv_append_paged(c.desc, k, k, torch.tensor(slot, **i32), c.tables, c.kp, c.vp,
                               seq_ids=torch.tensor(seq, **i32))
        with pytest.raises(lib.TpError) as e:
            lib.tp_check_device_error()
        assert e.value.status == lib.TP_ERR_INDEX
    same = lambda a, b: np.array_equal(f64(a), f64(b), equal_nan=True)
    assert same(c.kp, kp) and same(c.vp, vp)


# ----------------------------------------------------------------------------------- eviction
def run_evict(lib, c, budget, recent, in_place_lens=False):
    kp, vp, tables = c.host()
    keeps, score, kp, vp, nl = opaged.evict(c.score.cpu().numpy(), kp, vp, tables, c.lens_l, budget, recent)
    new_lens = c.lens if in_place_lens else torch.empty_like(c.lens)
    keep = torch.full((len(c.lens_l), c.n_kv, budget), 77, dtype=torch.int32, device=dev())
    ws = torch.full((lib.tp_kv_evict_paged_workspace(c.desc, budget),), 0xff, dtype=torch.uint8, device=dev())
    lib.tp_kv_evict_paged(c.desc, c.score, c.lens, budget, recent, c.kp, c.vp, c.tables, new_lens,
                          keep=keep, workspace=ws)
    assert new_lens.tolist() == nl
    for i, row in enumerate(keeps):
        for g, kept in enumerate(row):
            assert keep[i, g].tolist() == kept + [-1] * (budget - len(kept)), (i, g)
    assert np.array_equal(c.score.cpu().numpy(), score, equal_nan=True)
    assert np.array_equal(f64(c.kp), kp, equal_nan=True) and np.array_equal(f64(c.vp), vp, equal_nan=True)
    lib.tp_check_device_error()


@pytest.mark.parametrize("lens,budget,recent,n_kv,hd,page,dtype", [
    ([600], 512, 64, 8, 128, 16, "bf16"), ([2], 1, 0, 1, 8, 1, "bf16"), ([2], 1, 1, 1, 8, 1, "f32"),
    ([0, 1, 300, 77, 78], 77, 20, 2, 64, 24, "bf16"), ([5000, 1300, 2601], 1300, 0, 2, 32, 32, "bf16"),
    ([700, 90], 90, 90, 3, 80, 7, "f32"), ([2500, 2049], 2048, 1, 1, 256, 128, "f32"),
    ([3000], 2999, 100, 2, 96, 64, "bf16")])
@pytest.mark.parametrize("slot_major", [False, True])
def test_evict(lib, lens, budget, recent, n_kv, hd, page, dtype, slot_major):
    run_evict(lib, Cache(lib, lens, n_kv, n_kv, hd, page, dtype, slot_major=slot_major), budget, recent,
              in_place_lens=slot_major)


@pytest.mark.parametrize("kind", ["equal", "few values", "zeros of both signs", "nan", "infinite",
                                  "descending", "ascending", "negative"])
def test_evict_ties_and_special_scores(lib, kind):
    c = Cache(lib, [3000, 1400], 2, 2, 64, 16, seed=4)
    s = c.score
    if kind == "equal":
        s.fill_(0.25)
    elif kind == "few values":
        s.copy_((s * 4).floor())
    elif kind == "zeros of both signs":
        s.copy_(torch.where(s < 0.5, torch.zeros_like(s), -torch.zeros_like(s)))
    elif kind == "nan":
        s[s < 0.7] = float("nan")
    elif kind == "infinite":
        s[s < 0.2] = float("inf")
        s[s > 0.9] = -float("inf")
    elif kind == "descending":
        s.copy_(-torch.arange(s.shape[-1], device=dev()).float().expand_as(s))
    elif kind == "ascending":
        s.copy_(torch.arange(s.shape[-1], device=dev()).float().expand_as(s))
    else:
        s.copy_(-torch.exp(20 * s))
    run_evict(lib, c, 1111, 5)


def test_evict_scores_behind_the_length_are_not_read(lib):
    c = Cache(lib, [700, 650], 2, 2, 64, 16)
    for i, n in enumerate(c.lens_l):
        c.score[i, :, n:] = float("inf")
    run_evict(lib, c, 600, 10)


def test_evict_long(lib):
    # a row of scores that does not fit an SM's shared memory
    c = Cache(lib, [70001], 1, 1, 8, 64)
    run_evict(lib, c, 50001, 333)


def test_evict_captured(lib):
    c = Cache(lib, [900, 300], 2, 2, 64, 16)
    new_lens = torch.empty_like(c.lens)
    keep = torch.empty(2, 2, 500, dtype=torch.int32, device=dev())
    ws = torch.empty(lib.tp_kv_evict_paged_workspace(c.desc, 500), dtype=torch.uint8, device=dev())
    kp, vp, score = c.kp.clone(), c.vp.clone(), c.score.clone()
    args = (c.desc, c.score, c.lens, 500, 50, c.kp, c.vp, c.tables, new_lens)
    lib.tp_kv_evict_paged(*args, keep=keep, workspace=ws)
    want = [t.clone() for t in (c.kp, c.vp, c.score, keep)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.tp_kv_evict_paged(*args, keep=keep, workspace=ws)
    for t, s in ((c.kp, kp), (c.vp, vp), (c.score, score)):
        t.copy_(s)
    g.replay()
    for t, x in zip((c.kp, c.vp, c.score, keep), want):
        assert np.array_equal(f64(t), f64(x), equal_nan=True)


# ------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(lib, dtype):
    # prompts are appended, tokens decoded with their weights gathered, the cache is cut, decoding
    # goes on with positions that no longer equal the slots
    n_q, n_kv, hd, page, budget, recent = 8, 2, 64, 16, 48, 8
    g = torch.Generator().manual_seed(11)
    prompts = [70, 1, 33]
    b = len(prompts)
    c = Cache(lib, [0] * b, n_q, n_kv, hd, page, dtype, extra=100)
    c.score.zero_()
    rope = lib.rope_desc(hd, "half")
    freqs = torch.empty(hd // 2, dtype=torch.float64, device=dev())
    lib.tp_rope_freqs(rope, freqs)
    i32 = dict(dtype=torch.int32, device=dev())

    def append(seq, slots, pos):
        T = len(seq)
        qkv = torch.randn(T, n_q + 2 * n_kv, hd, generator=g).to(DT[dtype]).to(dev())
        q, k, v = qkv.split([n_q, n_kv, n_kv], dim=1)
        q_out = torch.empty(T, n_q, hd, dtype=DT[dtype], device=dev())
        lib.tp_kv_append_paged(c.desc, k, v, torch.tensor(slots, **i32), c.tables, c.kp, c.vp,
                               seq_ids=torch.tensor(seq, **i32), q=q, q_out=q_out, rope=rope,
                               freqs=freqs, positions=torch.tensor(pos, **i32))
        return q_out
    seq = [i for i, n in enumerate(prompts) for _ in range(n)]
    at = [s for n in prompts for s in range(n)]
    append(seq, at, at)
    lens, pos = list(prompts), list(prompts)
    for step in range(6):
        q = append(range(b), lens, pos)
        lens, pos = [n + 1 for n in lens], [p + 1 for p in pos]
        c.lens.copy_(torch.tensor(lens))
        c.lens_l = lens
        before = c.score.clone()
        c.check(*c.decode(q=q), before, q=q)
        if step == 3:
            run_evict(lib, c, budget, recent, in_place_lens=True)
            lens = c.lens.tolist()
            assert lens == [48, 5, 37]
            # the freed slots' weights start anew
            for i, n in enumerate(lens):
                c.score[i, :, n:] = 0
    lib.tp_check_device_error()


def test_tensors_elsewhere_are_refused(lib):
    c = Cache(lib, [40], 4, 2, 64, 16)
    with pytest.raises(ValueError):
        c.decode(q=c.q.cpu(), o=torch.empty_like(c.q))
    with pytest.raises(ValueError):
        c.decode(lens=c.lens.cpu())
    with pytest.raises(TypeError):
        c.decode(lens=c.lens.long())
    with pytest.raises(ValueError):
        c.decode(q=c.q[:, :2], o=torch.empty_like(c.q))
    with pytest.raises(lib.TpError) as e:
        c.decode(ws=torch.empty(16, dtype=torch.uint8, device=dev()))
    assert e.value.status == lib.TP_ERR_WORKSPACE
