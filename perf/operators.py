"""Timing cases of the serving-side attention operators: rotary positions, the append of new tokens
to a paged key/value cache, decode attention over that cache, and eviction by accumulated weight.

Each case is a dict of plain values.  ``prepare`` makes a case's inputs on the GPU, ``run`` makes
one pass: with ``own`` false by elementary torch operations in 32 bits (angles in 64), with ``own``
true by the library's calls.  ``exact`` computes the same outputs in 64 bits from the definition.
"""

import math
import random

import torch

own = False

# Head layouts: 64 query heads on 8 KV heads of 128 dims is this repository's attention block.


def listed():
    return [
        # a whole prompt's queries and keys (64 + 8 heads) before prefill attention
        dict(name="rope prefill", op="rope", T=4096, heads=72, hd=128, rot=128, layout="half",
             scaling="none", base=10000.0, factor=1.0, orig=0, far=4096, inverse=False, dtype="bf16"),
        # training at long context: the gradient of a part-rotated, interleaved fp32 tensor
        dict(name="rope gradient far", op="rope", T=2051, heads=16, hd=96, rot=64,
             layout="interleaved", scaling="parts", base=500000.0, factor=8.0, orig=8192,
             far=1000000, inverse=True, dtype="f32"),
        # one decode step of a batch: rotate q and k, put k and v into their pages
        dict(name="append decode", op="append", b=64, n_q=64, n_kv=8, hd=128, rot=128,
             layout="half", scaling="linear", base=10000.0, factor=4.0, orig=4096, page=16,
             len=4096, new=1, dtype="bf16"),
        # ragged prompts of a batch written after their prefill
        dict(name="append prompts", op="append", b=7, n_q=32, n_kv=4, hd=128, rot=64,
             layout="interleaved", scaling="ntk", base=10000.0, factor=2.0, orig=2048, page=64,
             len=900, new=900, dtype="bf16"),
        # the first tokens of one conversation: latency alone
        dict(name="decode one short", op="decode", b=1, n_q=64, n_kv=8, hd=128, page=16, len=200,
             ragged=False, dtype="bf16", weights=False),
        # a full batch of conversations at the decode stack's cache length
        dict(name="decode batch", op="decode", b=16, n_q=64, n_kv=8, hd=128, page=16, len=4096,
             ragged=True, dtype="bf16", weights=False),
        # one long document: parallel over the cache's length alone
        dict(name="decode one long", op="decode", b=1, n_q=64, n_kv=8, hd=128, page=64,
             len=131071, ragged=False, dtype="bf16", weights=False),
        # the largest: many long conversations of different lengths
        dict(name="decode large", op="decode", b=32, n_q=64, n_kv=8, hd=128, page=32, len=16384,
             ragged=True, dtype="bf16", weights=False),
        # fp32 blocks, one query head per KV head, pages that are no power of two
        dict(name="decode fp32", op="decode", b=9, n_q=12, n_kv=12, hd=64, page=24, len=1111,
             ragged=True, dtype="f32", weights=False),
        # decode that also keeps the accumulated attention weight of every key
        dict(name="decode weights", op="decode", b=16, n_q=64, n_kv=8, hd=128, page=16, len=4100,
             ragged=True, dtype="bf16", weights=True),
        # one conversation that just passed its cache budget
        dict(name="evict one", op="evict", b=1, n_q=64, n_kv=8, hd=128, page=16, len=600,
             ragged=False, budget=512, recent=64, dtype="bf16"),
        # a batch cut back to half of its cache
        dict(name="evict batch", op="evict", b=24, n_q=64, n_kv=8, hd=128, page=32, len=8000,
             ragged=True, budget=4096, recent=256, dtype="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    hd = rng.choice([32, 64, 80, 96, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n_kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 5, 8, 8, 16])
    n_q = n_kv * group
    page = rng.choice([8, 16, 24, 32, 64, 128])
    rot = rng.choice([hd, hd, hd // 2])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "parts"])
    pos = dict(rot=rot, layout=layout, scaling=scaling, base=rng.choice([10000.0, 500000.0]),
               factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
               orig=rng.choice([2048, 4096, 8192]))
    if op == "rope":
        T = log(1, 6000)
        return dict(op="rope", T=T, heads=log(1, max(1, min(96, 16_000_000 // (T * hd)))), hd=hd,
                    far=log(max(T, 16), 1000000), inverse=rng.random() < 0.5, dtype=dtype, **pos)
    if op == "append":
        new = rng.choice([1, 1, log(2, 1500)])
        b = log(1, max(1, min(128, 6000 // new)))
        return dict(op="append", b=b, n_q=n_q, n_kv=n_kv, hd=hd, page=page,
                    len=max(new, log(1, 4096)), new=new, dtype=dtype, **pos)
    e = 2 if dtype == "bf16" else 4
    b = log(1, 64)
    most = 500_000_000 // (b * n_kv * hd * e * 2)  # keys per sequence: a quarter of the largest
    if op == "decode":
        return dict(op="decode", b=b, n_q=n_q, n_kv=n_kv, hd=hd, page=page,
                    len=log(1, max(64, min(100000, most))), ragged=rng.random() < 0.7, dtype=dtype,
                    weights=rng.random() < 0.4)
    n = log(64, max(128, min(30000, most // 2)))
    budget = max(2, int(n * rng.uniform(0.2, 0.95)))
    return dict(op="evict", b=b, n_q=n_q, n_kv=n_kv, hd=hd, page=page, len=n,
                ragged=rng.random() < 0.5, budget=budget, recent=int(budget * rng.uniform(0, 0.5)),
                dtype=dtype)


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case):
    """The sequences' lengths: of the case alone.  Ragged batches span an eighth to the whole."""
    if not case.get("ragged"):
        return [case["len"]] * case["b"]
    r = random.Random(case["len"] * 131 + case["b"])
    lens = [max(1, int(case["len"] * r.uniform(0.125, 1.0))) for _ in range(case["b"])]
    lens[0] = case["len"]
    return lens


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std)


def _pool(g, case, cap, dtype):
    """A shuffled pool of pages: [n_pages][n_kv][page][hd] twice, and the sequences' tables."""
    b, page = case["b"], case["page"]
    used = [-(-n // page) for n in cap]
    n_pages, width = sum(used) + 3, max(used)
    kp = torch.empty(n_pages, case["n_kv"], page, case["hd"], dtype=dtype, device="cuda")
    vp = torch.empty_like(kp)
    kp.normal_(generator=g)
    vp.normal_(generator=g)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(used, device="cuda")
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col[None, :]).clamp_(max=n_pages - 1)
    tables = torch.where(col[None, :] < n[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
    return kp, vp, tables.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DT[case["dtype"]]
    st = {"case": case}
    op = case["op"]
    if op == "rope":
        st["x"] = _normal(g, case["T"], case["heads"], case["hd"]).to(dt)
        # a run of positions, as of one sequence, somewhere below the farthest
        start = torch.randint(0, max(1, case["far"] - case["T"] + 1), (1,), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(case["T"], device="cuda")).to(torch.int32)
        st["out"] = torch.empty_like(st["x"])
    elif op == "append":
        b, new, T = case["b"], case["new"], case["b"] * case["new"]
        st["kp"], st["vp"], st["tables"] = _pool(g, case, [case["len"]] * b, dt)
        # the projection's output: q, k and v of a token side by side
        qkv = _normal(g, T, case["n_q"] + 2 * case["n_kv"], case["hd"]).to(dt)
        st["q"], st["k"], st["v"] = qkv.split([case["n_q"], case["n_kv"], case["n_kv"]], dim=1)
        st["seq_ids"] = torch.arange(b, device="cuda").repeat_interleave(new).to(torch.int32)
        first = torch.randint(0, case["len"] - new + 1, (b, 1), generator=g, device="cuda")
        st["positions"] = (first + torch.arange(new, device="cuda")[None]).reshape(-1).to(torch.int32)
        st["q_out"] = torch.empty(T, case["n_q"], case["hd"], dtype=dt, device="cuda")
    else:
        lens = _lens(case)
        st["kp"], st["vp"], st["tables"] = _pool(g, case, lens, dt)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cap = st["tables"].shape[1] * case["page"]
        if op == "decode":
            st["q"] = _normal(g, case["b"], case["n_q"], case["hd"], std=2.0).to(dt)
            st["o"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(case["b"], case["n_q"], device="cuda")
            if case["weights"]:  # what earlier steps gathered
                st["score"] = _normal(g, case["b"], case["n_kv"], cap).abs_()
        else:
            # accumulated weights: a few keys hold most of it
            st["score"] = _normal(g, case["b"], case["n_kv"], cap, std=2.0).exp_()
            st["new_lens"] = torch.empty_like(st["lens"])
            st["keep"] = torch.empty(case["b"], case["n_kv"], case["budget"], dtype=torch.int32,
                                     device="cuda")
            # the kept rows' sequence and slot, known to the program from its lengths
            n = [min(x, case["budget"]) for x in lens]
            st["rows"] = (torch.arange(case["b"], device="cuda").repeat_interleave(torch.tensor(n, device="cuda")),
                          torch.cat([torch.arange(x) for x in n]).cuda())
    if own:
        from tensor_transformer_matmul_b200 import tpblock as tp
        if op in ("rope", "append"):
            st["rope"] = tp.rope_desc(case["rot"], case["layout"], case["base"], case["scaling"],
                                      case["factor"], case["orig"])
            st["freqs"] = torch.empty(case["rot"] // 2, dtype=torch.float64, device="cuda")
            tp.tp_rope_freqs(st["rope"], st["freqs"])
        if op != "rope":
            st["desc"] = tp.paged_desc(case["n_q"], st["kp"], st["tables"])
        if op == "decode":
            st["ws"] = torch.empty(tp.tp_attn_decode_paged_workspace(st["desc"], case["weights"]),
                                   dtype=torch.uint8, device="cuda")
        if op == "evict":
            st["ws"] = torch.empty(tp.tp_kv_evict_paged_workspace(st["desc"], case["budget"]),
                                   dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------- plain forms
def _freqs(case):
    """Angle per position of each pair, and the magnitude of the rotated part."""
    R, base, s = case["rot"], case["base"], case["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk":
        base = base * s ** (R / (R - 2))
    w = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        return w / s, 1.0
    if case["scaling"] == "parts":
        turns = case["orig"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return w * (keep + (1 - keep) / s), 0.1 * math.log(s) + 1.0
    return w, 1.0


def _rotate(x, positions, case, inverse=False):
    w, mag = _freqs(case)
    a = positions.double()[:, None] * w[None]
    c, s = (a.cos() * mag).float()[:, None], (a.sin() * mag).float()[:, None]
    if inverse:
        s = -s
    R = case["rot"]
    x = x.float()
    r = x[..., :R]
    if case["layout"] == "half":
        x1, x2 = r[..., : R // 2], r[..., R // 2:]
        y = torch.cat([x1 * c - x2 * s, x1 * s + x2 * c], -1)
    else:
        x1, x2 = r[..., 0::2], r[..., 1::2]
        y = torch.stack([x1 * c - x2 * s, x1 * s + x2 * c], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _logical(pages, tables):
    """[b][n_kv][keys][hd] of the paged array (table entries of no page read page 0)."""
    t = pages[tables.clamp(min=0).long()]
    b, n, h, p, d = t.shape
    return t.permute(0, 2, 1, 3, 4).reshape(b, h, n * p, d)


def _append(st):
    case = st["case"]
    st["q_out"].copy_(_rotate(st["q"], st["positions"], case))
    seq, pos = st["seq_ids"].long(), st["positions"].long()
    page = st["tables"][seq, pos // case["page"]].long()
    slot = pos % case["page"]
    st["kp"][page, :, slot] = _rotate(st["k"], st["positions"], case).to(st["kp"].dtype)
    st["vp"][page, :, slot] = st["v"]
    return st["q_out"], st["kp"], st["vp"]


def _decode(st):
    case = st["case"]
    b, n_kv, hd = case["b"], case["n_kv"], case["hd"]
    k = _logical(st["kp"], st["tables"]).float()
    q = st["q"].float().view(b, n_kv, -1, hd)
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    del k
    there = torch.arange(s.shape[-1], device="cuda")[None, :] < st["lens"][:, None]
    s.masked_fill_(~there[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    p /= l
    v = _logical(st["vp"], st["tables"]).float()
    v.masked_fill_(~there[:, None, :, None], 0.0)
    st["o"].copy_((p @ v).view(b, -1, hd))
    st["lse"].copy_((m + l.log()).view(b, -1))
    if not case["weights"]:
        return st["o"], st["lse"]
    st["score"] += p.sum(2)
    return st["o"], st["lse"], st["score"]


def _evict(st):
    case, lens = st["case"], st["lens"][:, None, None]
    cap, budget = st["score"].shape[-1], case["budget"]
    pos = torch.arange(cap, device="cuda")
    rank = torch.where(pos < lens - case["recent"], st["score"], math.inf)
    rank = torch.where(pos < lens, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = order.sort(dim=-1).values
    seq, j = st["rows"]
    page, slot = st["tables"][seq, j // case["page"]].long(), j % case["page"]
    for pages in (st["kp"], st["vp"]):
        rows = _logical(pages, st["tables"]).gather(2, keep[..., None].expand(-1, -1, -1, case["hd"]))
        pages[page, :, slot] = rows[seq, :, j]
    live = torch.arange(keep.shape[-1], device="cuda") < lens
    moved = st["score"].gather(2, keep)
    st["score"][..., : keep.shape[-1]] = torch.where(live, moved, st["score"][..., : keep.shape[-1]])
    st["keep"].fill_(-1)
    st["keep"][..., : keep.shape[-1]] = torch.where(live, keep, -1)
    torch.clamp(st["lens"], max=budget, out=st["new_lens"])
    return st["keep"], st["new_lens"], st["score"], st["kp"], st["vp"]


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        from tensor_transformer_matmul_b200 import tpblock as tp
        if op == "rope":
            tp.tp_rope(st["rope"], st["x"], st["positions"], st["freqs"], st["out"],
                       inverse=case["inverse"])
            return st["out"]
        if op == "append":
            tp.tp_kv_append_paged(st["desc"], st["k"], st["v"], st["positions"], st["tables"],
                                  st["kp"], st["vp"], seq_ids=st["seq_ids"], q=st["q"],
                                  q_out=st["q_out"], rope=st["rope"], freqs=st["freqs"])
            return st["q_out"], st["kp"], st["vp"]
        if op == "decode":
            tp.tp_attn_decode_paged(st["desc"], st["q"], st["kp"], st["vp"], st["tables"],
                                    st["lens"], st["o"], lse=st["lse"], score=st.get("score"),
                                    workspace=st["ws"])
            return (st["o"], st["lse"], st["score"]) if case["weights"] else (st["o"], st["lse"])
        tp.tp_kv_evict_paged(st["desc"], st["score"], st["lens"], case["budget"], case["recent"],
                             st["kp"], st["vp"], st["tables"], st["new_lens"], keep=st["keep"],
                             workspace=st["ws"])
        return st["keep"], st["new_lens"], st["score"], st["kp"], st["vp"]
    if op == "rope":
        st["out"].copy_(_rotate(st["x"], st["positions"], case, case["inverse"]))
        return st["out"]
    return {"append": _append, "decode": _decode, "evict": _evict}[op](st)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, hd = case["op"], case["hd"]
    if op == "rope":
        n = case["T"] * case["heads"]
        return {"bytes": 2 * n * hd * e + 4 * case["T"], "flops": 3 * n * case["rot"]}
    if op == "append":
        T = case["b"] * case["new"]
        return {"bytes": 2 * T * (case["n_q"] + 2 * case["n_kv"]) * hd * e + 12 * T,
                "flops": 3 * T * (case["n_q"] + case["n_kv"]) * case["rot"]}
    lens = _lens(case)
    if op == "decode":
        keys = sum(lens)
        rows = case["b"] * case["n_q"]
        return {"bytes": 2 * keys * case["n_kv"] * hd * e + rows * (2 * hd * e + 4)
                + (8 * keys * case["n_kv"] if case["weights"] else 0),
                "flops": 4 * keys * case["n_q"] * hd}
    cut = [n for n in lens if n > case["budget"]]
    per = 4 * sum(cut) + len(cut) * case["budget"] * (4 + 4 * hd * e)
    kept = 4 * sum(min(n, case["budget"]) for n in lens)
    return {"bytes": case["n_kv"] * (per + kept), "flops": case["n_kv"] * sum(cut)}


# -------------------------------------------------------------------------- 64-bit definition
def _angles64(case, positions):
    """(cos, sin) times the magnitude: one frequency at a time, as the definition reads."""
    out_c, out_s = [], []
    R, s = case["rot"], case["factor"]
    mag = 1.0
    for i in range(R // 2):
        theta = math.pow(case["base"], -2.0 * i / R)
        if case["scaling"] == "linear":
            theta /= s
        elif case["scaling"] == "ntk":
            theta = math.pow(case["base"] * math.pow(s, R / (R - 2.0)), -2.0 * i / R)
        elif case["scaling"] == "parts":
            r = case["orig"] * theta / (2.0 * math.pi)
            ramp = min(1.0, max(0.0, (r - 1.0) / 31.0))
            theta = (1.0 - ramp) * theta / s + ramp * theta
            mag = 1.0 + 0.1 * math.log(s)
        angle = positions.double() * theta
        out_c.append(torch.cos(angle) * mag)
        out_s.append(torch.sin(angle) * mag)
    return torch.stack(out_c, 1), torch.stack(out_s, 1)


def _rope64(case, x, positions, sign):
    c, s = _angles64(case, positions)
    s = s * sign
    y = x.double().clone()
    half = case["rot"] // 2
    for i in range(half):
        a, b = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        u, w = x[:, :, a].double(), x[:, :, b].double()
        y[:, :, a] = u * c[:, i, None] - w * s[:, i, None]
        y[:, :, b] = w * c[:, i, None] + u * s[:, i, None]
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, page = case["op"], case.get("page")
    if op == "rope":
        return _rope64(case, st["x"], st["positions"], -1.0 if case["inverse"] else 1.0)
    if op == "append":
        kp, vp = st["kp"].double(), st["vp"].double()
        k = _rope64(case, st["k"], st["positions"], 1.0)
        where = st["tables"].long()[st["seq_ids"].long(), torch.div(st["positions"].long(), page, rounding_mode="floor")]
        flat = where * page + torch.remainder(st["positions"].long(), page)
        for dst, src in ((kp, k), (vp, st["v"].double())):
            for h in range(case["n_kv"]):
                plane = dst[:, h].reshape(-1, case["hd"])
                plane[flat] = src[:, h]
                dst[:, h] = plane.view(-1, page, case["hd"])
        return _rope64(case, st["q"], st["positions"], 1.0), kp, vp
    lens = _lens(case)
    group = case["n_q"] // case["n_kv"]
    if op == "decode":
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        score = st["score"].double() if case["weights"] else None
        for i, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            pg = st["tables"][i].long()[at // page]
            for h in range(case["n_kv"]):
                k, v = st["kp"][pg, h, at % page].double(), st["vp"][pg, h, at % page].double()
                q = st["q"][i, h * group:(h + 1) * group].double()
                z = torch.mm(q, k.t()) / math.sqrt(case["hd"])
                w = torch.softmax(z, 1)
                o[i, h * group:(h + 1) * group] = torch.mm(w, v)
                lse[i, h * group:(h + 1) * group] = torch.logsumexp(z, 1)
                if score is not None:
                    score[i, h, :n] += w.sum(0)
        return (o, lse, score) if case["weights"] else (o, lse)
    kp, vp, score = st["kp"].double(), st["vp"].double(), st["score"].double()
    keep = torch.full(st["keep"].shape, -1, dtype=torch.int32, device="cuda")
    budget, recent = case["budget"], case["recent"]
    for i, n in enumerate(lens):
        for h in range(case["n_kv"]):
            if n <= budget:
                keep[i, h, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
                continue
            w = st["score"][i, h, : n - recent]
            best = torch.argsort(-w, stable=True)[: budget - recent]
            kept = torch.cat([torch.sort(best).values, torch.arange(n - recent, n, device="cuda")])
            keep[i, h] = kept.to(torch.int32)
            score[i, h, :budget] = st["score"][i, h, kept].double()
            new = torch.arange(budget, device="cuda")
            frm, to = st["tables"][i].long()[kept // page], st["tables"][i].long()[new // page]
            kp[to, h, new % page] = st["kp"][frm, h, kept % page].double()
            vp[to, h, new % page] = st["vp"][frm, h, kept % page].double()
    return keep, torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device="cuda"), score, kp, vp
