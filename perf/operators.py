"""Workloads of the rotary and paged-cache operators, with their plain forms.

Four operators that stand around jagged attention: ``rotate`` (rotary
positions with several axes over packed rows, and its gradient),
``paged_tables`` (block tables, slots and positions of new tokens from request
lengths), ``paged_append`` (new keys and values into the pages, rotated on the
way) and ``paged_decode`` (attention of one new token over the paged cache).

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the calls of ``jagged_attention_gb300``.  Lengths follow from the
case alone (their order from the seed), tensors from the seed.
"""
from __future__ import annotations

import math
from statistics import NormalDist

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the dense query block of a broadcast workload (256 rows, 4 heads): one short call before the forward
        dict(name="rotate_query_block", op="rotate", rows=256, hq=4, hk=0, D=128, R=128, axes=3,
             interleaved=False, inverse=False, q32=False, far=4096, fused=False),
        # 768 sequences of 1024 tokens, 4 heads, q and k as slices of a fused projection, time/height/width positions
        dict(name="rotate_packed", op="rotate", rows=786432, hq=4, hk=4, D=128, R=128, axes=3,
             interleaved=False, inverse=False, q32=False, far=1000000, fused=True),
        # gradients of a jagged self-attention batch (32 sequences up to 1024): dQ in fp32, dK in bf16, part of the head turned
        dict(name="rotate_gradients", op="rotate", rows=17311, hq=4, hk=4, D=128, R=96, axes=2,
             interleaved=True, inverse=True, q32=True, far=131072, fused=False),
        # one decoding step of 256 requests: a token each, some of them leaving
        dict(name="tables_decode", op="tables", B=256, page=16, median=900, longest=8192, new=1, leave=8, spare=0),
        # a prefill step: 48 prompts of very different lengths enter, others leave
        dict(name="tables_prefill", op="tables", B=96, page=16, median=600, longest=16384, new=1024, leave=48,
             spare=500),
        # the new tokens of a decoding step: q, k, v from one projection, rotated and written, some rows padding
        dict(name="append_decode", op="append", rows=64, pad=3, hq=32, hk=8, D=128, R=128, axes=3,
             interleaved=False, page=16, pages=4096, far=131072, fused=True),
        # the keys and values of a prefill step, positions already in them
        dict(name="append_prefill", op="append", rows=32769, pad=31, hq=0, hk=8, D=128, R=0, axes=1,
             interleaved=False, page=16, pages=4096, far=32768, fused=False),
        # one request with a short cache: the latency of a call
        dict(name="decode_one_short", op="decode", B=1, hq=4, hk=4, D=128, page=16, median=300, longest=300,
             heads_first=False),
        # a batch of short requests and some long ones, grouped heads
        dict(name="decode_mixed", op="decode", B=128, hq=32, hk=8, D=128, page=16, median=512, longest=8192,
             heads_first=False),
        # one request with a long cache: all of the card has to work on one row
        dict(name="decode_one_long", op="decode", B=1, hq=32, hk=4, D=128, page=64, median=131072, longest=131072,
             heads_first=False),
        # odd sizes: one head of keys for twelve of queries, 64 wide, pages that end inside every tile, heads outside rows
        dict(name="decode_odd", op="decode", B=17, hq=12, hk=1, D=64, page=24, median=1200, longest=5001,
             heads_first=True),
        # a full cache
        dict(name="decode_full", op="decode", B=96, hq=64, hk=8, D=128, page=16, median=16384, longest=32768,
             heads_first=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "tables", "append", "decode", "decode"])
    D = rng.choice([64, 128])
    if op == "rotate":
        hq, hk = rng.choice([1, 2, 4, 5, 8, 16, 32]), rng.choice([0, 1, 2, 4, 8])
        rows = max(1, min(_log(rng, 1, 786432), 786432 * 8 * 128 // (2 * (hq + hk) * D)))
        return dict(op=op, rows=rows, hq=hq, hk=hk, D=D, R=16 * rng.randint(1, D // 16), axes=rng.randint(1, 4),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, q32=rng.random() < 0.4,
                    far=_log(rng, 16, 1 << 24), fused=rng.random() < 0.5)
    if op == "tables":
        B = _log(rng, 1, 2048)
        new = rng.choice([1, 1, 4, _log(rng, 1, 2048)])
        new = max(1, min(new, 131072 // B))
        return dict(op=op, B=B, page=rng.choice([1, 8, 16, 24, 32, 64, 128]), median=_log(rng, 16, 2048),
                    longest=_log(rng, 2048, 16384), new=new, leave=rng.randint(0, B // 2),
                    spare=rng.randint(0, 300))
    if op == "append":
        hk, rotary = rng.choice([1, 2, 4, 8]), rng.random() < 0.6
        hq = rng.choice([0, 1, 3, 8]) * hk if rotary else 0
        rows = _log(rng, 1, 32768)
        if hq:
            rows = max(1, min(rows, 32768 * 16 // (hq + 2 * hk)))
        page = rng.choice([1, 8, 16, 24, 64, 128])
        return dict(op=op, rows=rows, pad=rng.randint(0, min(rows - 1, 40)), hq=hq, hk=hk, D=D,
                    R=16 * rng.randint(1, D // 16) if rotary else 0, axes=rng.randint(1, 3),
                    interleaved=rng.random() < 0.5, page=page, pages=-(-max(rows, 4096) // page) + rng.randint(0, 64),
                    far=_log(rng, 64, 1 << 20), fused=rng.random() < 0.5)
    hk, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16, 24])
    B, longest = _log(rng, 1, 256), _log(rng, 1, 131072)
    longest = max(1, min(longest, 96 * 32768 * 8 // (2 * B * hk)))
    return dict(op=op, B=B, hq=hk * group, hk=hk, D=D, page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                median=max(1, int(longest * rng.choice([0.05, 0.3, 1.0]))), longest=longest,
                heads_first=rng.random() < 0.4)


def _lengths(case):
    """Log-normal lengths around the median, up to the longest, which one request has."""
    n, bell = case["B"], NormalDist()
    got = [int(round(case["median"] * math.exp(bell.inv_cdf((i + 0.5) / n)))) for i in range(n)]
    got = [max(0 if i == 1 else 1, min(case["longest"], v)) for i, v in enumerate(got)]
    got[-1] = case["longest"]
    if n > 2:
        got[0] = 0  # a request without a cache
    return got


def _deltas(case):
    """New tokens a request (negative: it leaves), for the lengths of _lengths."""
    lens, n = _lengths(case), case["B"]
    leave = {(i * n) // max(1, case["leave"]) for i in range(case["leave"])}
    got = [-v if i in leave else case["new"] if case["new"] <= 4 else 1 + (i * 7919) % (2 * case["new"] - 1)
           for i, v in enumerate(lens)]
    return [min(d, case["longest"] + 2 * case["new"] - v) for d, v in zip(got, lens)]


def _tables_sizes(case):
    lens, deltas, page = _lengths(case), _deltas(case), case["page"]
    rows = sum(max(0, d) for d in deltas) + case["spare"]
    width = -(-(case["longest"] + 2 * case["new"]) // page)
    held = [-(-v // page) for v in lens]
    need = [-(-(v + d) // page) for v, d in zip(lens, deltas)]
    return rows, width, sum(held), sum(max(0, a - b) for a, b in zip(need, held)), sum(max(0, b - a) for a, b in zip(need, held))


def work(case):
    D, op = case.get("D"), case["op"]
    if op == "rotate":
        item = case["rows"] * D * (case["hq"] * (4 if case["q32"] else 2) + case["hk"] * 2)
        pairs = case["rows"] * (case["hq"] + case["hk"]) * case["R"] // 2
        return {"bytes": 2 * item + 4 * case["rows"] * case["axes"], "flops": 6 * pairs}
    if op == "tables":
        rows, _, _, taken, freed = _tables_sizes(case)
        return {"bytes": 4 * (4 * case["B"] + 2 * (taken + freed) + 2 * rows), "flops": 8 * (case["B"] + rows)}
    if op == "append":
        live = case["rows"] - case["pad"]
        moved = 2 * 2 * D * (2 * live * case["hk"] + case["rows"] * case["hq"])
        return {"bytes": moved + 4 * case["rows"] * (1 + (case["axes"] if case["R"] else 0)),
                "flops": 3 * case["R"] * (live * case["hk"] + case["rows"] * case["hq"])}
    tokens, page = sum(_lengths(case)), case["page"]
    return {"bytes": 4 * tokens * case["hk"] * D + case["B"] * case["hq"] * (4 * D + 4)
            + 4 * (case["B"] + sum(-(-v // page) for v in _lengths(case))),
            "flops": 4 * tokens * case["hq"] * D}


# ------------------------------------------------------------- their inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32 if dtype == F32 else BF16)


def _pairs(case):
    """(inverse frequencies, axis of each pair): the axes share the pairs in runs, the first with the remainder."""
    half = case["R"] // 2
    freq = [10000.0 ** (-2.0 * i / case["R"]) for i in range(half)]
    axis = [max(0, i - half % case["axes"]) // max(1, half // case["axes"]) for i in range(half)]
    return freq, [min(a, case["axes"] - 1) for a in axis]


def _positions(case, g):
    return torch.randint(0, case["far"], (case["rows"], case["axes"]), generator=g, device="cuda").to(I32)


def _shuffled(values, g):
    order = torch.randperm(len(values), generator=g, device="cuda").cpu().tolist()
    return [values[i] for i in order]


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = dict(case=case)
    if own:  # the handles a user's program keeps
        import jagged_attention_gb300 as jfa
        s["jfa"] = jfa
    if case.get("R"):
        freq, axis = _pairs(case)
        s.update(freq=torch.tensor(freq, dtype=F64, device="cuda"), axis=torch.tensor(axis, device="cuda"),
                 positions=_positions(case, g))
        if own:
            s["rotary"] = s["jfa"].Rotary(freq, axis, D=case["D"], interleaved=case["interleaved"])
    if op == "rotate":
        n, hq, hk, D = case["rows"], case["hq"], case["hk"], case["D"]
        if case["fused"] and not case["q32"]:
            x = _normal((n, hq + 2 * hk, D), g)
            s.update(q=x[:, :hq], k=x[:, hq:hq + hk] if hk else None)
        else:
            s.update(q=_normal((n, hq, D), g, F32 if case["q32"] else BF16), k=_normal((n, hk, D), g) if hk else None)
        return s
    if op == "tables":
        rows, width, held, taken, freed = _tables_sizes(case)
        page, pages = case["page"], held + taken + 64
        pairs = _shuffled(list(zip(_lengths(case), _deltas(case))), g)
        order = torch.randperm(pages, generator=g, device="cuda").to(I32)
        table = torch.zeros((case["B"], width), dtype=I32)
        count = torch.tensor([-(-v // page) for v, _ in pairs])
        mask = torch.arange(width)[None, :] < count[:, None]
        table[mask] = order[:held].cpu()
        free = torch.zeros(pages, dtype=I32, device="cuda")
        free[:pages - held] = order[held:]
        s.update(lens=torch.tensor([v for v, _ in pairs], dtype=I32, device="cuda"),
                 delta=torch.tensor([d for _, d in pairs], dtype=I32, device="cuda"), table=table.cuda(), free=free,
                 n_free=torch.tensor([pages - held], dtype=I32, device="cuda"), rows=rows, page=page)
        if own:
            s["pager"] = s["jfa"].Pager(max_seqs=case["B"], max_pages=width, num_pages=pages, page_size=page,
                                        H=1, Hkv=1, D=128)
        return s
    if op == "append":
        n, hq, hk, D, page, pages = (case[k] for k in ("rows", "hq", "hk", "D", "page", "pages"))
        x = _normal((n, hq + 2 * hk, D), g)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(I32)
        slots[n - case["pad"]:] = -1
        s.update(q=q if hq else None, k=k, v=v, slots=slots, k_pages=_normal((pages, page, hk, D), g),
                 v_pages=_normal((pages, page, hk, D), g))
        if own:
            s["pager"] = s["jfa"].Pager(max_seqs=1, max_pages=pages, num_pages=pages, page_size=page,
                                        H=max(hq, hk), Hkv=hk, D=D)
        return s
    B, hq, hk, D, page = (case[k] for k in ("B", "hq", "hk", "D", "page"))
    lens = _shuffled(_lengths(case), g)
    count = torch.tensor([-(-v // page) for v in lens])
    pages, width = int(count.sum()) + 5, int(count.max())
    table = torch.zeros((B, width), dtype=I32)
    order = torch.randperm(pages, generator=g, device="cuda").to(I32).cpu()
    table[torch.arange(width)[None, :] < count[:, None]] = order[:int(count.sum())]
    shape = (pages, hk, page, D) if case["heads_first"] else (pages, page, hk, D)
    k_pages, v_pages = _normal(shape, g), _normal(shape, g)
    if case["heads_first"]:
        k_pages, v_pages = k_pages.transpose(1, 2), v_pages.transpose(1, 2)
    s.update(q=_normal((B, hq, D), g), k_pages=k_pages, v_pages=v_pages, table=table.cuda(),
             lens=torch.tensor(lens, dtype=I32, device="cuda"), scale=1.0 / math.sqrt(D))
    if own:
        s["pager"] = s["jfa"].Pager(max_seqs=B, max_pages=width, num_pages=pages, page_size=page, H=hq, Hkv=hk, D=D)
        s["out"] = torch.empty((B, hq, D), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((hq, B), dtype=F32, device="cuda")
    return s


# ------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "rotate":
        sign = -1.0 if case["inverse"] else 1.0
        cos, sin = _cos_sin(s)
        got = [_turn(s["q"], cos, sign * sin, case["interleaved"])]
        if s["k"] is not None:
            got.append(_turn(s["k"], cos, sign * sin, case["interleaved"]))
        return got
    return {"tables": _tables, "append": _append, "decode": _decode}[case["op"]](s, case)


def _own(s, case):
    jfa, op = s["jfa"], case["op"]
    if op == "rotate":
        got = jfa.rotate(s["rotary"], s["positions"], s["q"], s["k"], inverse=case["inverse"])
        return [got] if s["k"] is None else list(got)
    if op == "tables":
        lens, n_free, slots, positions, offsets = jfa.paged_tables(
            s["pager"], s["lens"], s["delta"], s["table"], s["free"], s["n_free"], rows=s["rows"])
        return lens, n_free, slots, positions, offsets, s["table"], s["free"]
    if op == "append":
        q = jfa.paged_append(s["pager"], s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"],
                             rotary=s.get("rotary"), positions=s.get("positions"), q=s["q"])
        return [s["k_pages"], s["v_pages"]] + ([] if q is None else [q])
    return jfa.paged_decode(s["pager"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"],
                            out=s["out"], lse=s["lse"])


def _cos_sin(s):
    angle = s["positions"].to(F64)[:, s["axis"]] * s["freq"]
    return torch.cos(angle).to(F32), torch.sin(angle).to(F32)


def _turn(x, cos, sin, interleaved):
    half, y = cos.shape[1], x.to(F32)
    c, z = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * z, b * c + a * z), dim=-1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * c - b * z, b * c + a * z), dim=-1)
    return torch.cat((turned, y[..., 2 * half:]), dim=-1).to(x.dtype)


def _tables(s, case):
    lens, delta, table, free, page = s["lens"].long(), s["delta"].long(), s["table"], s["free"], s["page"]
    rows, width, n_free = s["rows"], table.shape[1], s["n_free"].long()
    after = lens + delta
    held, need = (lens + page - 1) // page, (after + page - 1) // page
    grow, shrink = (need - held).clamp(min=0), (held - need).clamp(min=0)
    take, give = grow.cumsum(0) - grow, shrink.cumsum(0) - shrink
    j = torch.arange(width, device="cuda")[None, :]
    # pages that go back come onto the free list's end, and are taken from there again
    back = (j >= need[:, None]) & (j < held[:, None])
    stack = torch.cat((free, free[:1]))
    stack[torch.where(back, n_free + give[:, None] + j - need[:, None], len(free))] = table
    stack = stack[:-1]
    top = n_free + shrink.sum()
    new = (j >= held[:, None]) & (j < need[:, None])
    source = (top - 1 - take[:, None] - (j - held[:, None])).clamp(0, len(free) - 1)
    table = torch.where(new, stack[source], table)
    count = delta.clamp(min=0)
    offsets = torch.cat((count.new_zeros(1), count.cumsum(0)))
    r = torch.arange(rows, device="cuda")
    owner = torch.searchsorted(offsets, r, right=True) - 1
    live = r < offsets[-1]
    owner = owner.clamp(max=len(lens) - 1)
    position = torch.where(live, lens[owner] + r - offsets[owner], 0)
    slots = table[owner, position // page].long() * page + position % page
    return (after.to(I32), (top - grow.sum()).to(I32), torch.where(live, slots, -1).to(I32), position.to(I32),
            offsets.to(I32), table, stack)


def _append(s, case):
    k, q, interleaved = s["k"], s["q"], case["interleaved"]
    if case["R"]:
        cos, sin = _cos_sin(s)
        k = _turn(k, cos, sin, interleaved)
        q = None if q is None else _turn(q, cos, sin, interleaved)
    n = case["rows"] - case["pad"]  # the rows behind are padding
    at = s["slots"][:n].long()
    s["k_pages"].flatten(0, 1)[at] = k[:n]
    s["v_pages"].flatten(0, 1)[at] = s["v"][:n]
    return [s["k_pages"], s["v_pages"]] + ([] if q is None else [q])


def _decode(s, case):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    B, H, D = q.shape
    hk = case["hk"]
    k = s["k_pages"][table].flatten(1, 2).to(F32)  # [B, tokens, hk, D]
    score = torch.einsum("bhgd,bthd->bhgt", q.to(F32).view(B, hk, H // hk, D), k) * s["scale"]
    del k
    score = score.masked_fill(torch.arange(score.shape[-1], device="cuda") >= lens[:, None, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_pages"][table].flatten(1, 2).to(F32)
    out = torch.einsum("bhgt,bthd->bhgd", p, v) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, H, D).to(BF16), (top + torch.log(total)).reshape(B, H).T.contiguous()


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s, case)
    if case["R"]:
        axis = s["axis"].cpu().tolist()
        angle = torch.stack([s["positions"][:, a].double() * f for a, f in zip(axis, s["freq"].cpu().tolist())], 1)
        turn = torch.polar(torch.ones_like(angle), -angle if case.get("inverse") else angle)
    outs = []
    for name in ("q", "k"):
        x = s[name]
        if x is None or x.numel() == 0:
            continue
        y = x.double()
        if case["R"]:
            for h in range(x.shape[1]):
                part = y[:, h, :case["R"]].clone()
                if case["interleaved"]:
                    z = torch.view_as_complex(part.view(len(x), -1, 2).contiguous()) * turn
                    y[:, h, :case["R"]] = torch.view_as_real(z).reshape(len(x), -1)
                else:
                    z = torch.complex(*part.chunk(2, dim=1)) * turn
                    y[:, h, :case["R"]] = torch.cat((z.real, z.imag), dim=1)
        outs.append(y)
    if case["op"] == "rotate":
        return outs
    k = outs.pop()
    pages = []
    for new, held in ((k, s["k_pages"]), (s["v"].double(), s["v_pages"])):
        rows = held.double().view(-1, *held.shape[2:])
        live = s["slots"] >= 0
        rows[s["slots"][live].long()] = new[live]
        pages.append(rows.view(held.shape))
    return pages + outs


def _exact_decode(s, case):
    B, H, D = s["q"].shape
    group = H // case["hk"]
    out = torch.zeros((B, H, D), dtype=F64, device="cuda")
    lse = torch.full((H, B), -math.inf, dtype=F64, device="cuda")
    for b, n in enumerate(s["lens"].cpu().tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["hk"]):
            k, v = (s[x][pages, :, h].reshape(-1, D)[:n].double() for x in ("k_pages", "v_pages"))
            heads = slice(h * group, (h + 1) * group)
            score = s["q"][b, heads].double() @ k.T * s["scale"]
            lse[heads, b] = torch.logsumexp(score, 1)
            out[b, heads] = torch.softmax(score, 1) @ v
    return out, lse
