"""Workloads of the operators on a key/value cache held in 8 or 4 bits, with their plain forms.

Three operators: ``append`` (``paged_append`` into such a cache: new keys, rotated on
the way, and values are quantised as they are written, and read back as the prompt's
attention sees them), ``gather`` (``paged_gather``: cached rows of requests read back
into packed bf16 rows, as ``fwd`` takes them) and ``decode`` (``paged_decode``:
attention of one new token per request over the cached codes).

How a row of a head is held:

* 8 bits: e4m3 codes, and one byte c for all of them: value = code * 2^(c - 127).
  2^(c - 127) is the least power of two that takes the row's largest magnitude to at
  most 448, c from 79 to 175; 255 where a value is not finite: all of them are NaN then.
* 4 bits: e2m1 codes, the value of the lower nibble first, and a byte for each 16: the
  scale, in 5 exponent and 3 mantissa bits (bits 14 to 7 of the fp16 number), is the
  block's largest magnitude / 6, rounded to nearest even, 10240 at most; 255 where a
  value is not finite: the 16 are NaN then.

Either way a value is divided by its scale and rounded to nearest even, and what
is larger than the largest code is that.  Keys that are rotated are rounded to bf16
first, as they would be in a cache of 16 bits.

``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through the calls of ``jagged_attention_gb300``.  Lengths follow from the
case alone (their order from the seed), tensors from the seed.
"""
from __future__ import annotations

import math
from statistics import NormalDist

import torch

own = False

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the new tokens of a decoding step, 64 requests: q, k, v from one projection, rotated; a launch each
        dict(name="append8_step", op="append", bits=8, B=64, new=1, median=700, longest=4000, pad=3, hq=32, hk=8, D=128,
             R=128, axes=3, interleaved=False, page=16, fused=True, whole=False),
        # prompts of very different lengths enter, and are read back for their attention
        dict(name="append4_prompts", op="append", bits=4, B=48, new=680, median=0, longest=0, pad=31, hq=0, hk=8, D=128,
             R=128, axes=1, interleaved=False, page=16, fused=False, whole=False),
        # chunks of prompts of which a part is cached, odd sizes, part of the head turned; read back with what was there
        dict(name="append8_chunks", op="append", bits=8, B=13, new=301, median=900, longest=5001, pad=0, hq=0, hk=3, D=64,
             R=32, axes=2, interleaved=True, page=24, fused=False, whole=True),
        # a few short requests read back: the latency of a call
        dict(name="gather8_short", op="gather", bits=8, B=4, median=200, longest=300, hk=4, D=128, page=16,
             heads_first=False, tail=0),
        # the cached prefixes of a large batch
        dict(name="gather4_prefixes", op="gather", bits=4, B=96, median=2048, longest=16384, hk=8, D=128, page=16,
             heads_first=False, tail=0),
        # one request with a short cache: the latency of a call
        dict(name="decode8_one_short", op="decode", bits=8, B=1, hq=4, hk=4, D=128, page=16, median=300, longest=300,
             heads_first=False),
        # a batch of short requests and some long ones, grouped heads
        dict(name="decode8_mixed", op="decode", bits=8, B=128, hq=32, hk=8, D=128, page=16, median=512, longest=8192,
             heads_first=False),
        # a full cache of 8 bits
        dict(name="decode8_full", op="decode", bits=8, B=96, hq=64, hk=8, D=128, page=16, median=16384, longest=32768,
             heads_first=False),
        # odd sizes: one head of keys for twelve of queries, 64 wide, pages that end inside every tile, heads outside rows
        dict(name="decode4_odd", op="decode", bits=4, B=17, hq=12, hk=1, D=64, page=24, median=1200, longest=5001,
             heads_first=True),
        # the mixed batch in 4 bits
        dict(name="decode4_mixed", op="decode", bits=4, B=128, hq=32, hk=8, D=128, page=16, median=512, longest=8192,
             heads_first=False),
        # one request with a long cache: all of the card has to work on one row
        dict(name="decode4_one_long", op="decode", bits=4, B=1, hq=32, hk=4, D=128, page=64, median=131072,
             longest=131072, heads_first=False),
        # a full cache of 4 bits
        dict(name="decode4_full", op="decode", bits=4, B=96, hq=64, hk=8, D=128, page=16, median=16384, longest=32768,
             heads_first=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, bits, D = rng.choice(["append", "gather", "decode", "decode"]), rng.choice([8, 4]), rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128])
    if op == "append":
        hk, rotary = rng.choice([1, 2, 3, 4, 8]), rng.random() < 0.7
        hq = rng.choice([0, 1, 3, 8]) * hk if rotary else 0
        most = 32768 * 16 // (hq + 2 * hk)  # rows
        B = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, most // B))
        longest = rng.choice([0, _log(rng, 1, max(1, min(8192, 4 * most // B)))])
        return dict(op=op, bits=bits, B=B, new=new, median=longest // rng.choice([1, 3, 10]), longest=longest,
                    pad=rng.randint(0, 40), hq=hq, hk=hk, D=D, R=16 * rng.randint(1, D // 16) if rotary else 0,
                    axes=rng.randint(1, 3), interleaved=rng.random() < 0.5, page=page, fused=rng.random() < 0.5,
                    whole=rng.random() < 0.4)
    hk = rng.choice([1, 2, 3, 4, 8])
    B, longest = _log(rng, 1, 256), _log(rng, 1, 131072)
    if op == "gather":
        longest = max(1, min(longest, 400000 * 8 // (B * hk)))
        return dict(op=op, bits=rng.choice([bits, bits, 16]), B=B, median=max(1, int(longest * rng.choice([0.05, 0.3, 1.0]))),
                    longest=longest, hk=hk, D=D, page=page, heads_first=rng.random() < 0.4,
                    tail=rng.choice([0, 0, _log(rng, 1, 64)]))
    group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16, 24])
    longest = max(1, min(longest, 96 * 32768 * 8 // (2 * B * hk)))
    return dict(op=op, bits=bits, B=B, hq=hk * group, hk=hk, D=D, page=page,
                median=max(1, int(longest * rng.choice([0.05, 0.3, 1.0]))), longest=longest,
                heads_first=rng.random() < 0.4)


def _lengths(case):
    """Log-normal lengths around the median, up to the longest, which one request has."""
    n, bell = case["B"], NormalDist()
    if case["longest"] == 0:
        return [0] * n
    got = [int(round(case["median"] * math.exp(bell.inv_cdf((i + 0.5) / n)))) for i in range(n)]
    got = [max(0 if i == 1 else 1, min(case["longest"], v)) for i, v in enumerate(got)]
    got[-1] = case["longest"]
    if n > 2:
        got[0] = 0  # a request without a cache
    return got


def _news(case):
    """New rows of each request: one each, or spread evenly from 1 to 2 new - 1."""
    return [1 + (i * 7919) % (2 * case["new"] - 1) for i in range(case["B"])]


def _scale_bytes(case):
    return 1 if case["bits"] == 8 else case["D"] // 16 if case["bits"] == 4 else 0


def _row_bytes(case):
    """Bytes of a cached row of one head, key or value."""
    return case["D"] * case["bits"] // 8 + _scale_bytes(case)


def _read_rows(case):
    """Rows of each request that a pass reads back."""
    lens = _lengths(case)
    if case["op"] == "append":
        return [n + d if case["whole"] else d for n, d in zip(lens, _news(case))]
    return [min(n, case["tail"]) if case["tail"] else n for n in lens]


def work(case):
    D, hk, lens, pages = case["D"], case["hk"], _lengths(case), lambda v: -(-v // case["page"])
    if case["op"] == "decode":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * hk * _row_bytes(case) + case["B"] * case["hq"] * (4 * D + 4)
                + 4 * (case["B"] + sum(pages(v) for v in lens)), "flops": 4 * tokens * case["hq"] * D}
    read = sum(_read_rows(case))
    back = read * hk * (2 * 2 * D)  # the rows written as bf16
    if case["op"] == "gather":
        return {"bytes": back + 2 * read * hk * _row_bytes(case) + 4 * sum(pages(v) for v in _read_rows(case)),
                "flops": 2 * read * hk * D}
    new, rows = sum(_news(case)), sum(_news(case)) + case["pad"]
    old = read - new if case["whole"] else 0  # new rows need not be read again: they were just made
    return {"bytes": back + 2 * D * (2 * new * hk + 2 * rows * case["hq"]) + 2 * (new + old) * hk * _row_bytes(case)
            + 4 * rows * (1 + (case["axes"] if case["R"] else 0)),
            "flops": 3 * case["R"] * (new * hk + rows * case["hq"]) + 4 * 2 * new * hk * D}


# ------------------------------------------------------------- their inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _channels(hk, D, g):
    """Keys have some channels that are larger than others."""
    return torch.exp(0.6 * _normal((hk, D), g, F32))


def _pairs(case):
    """(inverse frequencies, axis of each pair): the axes share the pairs in runs, the first with the remainder."""
    half = case["R"] // 2
    freq = [10000.0 ** (-2.0 * i / case["R"]) for i in range(half)]
    axis = [max(0, i - half % case["axes"]) // max(1, half // case["axes"]) for i in range(half)]
    return freq, [min(a, case["axes"] - 1) for a in axis]


def _offsets(counts):
    at = torch.zeros(len(counts) + 1, dtype=I32)
    at[1:] = torch.tensor(counts).cumsum(0)
    return at.cuda()


def _cache(case, pages, g):
    """Pages full of quantised rows: codes [pages, page, hk, D bits / 8] and scale bytes [pages, page, hk, n]."""
    s, hk, D, page, bits = {}, case["hk"], case["D"], case["page"], case["bits"]
    some = max(1, (1 << 28) // (page * hk * D))  # pages quantised at once
    heads_first = case.get("heads_first", False)
    for x in ("k", "v"):
        size = _channels(hk, D, g) if x == "k" else 0.4
        shape = [pages, hk, page, D] if heads_first else [pages, page, hk, D]
        if bits == 16:
            held = (_normal(shape, g, F32) * (size[:, None] if heads_first and x == "k" else size)).to(BF16)
        else:
            held = torch.empty(shape[:3] + [D * bits // 8], dtype=U8, device="cuda")
            scales = torch.empty((pages, hk, page, _scale_bytes(case)), dtype=U8, device="cuda").transpose(1, 2)
            s[x + "_scales"] = scales
        for at in range(0, pages if bits < 16 else 0, some):
            n = min(some, pages - at)
            codes, bytes_ = _quantise((_normal((n, page, hk, D), g, F32) * size).to(BF16), bits)
            (held.transpose(1, 2) if heads_first else held)[at:at + n] = codes
            scales[at:at + n] = bytes_
        s[x + "_pages"] = held.transpose(1, 2) if heads_first else held
    return s


def _table(case, lens, g):
    """(block table, pages): pages dealt out at random, five of nobody."""
    count = torch.tensor([-(-v // case["page"]) for v in lens])
    pages, width = int(count.sum()) + 5, max(1, int(count.max()))
    table = torch.zeros((len(lens), width), dtype=I32)
    order = torch.randperm(pages, generator=g, device="cuda").to(I32).cpu()
    table[torch.arange(width)[None, :] < count[:, None]] = order[:int(count.sum())]
    return table.cuda(), pages


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    B, hk, D, page, bits = (case[x] for x in ("B", "hk", "D", "page", "bits"))
    hq = case.get("hq") or hk
    order = torch.randperm(B, generator=g, device="cuda").cpu().tolist()
    lens, counts = [_lengths(case)[i] for i in order], None
    s = dict(case=case)
    if op != "decode":
        counts = [_read_rows(case)[i] for i in order]
        s.update(offsets=_offsets(counts), rows=sum(counts), starts=None)
    if op == "append":
        news = [_news(case)[i] for i in order]
        ends = [a + b for a, b in zip(lens, news)]
        if not case["whole"]:
            s["starts"] = torch.tensor(lens, dtype=I32, device="cuda")
    else:
        ends = lens
        if op == "gather" and case["tail"]:
            s["starts"] = torch.tensor([a - b for a, b in zip(lens, counts)], dtype=I32, device="cuda")
    s["table"], pages = _table(case, ends, g)
    s.update(_cache(case, pages, g))
    if op == "append":
        n = sum(news) + case["pad"]
        x = _normal((n, case["hq"] + 2 * hk, D), g)
        x[:, case["hq"]:case["hq"] + hk] *= _channels(hk, D, g).to(BF16)
        q, k, v = x[:, :case["hq"]], x[:, case["hq"]:case["hq"] + hk], x[:, case["hq"] + hk:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        owner = torch.repeat_interleave(torch.arange(B), torch.tensor(news)).cuda()
        at = torch.arange(sum(news), device="cuda")
        pos = torch.tensor(lens, device="cuda")[owner] + at - _offsets(news).long()[owner]
        slots = torch.full((n,), -1, dtype=I32, device="cuda")  # the rows behind are padding
        slots[:len(at)] = (s["table"][owner, pos // page] * page + pos % page).to(I32)
        s.update(q=q if case["hq"] else None, k=k, v=v, slots=slots)
        if case["R"]:
            freq, axis = _pairs(case)
            where = torch.zeros((n, case["axes"]), dtype=I32, device="cuda")
            where[:len(at), 0] = pos.to(I32)
            if case["axes"] > 1:
                where[:, 1:] = torch.randint(0, 4096, (n, case["axes"] - 1), generator=g, device="cuda").to(I32)
            s.update(freq=torch.tensor(freq, dtype=F64, device="cuda"), axis=torch.tensor(axis, device="cuda"),
                     positions=where)
    if op == "decode":
        s.update(q=_normal((B, hq, D), g), lens=torch.tensor(lens, dtype=I32, device="cuda"), scale=1.0 / math.sqrt(D))
    if own:  # the handles and buffers a user's program keeps
        import jagged_attention_gb300 as jfa
        s["jfa"] = jfa
        s["pager"] = jfa.Pager(max_seqs=B, max_pages=s["table"].shape[1], num_pages=pages, page_size=page, H=hq, Hkv=hk,
                               D=D, bits=bits)
        if case.get("R"):
            s["rotary"] = jfa.Rotary(*_pairs(case), D=D, interleaved=case["interleaved"])
        if op == "decode":
            s["out"] = torch.empty((B, hq, D), dtype=BF16, device="cuda")
            s["lse"] = torch.empty((hq, B), dtype=F32, device="cuda")
    return s


# ------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"append": _append, "gather": _gather, "decode": _decode}[case["op"]](s, case)


def _own(s, case):
    jfa, op = s["jfa"], case["op"]
    held = dict(k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
    if op == "decode":
        return jfa.paged_decode(s["pager"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scale"],
                                out=s["out"], lse=s["lse"], **held)
    q = None
    if op == "append":
        q = jfa.paged_append(s["pager"], s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"],
                             rotary=s.get("rotary"), positions=s.get("positions"), q=s["q"], **held)
    k, v = jfa.paged_gather(s["pager"], s["k_pages"], s["v_pages"], s["table"], s["offsets"], rows=s["rows"],
                            starts=s["starts"], **held)
    return [k, v] if q is None else [k, v, q]


def _quantise(x, bits):
    """(codes, scale bytes) of bf16 values [..., D], as the file's head says."""
    y = x.to(F32)
    if bits == 8:
        top = y.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(top / 448.0)  # m in [1/2, 1): 2^(e - 1) where m is 1/2, else 2^e
        e = torch.where(m == 0.5, e - 1, torch.where(m == 0, -48, e)).clamp(-48, 48)
        codes = torch.ldexp(y, -e).clamp(-448.0, 448.0).to(E4M3).view(U8)
        return codes, torch.where(torch.isfinite(top), e + 127, 255).to(U8)
    blocks = y.unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    third = (top / 6.0).clamp(max=10240.0)
    step = torch.ldexp(torch.ones_like(third), (torch.frexp(third)[1] - 4).clamp(min=-17))
    scale = torch.round(third / step) * step  # 4 bits, multiples of 2^-17
    byte = (scale.to(torch.float16).view(torch.int16) >> 7).to(U8)
    z = torch.where(scale[..., None] > 0, blocks / scale[..., None], 0.0).abs()
    code = (z > 0.25).to(U8) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0)
    code = (code | torch.signbit(blocks).to(U8) << 3).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4), torch.where(torch.isfinite(top), byte, 255).to(U8)


def _values(codes, scales, bits):
    """fp32 values of codes [..., D bits / 8] and their scale bytes."""
    if bits == 16:
        return codes.to(F32)
    if bits == 8:
        by = torch.ldexp(torch.ones_like(scales, dtype=F32), scales.to(I32) - 127)
        return codes.view(E4M3).to(F32) * torch.where(scales == 255, math.nan, by)
    both = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    low = (both & 7).to(F32)
    # 0, 1/2, 1, 3/2, 2, 3, 4, 6
    size = torch.where(low < 4, 0.5 * low, torch.where(low < 6, low - 2.0, 2.0 * low - 8.0))
    by = (scales.to(torch.int16) << 7).view(torch.float16).to(F32)
    signed = torch.where(both > 7, -size, size)
    return (signed.unflatten(-1, (-1, 16)) * by[..., None]).flatten(-2)


def _at(s, x, index):
    """fp32 values of the cached rows `index` = (pages, rows)."""
    scales = s.get(x + "_scales")
    return _values(s[x + "_pages"][index], None if scales is None else scales[index], s["case"]["bits"])


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


def _append(s, case):
    k, q, page = s["k"], s["q"], case["page"]
    if case["R"]:
        cos, sin = _cos_sin(s)
        k = _turn(k, cos, sin, case["interleaved"])
        q = None if q is None else _turn(q, cos, sin, case["interleaved"])
    n = len(k) - case["pad"]
    at = s["slots"][:n].long()
    at = at // page, at % page
    for x, new in (("k", k), ("v", s["v"])):
        s[x + "_pages"][at], s[x + "_scales"][at] = _quantise(new[:n], case["bits"])
    return _gather(s, case) + ([] if q is None else [q])


def _gather(s, case):
    offsets, page = s["offsets"].long(), case["page"]
    r = torch.arange(s["rows"], device="cuda")
    owner = torch.searchsorted(offsets, r, right=True) - 1
    t = r - offsets[owner]
    if s["starts"] is not None:
        t = t + s["starts"].long()[owner]
    at = s["table"][owner, t // page].long(), t % page
    return [_at(s, x, at).to(BF16) for x in ("k", "v")]


def _decode(s, case):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    B, H, D = q.shape
    hk, page = case["hk"], case["page"]
    t = torch.arange(table.shape[1] * page, device="cuda")
    at = table[:, t // page], t % page
    k = _at(s, "k", at)  # [B, tokens, hk, D]
    score = torch.einsum("bhgd,bthd->bhgt", q.to(F32).view(B, hk, H // hk, D), k) * s["scale"]
    del k
    score = score.masked_fill(torch.arange(score.shape[-1], device="cuda") >= lens[:, None, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgt,bthd->bhgd", p, _at(s, "v", at)) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, H, D).to(BF16), (top + torch.log(total)).reshape(B, H).T.contiguous()


# ------------------------------------------------- the definition in 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e4m3_table():
    """Values of the 127 finite codes without sign, in order."""
    low = [m / 8 * 2.0 ** -6 for m in range(8)]
    return low + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]


def _nearest(x, grid):
    """Each |x| at its nearest grid value, halves to the even place, the last for all above."""
    grid = torch.tensor(grid, dtype=F64, device=x.device)
    size = x.abs().clamp(max=float(grid[-1]))
    up = torch.searchsorted(grid, size).clamp(1, len(grid) - 1)  # the first not below
    below, above = size - grid[up - 1], grid[up] - size
    up = torch.where((below < above) | ((below == above) & (up % 2 == 1)), up - 1, up)
    return torch.copysign(grid[up], x)


def _held(x, bits):
    """What a cache of that many bits holds of finite bf16 values [..., D], in 64 bits."""
    y = x.double()
    if bits == 8:
        top = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448.0).clamp(-48, 48))
        for by in (e - 1, e + 1):  # log2 may be off where the quotient is near a power of two
            fits = top <= 448.0 * torch.exp2(by)
            e = torch.where(fits & (by < e) & (by >= -48), by, torch.where(~(top <= 448.0 * torch.exp2(e)) & (by > e) & (by <= 48), by, e))
        return _nearest(y / torch.exp2(e), _e4m3_table()) * torch.exp2(e)
    grid = [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 29) for m in range(8)]
    blocks = y.unflatten(-1, (-1, 16))
    scale = _nearest(blocks.abs().amax(-1, keepdim=True) / 6.0, [v for v in grid if v <= 10240.0])
    codes = _nearest(torch.where(scale > 0, blocks / torch.where(scale > 0, scale, 1.0), 0.0), _E2M1)
    return (codes * scale).flatten(-2)


def _decoded(codes, scales, bits):
    """float64 values of codes, by tables of the two formats."""
    if bits == 16:
        return codes.double()
    if bits == 8:
        one = _e4m3_table() + [math.nan]
        table = torch.tensor(one + [-v for v in one], dtype=F64, device="cuda")
        return table[codes.long()] * torch.exp2(scales.double() - 127)
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=F64, device="cuda")
    value = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=F64, device="cuda")
    value[..., 0::2], value[..., 1::2] = table[codes.long() % 16], table[codes.long() // 16]
    b = scales.double()
    e, m = torch.floor(b / 8), b % 8
    by = torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e - 18))
    return value * by.repeat_interleave(16, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s, case)
    page, table = case["page"], s["table"].cpu()
    slots = []
    offsets, starts = s["offsets"].tolist(), None if s["starts"] is None else s["starts"].tolist()
    for b in range(case["B"]):
        t = torch.arange(offsets[b + 1] - offsets[b]) + (starts[b] if starts else 0)
        slots.append(table[b, t // page].long() * page + t % page)
    slots = torch.cat(slots).cuda()
    got = []
    for x in ("k", "v"):
        scales = s.get(x + "_scales")
        at = slots // page, slots % page
        got.append(_decoded(s[x + "_pages"][at], None if scales is None else scales[at], case["bits"]))
    if case["op"] == "gather":
        return got
    turned = {"k": s["k"], "q": s["q"]}
    if case["R"]:
        axis = s["axis"].cpu().tolist()
        angle = torch.stack([s["positions"][:, a].double() * f for a, f in zip(axis, s["freq"].cpu().tolist())], 1)
        turn = torch.polar(torch.ones_like(angle), angle)
        for name, x in turned.items():
            y = None if x is None else x.double()
            for h in range(0 if x is None else x.shape[1]):
                part = y[:, h, :case["R"]].clone()
                if case["interleaved"]:
                    z = torch.view_as_complex(part.view(len(x), -1, 2).contiguous()) * turn
                    y[:, h, :case["R"]] = torch.view_as_real(z).reshape(len(x), -1)
                else:
                    z = torch.complex(*part.chunk(2, dim=1)) * turn
                    y[:, h, :case["R"]] = torch.cat((z.real, z.imag), dim=1)
            turned[name] = y
    # the new rows take the places of what was cached there
    new_slots = s["slots"][s["slots"] >= 0].long()
    place = torch.full((s["k_pages"].shape[0] * page,), -1, dtype=torch.long, device="cuda")
    place[new_slots] = torch.arange(len(new_slots), device="cuda")
    source = place[slots]
    for i, new in enumerate((turned["k"].to(BF16), s["v"])):
        got[i][source >= 0] = _held(new, case["bits"])[source[source >= 0]]
    return got + ([] if s["q"] is None else [turned["q"]])


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
            k, v = (_decoded(s[x + "_pages"][pages, :, h].flatten(0, 1)[:n], s[x + "_scales"][pages, :, h].flatten(0, 1)[:n],
                             case["bits"]) for x in ("k", "v"))
            heads = slice(h * group, (h + 1) * group)
            score = s["q"][b, heads].double() @ k.T * s["scale"]
            lse[heads, b] = torch.logsumexp(score, 1)
            out[b, heads] = torch.softmax(score, 1) @ v
    return out, lse
