"""GPU tests of decode over 8 and 4 bits with scores of any size that the header allows: of
rows alike, where the output is known whatever the score, and of rows far below others."""
import math

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import coded_ref

pytestmark = pytest.mark.gpu
BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
STEP = torch.finfo(BF16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _draw(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


class Case:
    """A cache of requests of `lens` rows, of given values, on pages in order."""

    def __init__(self, bits, lens, hq, hk, D, page, k, v):
        self.bits, self.lens, self.scale = bits, lens, None
        count = [-(-n // page) for n in lens]
        self.pager = jfa.Pager(max_seqs=len(lens), max_pages=max(count), num_pages=sum(count), page_size=page, H=hq, Hkv=hk, D=D,
                               bits=bits)
        self.held = self.pager.pages()
        table, slots, at = np.full((len(lens), max(count)), -1), [], 0
        for b, n in enumerate(count):
            table[b, :n] = np.arange(at, at + n)
            slots.append(at * page + np.arange(lens[b]))
            at += n
        self.table = torch.as_tensor(table, dtype=I32).cuda()
        self.offsets = torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32).cuda()
        self.scales = dict(k_scales=self.held[2], v_scales=self.held[3])
        jfa.paged_append(self.pager, k, v, torch.as_tensor(np.concatenate(slots), dtype=I32).cuda(), *self.held[:2], **self.scales)

    def rows(self):
        """Cached values of each request, [n, Hkv, D] in 64 bits: (k, v)."""
        k, v = jfa.paged_gather(self.pager, *self.held[:2], self.table, self.offsets, rows=sum(self.lens), **self.scales)
        return list(zip(k.double().split(self.lens), v.double().split(self.lens)))

    def decode(self, q, scale):
        lens = torch.as_tensor(self.lens, dtype=I32).cuda()
        got = jfa.paged_decode(self.pager, q, *self.held[:2], self.table, lens, scale, **self.scales)
        again = jfa.paged_decode(self.pager, q, *self.held[:2], self.table, lens, scale, **self.scales)
        assert self.pager.status() == 0
        assert torch.equal(got[0].view(torch.int16), again[0].view(torch.int16))  # bit for bit, NaN too
        assert torch.equal(got[1].view(I32), again[1].view(I32))
        return got


def _bound(w, v, n, delta):
    """Of |out error| for weights w [rows] right to delta in their exponents, as coded_ref.decode: the
    sums, a weight's rounding to fp16, or half its smallest number, and the output's rounding."""
    mass, most = w @ v.abs(), v.abs().amax()
    off = (2 * delta + coded_ref.FP16_HALF_STEP) * mass + n * 2.0 ** -39 * most
    return off * (1 + STEP) + STEP * (w @ v).abs()


SIZES = [-3, 9, 10, 13, 20, 22, 23, 24, 25, 26, 27, 28, 31, 40, 77, 100]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,hq,hk", [(64, 4, 2), (128, 8, 1), (128, 24, 1), (64, 12, 1)])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_of_one_key(bits, D, hq, hk, sign):
    """All rows of a request have the same key: whatever their score, the output is the mean of the
    values, and log-sum-exp the score and log n.  One row, a tile of them, and many CTAs' worth."""
    lens = [1, 2, 64, 70, 3000, 1]
    rows = sum(lens)
    key = _draw((1, hk, D), 1).expand(rows, hk, D).contiguous()
    v = (_draw((rows, hk, D), 2).float() * torch.exp2(torch.randint(-20, 20, (rows, hk, 1), device="cuda").float())).to(BF16)
    case = Case(bits, lens, hq, hk, D, 16, key, v)
    cached = case.rows()
    base = _draw((len(lens), hq, D), 3) * sign
    for size in SIZES:
        # powers of two shared by q and the scale, each within its type
        q = (base.float() * 2.0 ** min(size, 60)).to(BF16)
        scale = 2.0 ** max(0, size - 60) / 8
        out, lse = case.decode(q, scale)
        for b, n in enumerate(lens):
            k, val = cached[b]
            for h in range(hq):
                g = h // (hq // hk)
                score = scale * float(q[b, h].double() @ k[0, g])
                # equal scores leave no error but what the powers of values add: scores up to 2^10 times log2 e
                # are rounded with them, to 2^-14 (half a step at 2^10 is 2^-14)
                delta = 2.0 ** -14 + 2.0 ** -17 + 2 * n * 2.0 ** -24
                w = torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")
                err = (out[b, h].double() - w @ val[:, g]).abs()
                assert (err <= _bound(w, val[:, g], n, delta)).all(), (size, b, h, float(err.max()))
                size_of = scale * float(q[b, h].double().abs() @ k[0, g].abs())
                off = 2 * D * 2.0 ** -24 * size_of + 2.0 ** -22 * (abs(score) + math.log(n) + 1) + delta
                assert abs(float(lse[h, b]) - score - math.log(n)) <= off, (size, b, h)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 24, 2.0 ** 26, 2.0 ** 33, 2.0 ** 90])
@pytest.mark.parametrize("hq,hk", [(4, 2), (8, 1), (24, 1)])
@pytest.mark.parametrize("where", ["first", "last", "spread", "one"])
def test_rows_far_above_and_below(bits, size, hq, hk, where):
    """Some rows' scores are so far above the rest that these count for nothing, or (q turned round) the
    other way: the output is the mean of the rows on top, wherever a stretch meets them."""
    D, lens = 64, [3, 200, 2500]
    rows = sum(lens)
    key, flags = _draw((hk, D), 1), []
    for n in lens:
        flag = np.zeros(n, dtype=bool)
        if where == "first":
            flag[:max(1, n // 3)] = True
        elif where == "last":
            flag[-max(1, n // 3):] = True
        elif where == "spread":
            flag[::7] = True
        else:
            flag[n // 2] = True
        flags.append(torch.as_tensor(flag).cuda())
    big = torch.cat(flags)
    k = torch.where(big[:, None, None], key, key / 8)
    v = _draw((rows, hk, D), 2)
    case = Case(bits, lens, hq, hk, D, 16, k, v)
    cached = case.rows()
    # a query that has the same sign as its key everywhere: scores of size and an eighth of it
    q = (key.sign()[:, None].expand(hk, hq // hk, D).reshape(1, hq, D).expand(len(lens), hq, D)).contiguous()
    per = float((q[0].double().view(hk, -1, D) * cached[1][0][big[3:203]][0][:, None].double()).sum(-1).min())
    scale = size / per
    for sign in (1, -1):
        out, lse = case.decode(q * sign, scale)
        for b, n in enumerate(lens):
            on_top = flags[b] if sign == 1 else ~flags[b]
            count = int(on_top.sum())
            val = cached[b][1][on_top]
            for h in range(hq):
                g = h // (hq // hk)
                w = torch.full((count,), 1.0 / count, dtype=torch.float64, device="cuda")
                delta = 2.0 ** -14 + 2.0 ** -17 + 2 * n * 2.0 ** -24
                # rows of 4 bits that are alike in bf16 are alike in codes; those below weigh exp(-size 7 / 8) at most
                assert ((out[b, h].double() - w @ val[:, g]).abs() <= _bound(w, val[:, g], n, delta)).all(), (sign, b, h)
                assert torch.isfinite(lse[h, b])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("size", [2.0 ** 11, 2.0 ** 25, 2.0 ** 33, 2.0 ** 60, 2.0 ** 100, math.inf])
@pytest.mark.parametrize("hq,hk,D", [(8, 1, 64), (12, 1, 128), (16, 2, 128)])
def test_heads_beside_one_of_large_scores(bits, size, hq, hk, D):
    """One head's large scores, as of what an unused head may hold up to the type's largest number
    (inf here), leave the heads beside it within their bounds."""
    lens = [700, 40, 5000]
    case = Case(bits, lens, hq, hk, D, 16, _draw((sum(lens), hk, D), 1), _draw((sum(lens), hk, D), 2))
    q = _draw((len(lens), hq, D), 3)
    if size < math.inf:
        q[:, 3] = (q[:, 3].float() * (size / 8)).to(BF16)
    else:
        q[:, 3] = torch.finfo(BF16).max * q[:, 3].sign()
    out, lse = case.decode(q, D ** -0.5)
    others = [h for h in range(hq) if h != 3]
    assert torch.isfinite(out[:, others]).all() and torch.isfinite(lse[others]).all()
    assert size == math.inf or torch.isfinite(out).all() and torch.isfinite(lse).all()
    for b, (k, v) in enumerate(case.rows()):
        n = lens[b]
        for h in others:
            g = h // (hq // hk)
            s = D ** -0.5 * (k[:, g] @ q[b, h].double())
            w = torch.softmax(s, 0)
            reach = D ** -0.5 * float((k[:, g].abs() @ q[b, h].double().abs()).max())
            delta = 2 * D * 2.0 ** -24 * reach + 2.0 ** -17 + 2 * n * 2.0 ** -24
            assert ((out[b, h].double() - w @ v[:, g]).abs() <= _bound(w, v[:, g], n, delta)).all(), (b, h)
            assert abs(float(lse[h, b]) - float(torch.logsumexp(s, 0))) <= delta + 2.0 ** -23 * abs(float(lse[h, b]))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hk,D", [(8, 1, 64), (24, 1, 128), (16, 4, 128)])
def test_heads_of_very_different_sizes(bits, hq, hk, D):
    """Heads from 2^-60 to 2^60 of one another, each with scores of its own size."""
    lens = [300, 64, 1]
    case = Case(bits, lens, hq, hk, D, 16, _draw((sum(lens), hk, D), 1), _draw((sum(lens), hk, D), 2))
    power = torch.linspace(-60, 60, hq, device="cuda").round()
    base = _draw((len(lens), hq, D), 3)
    q = (base.float() * torch.exp2(power)[:, None]).to(BF16)
    for scale in (2.0 ** -60, 2.0 ** 20):
        out, lse = case.decode(q, scale)
        for b, (k, v) in enumerate(case.rows()):
            n = lens[b]
            for h in range(hq):
                g = h // (hq // hk)
                s = scale * (k[:, g] @ q[b, h].double())
                reach = scale * float((k[:, g].abs() @ q[b, h].double().abs()).max())
                if reach > 100:
                    continue  # the bound says nothing any more
                w = torch.softmax(s, 0)
                delta = 2 * D * 2.0 ** -24 * reach + 2.0 ** -17 + 2 * n * 2.0 ** -24
                assert ((out[b, h].double() - w @ v[:, g]).abs() <= _bound(w, v[:, g], n, delta)).all(), (b, h)
                assert abs(float(lse[h, b]) - float(torch.logsumexp(s, 0))) <= delta + 2.0 ** -23 * abs(float(lse[h, b]))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("power,scale", [(120, 2.0 ** 30), (127, 2.0 ** 126), (-126, 2.0 ** -126), (120, 0.0), (0, -(2.0 ** 126))])
def test_keys_of_zeros(bits, power, scale):
    """The score of a key of zeros is 0 whatever the query and the scale, each within its limit."""
    lens, hq, hk, D = [1, 100, 2000], 8, 2, 64
    v = _draw((sum(lens), hk, D), 2)
    case = Case(bits, lens, hq, hk, D, 16, torch.zeros_like(v), v)
    out, lse = case.decode((_draw((len(lens), hq, D), 3).sign().float() * 2.0 ** power).to(BF16), scale)
    for b, (_, val) in enumerate(case.rows()):
        n = lens[b]
        w = torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")
        delta = 2.0 ** -17 + 2 * n * 2.0 ** -24
        for h in range(hq):
            assert ((out[b, h].double() - w @ val[:, h // 4]).abs() <= _bound(w, val[:, h // 4], n, delta)).all(), (b, h)
            assert abs(float(lse[h, b]) - math.log(n)) <= delta + 2.0 ** -22 * (1 + math.log(n))


@pytest.mark.parametrize("bits", [8, 4])
def test_queries_and_scales_at_their_limit(bits):
    """A query times the scale of 2^138, and keys small enough for a score of 2^124."""
    lens, hq, hk, D = [1, 100, 2000], 8, 2, 64
    v = _draw((sum(lens), hk, D), 2)
    key = torch.zeros_like(v)
    key[..., 0] = 6 * 2.0 ** -17
    case = Case(bits, lens, hq, hk, D, 16, key, v)
    q = torch.full((len(lens), hq, D), 2.0 ** 110, device="cuda").to(BF16)
    for scale in (2.0 ** 28, -(2.0 ** 28)):
        out, lse = case.decode(q, scale)
        for b, (k, val) in enumerate(case.rows()):
            n, score = lens[b], scale * 2.0 ** 110 * float(k[0, 0].sum())
            assert 2.0 ** 110 < abs(score) < 2.0 ** 127
            w = torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")
            for h in range(hq):
                assert ((out[b, h].double() - w @ val[:, h // 4]).abs() <= _bound(w, val[:, h // 4], n, 2.0 ** -17 + 2 * n * 2.0 ** -24)).all()
                assert abs(float(lse[h, b]) / score - 1) <= 2 * D * 2.0 ** -24


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 64), (12, 1, 128), (24, 1, 128)])
@pytest.mark.parametrize("captured", [False, True])
def test_requests_beside_ones_of_large_scores(bits, hq, hk, D, captured):
    """A warp's share goes over several requests, every second of large scores, and a graph is
    replayed with queries that are large where they were not: nothing is left over from one to the next."""
    B, page = 12000, 64
    rng = np.random.default_rng(hq)
    lens = rng.integers(1, page + 1, B).tolist()
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).cuda()
    odd = (torch.arange(B, device="cuda") % 2 == 1)[:, None, None]
    k = torch.where(odd[owner], _draw((B, hk, D), 1)[owner], _draw((sum(lens), hk, D), 4))  # odd ones' rows have one key
    case = Case(bits, lens, hq, hk, D, page, k, _draw((sum(lens), hk, D), 2))
    dl, at = torch.as_tensor(lens, dtype=I32).cuda(), torch.arange(B + 1, device="cuda", dtype=I32) * page
    kd, vd = jfa.paged_gather(case.pager, *case.held[:2], case.table, at, rows=B * page, **case.scales)
    dead = torch.arange(page, device="cuda")[None, None] >= dl[:, None, None]
    base, q = _draw((B, hq, D), 3), torch.empty((B, hq, D), dtype=BF16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((hq, B), device="cuda")

    def call():
        jfa.paged_decode(case.pager, q, *case.held[:2], case.table, dl, D ** -0.5, **case.scales, out=out, lse=lse)

    q.copy_(base)
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            call()
    for size in (2.0 ** 30, 1.0, -(2.0 ** 60), 2.0 ** 13):
        q.copy_(torch.where(odd, base.float() * size, base.float()).to(BF16))
        graph.replay() if captured else call()
        assert case.pager.status() == 0
        for g in range(hk):
            heads = slice(g * hq // hk, (g + 1) * hq // hk)
            key, val = (x.view(B, page, hk, D)[:, :, g].double() for x in (kd, vd))
            s = D ** -0.5 * torch.einsum("bhd,btd->bht", q[:, heads].double(), key)
            reach = D ** -0.5 * torch.einsum("bhd,btd->bht", q[:, heads].double().abs(), key.abs()).amax(2, keepdim=True)
            s = s.masked_fill(dead, -math.inf)
            # rows of one key have one score, whatever its error
            delta = 2.0 ** -14 + 2.0 ** -17 + 2 * page * 2.0 ** -24 + torch.where(odd, 0.0, 2 * D * 2.0 ** -24 * reach)
            w = torch.where(odd, (~dead) / dl.double()[:, None, None], torch.softmax(s, 2))
            want, mass = torch.einsum("bht,btd->bhd", w, val), torch.einsum("bht,btd->bhd", w, val.abs())
            off = (2 * delta + coded_ref.FP16_HALF_STEP) * mass + page * 2.0 ** -39 * val.abs().amax((1, 2))[:, None, None]
            assert ((out[:, heads].double() - want).abs() <= off * (1 + STEP) + STEP * want.abs()).all(), size
            ref, reach = torch.logsumexp(s, 2), reach[..., 0]
            off = 2 * D * 2.0 ** -24 * reach + 2.0 ** -22 * (ref.abs() + 1) + delta[..., 0]
            assert ((lse[heads].T.double() - ref).abs() <= off).all(), size
