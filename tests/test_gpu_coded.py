"""GPU tests of the cache in 8 and 4 bits -- append, gather, decode -- against their 64-bit
plain forms.  Codes and scale bytes are equal, and so is what is read back; bounds on
attention are derived in coded_ref."""
import ctypes
import math

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import coded_ref, paged_ref, parity

pytestmark = pytest.mark.gpu
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


def _draw(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(BF16)


def _bytes(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, device="cuda").to(U8)


def _pages(num_pages, page, hk, D, bits, layout, seed):
    """(k, v, k_scales, v_scales) full of whatever; layout: what lies outermost within a page of codes, of scales."""
    got = []
    for n, heads_first in ((D * bits // 8, layout in ("heads", "codes")), (coded_ref.scale_bytes(bits, D), layout in ("heads", "scales"))):
        for x in range(2):
            t = _bytes((num_pages, hk, page, n) if heads_first else (num_pages, page, hk, n), seed + x)
            got.append(t.transpose(1, 2) if heads_first else t)
        seed += 2
    return got


def _awkward(x):
    """Rows of what is hard to quantise: zeros, the smallest and largest numbers, borders of scales, halves, NaN, infinities."""
    rows, hk, D = x.shape
    g = torch.Generator(device="cuda").manual_seed(rows)
    x *= torch.exp2(torch.randint(-60, 60, (rows, hk, 1), generator=g, device="cuda").float()).to(BF16)
    n = [0]

    def put(row):
        if n[0] < rows:
            x[n[0], n[0] % hk] = row
            n[0] += 1

    grid = torch.arange(D, device="cuda").float()
    put(torch.zeros(D))
    put(-torch.zeros(D))
    put(torch.full((D,), 448.0))
    put(torch.full((D,), 450.0))
    put(grid / 4)                                # halves of both formats
    put((grid - 20) / 2)
    put(torch.where(grid < 1, 12.0, grid % 32 / 4 * 2))   # scale 2: quarters of a code
    put(torch.where(grid % 16 < 1, 6.0 * 1.0625, 0.25 + grid % 16))  # between two scales
    put(torch.where(grid % 16 < 1, 6.0 * 1.1875, 1.25))
    put(torch.full((D,), 2.0 ** -130))
    put(torch.full((D,), 2.0 ** -57))
    put(torch.full((D,), 3.0 * 2.0 ** -18))
    put(torch.full((D,), 3e38))
    put(torch.full((D,), 61440.0))
    put(torch.full((D,), 70000.0))
    for bad in (math.nan, math.inf, -math.inf):
        put(torch.where(grid == 17, bad, 1.0 + grid / 64))


# ------------------------------------------------------------------ append
SHAPES = [(1, 4, 4, 128, 16, "rows"), (37, 12, 3, 64, 24, "heads"), (300, 8, 1, 128, 1, "codes"),
          (129, 16, 8, 64, 128, "scales"), (700, 2, 2, 128, 7, "rows"), (65, 5, 5, 64, 3, "heads")]


def _slots(rows, num_pages, page):
    rng = np.random.default_rng(rows)
    slots = rng.permutation(num_pages * page)[:rows]
    slots[rng.random(rows) < 0.2] = -1
    if rows > 5:
        slots[1], slots[2] = -2**31, -5
    else:
        slots[0] = num_pages * page - 1
    return slots


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,hq,hk,D,page,layout", SHAPES)
def test_append_codes(bits, rows, hq, hk, D, page, layout):
    num_pages = -(-2 * rows // page) + 2
    pager = jfa.Pager(max_seqs=4, max_pages=4, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D, bits=bits)
    held = _pages(num_pages, page, hk, D, bits, layout, 1)
    want = [t.clone() for t in held]
    x = _draw((rows, 1 + 2 * hk, D), 3)
    k, v = x[:, 1:1 + hk], x[:, 1 + hk:]
    _awkward(k)
    slots = _slots(rows, num_pages, page)
    assert jfa.paged_append(pager, k, v, _ints(slots), *held[:2], k_scales=held[2], v_scales=held[3]) is None
    assert pager.status() == 0
    live = np.flatnonzero(slots >= 0)
    at = torch.as_tensor(slots[live] // page).cuda(), torch.as_tensor(slots[live] % page).cuda()
    for i, new in enumerate((k, v)):
        codes, scales = (torch.from_numpy(t).cuda() for t in coded_ref.quantise(new[live], bits))
        n = scales if bits == 8 else scales.repeat_interleave(8, -1)  # codes of what reads as NaN do not matter
        got = held[i][at]
        assert torch.equal(held[2 + i][at], scales)
        assert torch.equal(torch.where(n == 255, codes, got), codes)
        want[i][at], want[2 + i][at] = got, scales
    for a, b in zip(held, want):
        assert torch.equal(a, b)  # all other rows as they were


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,hq,hk,D,page,layout", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("short", [0, 8, 24])
def test_append_rotated_is_what_16_bits_would_hold(bits, rows, hq, hk, D, page, layout, interleaved, short):
    num_pages = -(-2 * rows // page) + 2
    args = dict(max_seqs=4, max_pages=4, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D)
    pager, plain = jfa.Pager(**args, bits=bits), jfa.Pager(**args)
    held = _pages(num_pages, page, hk, D, bits, layout, 1)
    kp, vp, _, _ = plain.pages()
    x = _draw((rows, hq + 2 * hk, D), 3)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    half = D // 2 - short
    freq, axis = jfa.rotary_pairs(2 * half, (half - 3, 3))
    rot = jfa.Rotary(freq, axis, D=D, interleaved=interleaved)
    pos = torch.randint(0, 10**6, (rows, 2), device="cuda", dtype=I32)
    slots = _slots(rows, num_pages, page)
    more = dict(rotary=rot, positions=pos, q=q)
    want_q = jfa.paged_append(plain, k, v, _ints(slots), kp, vp, **more)
    gq = parity.guarded((rows, hq, D), BF16)
    got_q = jfa.paged_append(pager, k, v, _ints(slots), *held[:2], k_scales=held[2], v_scales=held[3], q_out=gq.t, **more)
    assert pager.status() == 0 and got_q is gq.t and torch.equal(got_q, want_q)
    gq.check("q")
    live = np.flatnonzero(slots >= 0)
    at = torch.as_tensor(slots[live] // page).cuda(), torch.as_tensor(slots[live] % page).cuda()
    for i, pages in enumerate((kp, vp)):
        codes, scales = coded_ref.quantise(pages[at], bits)
        assert np.array_equal(held[2 + i][at].cpu().numpy(), scales)
        assert np.array_equal(held[i][at].cpu().numpy(), codes)


@pytest.mark.parametrize("bits", [8, 4])
def test_append_leaves_out_slots_outside_the_cache(bits):
    pager = jfa.Pager(max_seqs=1, max_pages=1, num_pages=3, page_size=5, H=2, Hkv=2, D=64, bits=bits)
    held = _pages(3, 5, 2, 64, bits, "rows", 1)
    was = [t.clone() for t in held]
    k, v = _draw((4, 2, 64), 3), _draw((4, 2, 64), 4)
    jfa.paged_append(pager, k, v, _ints([15, 14, 2**31 - 1, -1]), *held[:2], k_scales=held[2], v_scales=held[3])
    for i, new in enumerate((k, v)):
        codes, scales = (torch.from_numpy(t).cuda() for t in coded_ref.quantise(new[1], bits))
        was[i][2, 4], was[2 + i][2, 4] = codes, scales
    assert all(torch.equal(a, b) for a, b in zip(held, was))
    assert pager.status() == jfa.PAGER_BAD_PAGE and pager.status() == 0


# ------------------------------------------------------------------ a cache full of rows
def _case(lens, hq, hk, D, page, layout, bits, seed, spread=1.0, width=None):
    """(pager, pages and scales, table, lens): quantised rows on pages dealt out at random, random bytes everywhere else."""
    lens = np.asarray(lens)
    count = -(-lens // page)
    width = max(1, int(count.max())) if width is None else width
    rng = np.random.default_rng(seed)
    num_pages = int(count.sum()) + 3
    order, at = rng.permutation(num_pages), 0
    table = rng.integers(-2**31, 2**31, (len(lens), width))  # nothing behind the length is looked at
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    pager = jfa.Pager(max_seqs=len(lens), max_pages=width, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D, bits=bits)
    if bits == 16:
        held = [_draw((num_pages, page, hk, D), seed), _draw((num_pages, page, hk, D), seed + 1), None, None]
        return pager, held, _ints(table), _ints(lens)
    held = _pages(num_pages, page, hk, D, bits, layout, seed)
    slots = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(lens)] + [[]])
    if len(slots):
        s = torch.as_tensor(slots.astype(np.int64)).cuda()
        for i, size in ((0, spread), (1, 0.5)):
            new = (_draw((len(slots), hk, D), seed + 5 + i).float() * size * torch.exp(_draw((len(slots), hk, 1), seed + 9).float())).to(BF16)
            codes, scales = coded_ref.quantise(new, bits)
            held[i][s // page, s % page], held[2 + i][s // page, s % page] = (torch.from_numpy(t).cuda() for t in (codes, scales))
    return pager, held, _ints(table), _ints(lens)


def _scales(held):
    return {} if held[2] is None else dict(k_scales=held[2], v_scales=held[3])


def _values(held, bits):
    if bits == 16:
        return [t.cpu().double() for t in held[:2]]
    return [coded_ref.values(held[i], held[2 + i], bits) for i in range(2)]


# ------------------------------------------------------------------ gather
def _check_gather(pager, held, table, offsets, starts=None, rows=None, status=0, strided=False):
    offsets = np.asarray(offsets)
    rows = int(offsets[-1]) if rows is None else rows
    hk, D, page = pager.Hkv, pager.D, pager.page_size
    outs = []
    for _ in range(2):
        wide = torch.full((rows + 2, hk + (2 if strided else 0), D), 7.0, dtype=BF16, device="cuda")
        outs.append((wide, wide[1:1 + rows, :hk]))
    got = jfa.paged_gather(pager, *held[:2], table, _ints(offsets), rows=rows, starts=None if starts is None else _ints(starts),
                           **_scales(held), k_out=outs[0][1], v_out=outs[1][1])
    assert pager.status() == status and got[0] is outs[0][1]
    tab = table.cpu().numpy().astype(np.int64)
    for i, full in enumerate(_values(held, pager.bits)):
        want = torch.full(outs[i][0].shape, 7.0, dtype=torch.float64)
        for b in range(len(offsets) - 1):
            for r in range(offsets[b], min(offsets[b + 1], rows)):
                t = (0 if starts is None else int(starts[b])) + r - offsets[b]
                want[1 + r, :hk] = 0
                if 0 <= t < tab.shape[1] * page and 0 <= tab[b, t // page] < full.shape[0]:
                    want[1 + r, :hk] = full[tab[b, t // page], t % page]
        assert torch.equal(torch.nan_to_num(outs[i][0].cpu().double(), nan=-77.0), torch.nan_to_num(want, nan=-77.0))


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("lens,hk,D,page,layout", [
    ([300], 4, 128, 16, "rows"), ([1], 1, 64, 1, "heads"), ([0, 5, 0, 0, 17, 33, 0], 3, 64, 24, "heads"),
    ([40, 0, 129, 1, 16, 15, 17], 8, 128, 8, "codes"), (list(range(70)), 2, 64, 32, "scales"), ([700, 2], 5, 128, 100, "rows")])
def test_gather(bits, lens, hk, D, page, layout):
    pager, held, table, dl = _case(lens, hk, hk, D, page, layout, bits, 3)
    offsets = np.concatenate([[0], np.cumsum(lens)])
    _check_gather(pager, held, table, offsets)
    _check_gather(pager, held, table, offsets, rows=int(offsets[-1]) + 37, strided=True)
    # the last rows of each request alone
    tail = np.minimum(lens, 5)
    _check_gather(pager, held, table, np.concatenate([[0], np.cumsum(tail)]), starts=np.asarray(lens) - tail)
    # packed rows that begin later
    _check_gather(pager, held, table, offsets + 3)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("k_off,v_off,gap", [(8, 0, 0), (0, 24, 0), (16, 16, 8), (0, 0, 24), (16, 32, 16)])
def test_gather_to_any_16_bytes(bits, k_off, v_off, gap):
    """Outputs that begin at, and have rows, multiples of 16 bytes apart, not of 32."""
    pager, held, table, dl = _case([70, 0, 33], 2, 2, 64, 16, "rows", bits, 3)
    row, n = 2 * 64 + gap, 103
    bufs = [torch.full((n * row + 64,), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    outs = [x[off:].as_strided((n, 2, 64), (row, 64, 1)) for x, off in zip(bufs, (k_off, v_off))]
    assert outs[0].data_ptr() % 32 == 2 * k_off % 32
    want = jfa.paged_gather(pager, *held[:2], table, _ints([0, 70, 70, 103]), rows=n, **_scales(held))
    jfa.paged_gather(pager, *held[:2], table, _ints([0, 70, 70, 103]), rows=n, **_scales(held), k_out=outs[0], v_out=outs[1])
    for x, off, out, w in zip(bufs, (k_off, v_off), outs, want):
        assert torch.equal(out, w)
        out.fill_(7.0)
        assert (x == 7.0).all()  # nothing beside


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_gather_outputs_that_overlap(bits):
    """Slices of one tensor are fine; the same rows, shifted ones and half of them are refused."""
    pager, held, table, dl = _case([40, 7], 2, 2, 64, 16, "rows", bits, 3)
    call = lambda k, v: jfa.paged_gather(pager, *held[:2], table, _ints([0, 40, 47]), rows=47, **_scales(held), k_out=k, v_out=v)  # noqa: E731
    want = jfa.paged_gather(pager, *held[:2], table, _ints([0, 40, 47]), rows=47, **_scales(held))
    one = torch.zeros((100, 5, 64), dtype=BF16, device="cuda")
    for k, v in ((one[:47, :2], one[:47, 2:4]), (one[:47, 3:], one[:47, 1:3]), (one[:47, 3:], one[20:67, :2]), (one[:47, :2], one[47:94, :2])):
        got = call(k, v)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for k, v in ((one[:47, :2], one[:47, :2]), (one[:47, :2], one[:47, 1:3]), (one[:47, :2], one[20:67, :2]), (one[:47, 3:], one[20:67, 2:4]),
                 (one[:47, :2], one[:94:2, 3:])):
        with pytest.raises(jfa.JfaError) as e:
            call(k, v)
        assert e.value.code == 1


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_gather_of_any_bytes(bits):
    """What is not written by append reads as it says: NaN, other bytes as the nearest power, all codes."""
    hk, D, page, n = 2, 64, 16, 300
    pager, held, table, dl = _case([n], hk, hk, D, page, "rows", bits, 3)
    if bits < 16:
        held = _pages(pager.num_pages, page, hk, D, bits, "rows", 11)
        for t in held[2:]:
            t.copy_(torch.arange(t.numel(), device="cuda").view(t.shape).to(U8))
        if bits == 4:  # a scale beyond 10240 makes values beyond fp16
            for t in held[2:]:
                t[(t > 226) & (t < 249)] = 226
    _check_gather(pager, held, table, [0, n])


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_gather_bad_places(bits):
    """Rows outside the table and on pages outside the cache are zeros, and say so."""
    pager, held, table, dl = _case([40, 100, 64, 33, 16], 2, 2, 64, 16, "rows", bits, 5)
    off = [0, 40, 140, 204, 237, 253]
    _check_gather(pager, held, table, off, starts=[-1, 0, 100, 2**31 - 1, -2**31], status=jfa.PAGER_BAD_LENGTH | jfa.PAGER_BAD_PAGE)
    num = pager.num_pages
    table[1, 2], table[2, 0], table[3, 0], table[3, 1], table[3, 2], table[4, 0] = num, -1, num, 2**31 - 1, -2**31, num
    _check_gather(pager, held, table, off, status=jfa.PAGER_BAD_PAGE)
    _check_gather(pager, held, table, off, rows=30, status=jfa.PAGER_BAD_LENGTH)


@pytest.mark.parametrize("bits", [8, 4])
def test_gather_the_most_requests(bits):
    """16384 requests, most of them empty."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, 16384) * (rng.random(16384) < 0.3)
    lens[16000:] = 0
    pager, held, table, dl = _case(lens, 1, 1, 64, 2, "rows", bits, 6)
    _check_gather(pager, held, table, np.concatenate([[0], np.cumsum(lens)]))


# ------------------------------------------------------------------ decode
def _check_decode(pager, held, table, lens, scale=None, status=0, seed=7, q=None):
    B, H, D = len(lens), pager.H, pager.D
    scale = 1 / math.sqrt(D) if scale is None else scale
    q = _draw((B, H, D), seed) if q is None else q
    go, gl = parity.guarded((B, H, D), BF16), parity.guarded((H, B), F32)
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, lens, scale, **_scales(held), out=go.t, lse=gl.t)
    assert pager.status() == status
    go.check("out")
    gl.check("lse")
    again = jfa.paged_decode(pager, q, *held[:2], table, lens, scale, **_scales(held))
    pager.status()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)  # bit for bit
    ref, ref_lse, off, off_lse = coded_ref.decode(q, *_values(held, pager.bits), table, lens, scale)
    o, l = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(o).all()
    err = (o - ref).abs()
    assert (err <= off).all(), float((err / off.clamp(min=1e-300)).max())
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(l), empty) and (l[empty] < 0).all()
    assert ((l - ref_lse).abs()[~empty] <= off_lse[~empty]).all(), float((l - ref_lse).abs()[~empty].max())
    return q, out, lse


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 511, 1000]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 4), (6, 2), (15, 3), (8, 1), (9, 1), (16, 1), (17, 1), (48, 1),
                                   (66, 2), (130, 1), (300, 1)])
def test_decode_head_groups(bits, D, hq, hk):
    _check_decode(*_case(EDGES, hq, hk, D, 16, "rows", bits, hq * 100 + hk))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 32, 100, 128, 1024])
@pytest.mark.parametrize("layout", ["rows", "heads", "codes", "scales"])
def test_decode_pages(bits, D, page, layout):
    _check_decode(*_case(EDGES, 4, 2, D, page, layout, bits, page))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [1] * 700, [5000], [3, 20000], [20000, 0, 1], [129] * 152,
                                  list(range(300)), [0] * 300 + [4000]], ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_decode_splits(bits, lens, hq, hk):
    """Few long rows, many short ones, and both: every way a row is cut and joined."""
    _check_decode(*_case(lens, hq, hk, 128, 16, "rows", bits, len(lens)))


@pytest.mark.parametrize("bits", [8, 4])
def test_decode_peaked_scores_and_scales(bits):
    case = _case([40, 700, 3], 4, 2, 128, 16, "rows", bits, 3, spread=30.0, width=500)
    for scale in (None, 0.0, -0.3):
        _check_decode(*case, scale=scale)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hk", [(4, 2), (24, 1)])
def test_decode_rows_of_very_different_sizes(bits, hq, hk):
    """Values and keys from the smallest to the largest scales; queries of heads far apart, the largest and smallest."""
    lens, page, D = [300, 64, 5, 2000], 16, 64
    pager, held, table, dl = _case(lens, hq, hk, D, page, "rows", bits, 8)
    rng = np.random.default_rng(4)
    for b, n in enumerate(lens):
        for t in range(n):
            at = int(table[b, t // page]), t % page
            if bits == 8:
                held[2][at] = int(rng.integers(79, 120))
                held[3][at] = int(rng.integers(79, 176))
            else:
                held[2][at] = torch.from_numpy(rng.integers(0, 120, (hk, D // 16)).astype(np.uint8)).cuda()
                held[3][at] = torch.from_numpy(rng.integers(0, 227, (hk, D // 16)).astype(np.uint8)).cuda()
    _check_decode(pager, held, table, dl)
    q = _draw((len(lens), hq, D), 3)
    q *= torch.exp2(torch.arange(hq, device="cuda").float() - 12)[None, :, None].to(BF16)
    _check_decode(pager, held, table, dl, q=q)
    _check_decode(pager, held, table, dl, q=torch.zeros_like(q))
    for c in (0, 79, 175):  # all values as small or large as they get
        held[3].fill_(c if bits == 8 else min(c, 226))
        _check_decode(pager, held, table, dl, q=q)


@pytest.mark.parametrize("bits", [8, 4])
def test_decode_huge_and_tiny_queries(bits):
    """q as large and as small as bf16 has it, where the scores stay in fp32."""
    pager, held, table, dl = _case([300, 40], 4, 2, 64, 16, "rows", bits, 9)
    for size in (2.0 ** 100, 2.0 ** -120, 2.0 ** -130):
        q = (_draw((2, 4, 64), 2).float() * size).to(BF16)
        _check_decode(pager, held, table, dl, scale=0.1 / size if size < 1e38 and size > 1e-37 else 1.0, q=q)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_decode_queries_that_are_not_finite(bits, bad):
    """One head's infinities and NaN leave the heads beside it, of the same keys, as they are."""
    pager, held, table, dl = _case([300, 40, 1], 12, 2, 64, 16, "rows", bits, 9)
    q = _draw((3, 12, 64), 2)
    want = jfa.paged_decode(pager, q, *held[:2], table, dl, 0.1, **_scales(held))
    q[0, 3, 5], q[1, 7, 63], q[2, 0] = bad, bad, bad
    hit = torch.zeros((3, 12), dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 7] = hit[2, 0] = True
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, dl, 0.1, **_scales(held))
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse.T[~hit], want[1].T[~hit])
    assert not torch.isfinite(lse.T[hit]).any()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens", [[1], [2, 0, 31], [300, 17], [9000, 40, 1]], ids=str)
@pytest.mark.parametrize("hq,hk,D", [(1, 1, 64), (4, 2, 128), (24, 1, 64)])
def test_decode_nan_rows(bits, lens, hq, hk, D):
    """A NaN value of V in a counted row makes its places of out NaN, one of K the head's out and lse; no others."""
    pager, held, table, dl = _case(lens, hq, hk, D, 16, "rows", bits, 3)
    q, was, was_lse = _check_decode(pager, held, table, dl)
    b = int(np.argmax(lens))
    t = lens[b] - 1
    at = int(table[b, t // 16]), t % 16, hk - 1
    keep = held[3][at].clone()
    held[3][at][-1] = 255
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, dl, D ** -0.5, **_scales(held))
    bad = torch.zeros((len(lens), hq, D), dtype=torch.bool, device="cuda")
    bad[b, (hk - 1) * (hq // hk):, 0 if bits == 8 else D - 16:] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], was[~bad])
    near = 2 * coded_ref.decode(q, *_values(held, bits), table, dl, D ** -0.5)[3].cuda()  # of two values in their bounds
    assert (torch.nan_to_num(lse - was_lse, nan=0.0).abs() <= near).all() and torch.equal(torch.isinf(lse), torch.isinf(was_lse))
    held[3][at] = keep
    held[2][at][0] = 255
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, dl, D ** -0.5, **_scales(held))
    bad[b, (hk - 1) * (hq // hk):] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(torch.isnan(lse), bad[:, :, 0].T)
    assert torch.equal(out[~bad], was[~bad])


@pytest.mark.parametrize("bits", [8, 4])
def test_strided_tables_and_queries(bits):
    """Rows of tables and queries that lie apart; fewer requests than the pager holds."""
    pager, held, table, dl = _case([300, 17, 0, 900], 8, 2, 128, 16, "rows", bits, 6)
    q = _draw((4, 8, 128), 2)
    want = jfa.paged_decode(pager, q, *held[:2], table, dl, 0.1, **_scales(held))
    off = _ints([0, 300, 317, 317, 1217])
    rows = jfa.paged_gather(pager, *held[:2], table, off, rows=1217, **_scales(held))
    wide = torch.full((4, pager.max_pages + 5), -9, dtype=I32, device="cuda")
    wide[:, :pager.max_pages] = table
    more = torch.zeros((4, 13, 128), dtype=BF16, device="cuda")
    more[:, 2:10] = q
    big = jfa.Pager(max_seqs=50, max_pages=pager.max_pages, num_pages=pager.num_pages, page_size=16, H=8, Hkv=2, D=128, bits=bits)
    got = jfa.paged_decode(big, more[:, 2:10], *held[:2], wide[:, :pager.max_pages], dl, 0.1, **_scales(held))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = jfa.paged_gather(big, *held[:2], wide[:, :pager.max_pages], off, rows=1217, **_scales(held))
    assert torch.equal(got[0], rows[0]) and torch.equal(got[1], rows[1]) and big.status() == 0
    for n in (1, 2, 3):
        got = jfa.paged_decode(big, q[:n], *held[:2], table[:n], dl[:n], 0.1, **_scales(held))
        ref, ref_lse, bound, _ = coded_ref.decode(q[:n], *_values(held, bits), table[:n], dl[:n], 0.1)
        assert ((got[0].cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_every_page_and_length_at_its_limit(bits):
    """A table as full as it can be, the last page of the cache, and offsets up to all of it."""
    page, width, B, hk, D = 16, 5, 7, 2, 64
    pager, held, table, dl = _case([page * width] * B, 4, hk, D, page, "rows", bits, 6, width=width)
    full = pager.num_pages - 3
    assert int(table.max()) < pager.num_pages and full == B * width
    _check_decode(pager, held, table, dl)
    _check_gather(pager, held, table, np.arange(B + 1) * page * width)
    tight = jfa.Pager(max_seqs=B, max_pages=width, num_pages=int(table.max()) + 1, page_size=page, H=4, Hkv=hk, D=D, bits=bits)
    some = [t[:tight.num_pages] for t in held]
    _check_decode(tight, some, table, dl)
    _check_gather(tight, some, table, np.arange(B + 1) * page * width)
    dl += 1
    _check_decode(tight, some, table, dl, status=jfa.PAGER_BAD_LENGTH)


@pytest.mark.parametrize("bits", [8, 4])
def test_decode_bad_lengths_and_pages(bits):
    pager, held, table, lens = _case([40, 100, 64, 33, 16], 4, 2, 64, 16, "heads", bits, 5)
    lens[0], lens[3] = -1, 2**31 - 1
    _check_decode(pager, held, table, lens, status=jfa.PAGER_BAD_LENGTH)
    lens[0], lens[3] = 40, 33
    num = pager.num_pages
    table[1, 2], table[2, 0], table[3, 0], table[3, 1], table[3, 2], table[4, 0] = num, -1, num, 2**31 - 1, -2**31, num
    _check_decode(pager, held, table, lens, status=jfa.PAGER_BAD_PAGE)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("layout", ["rows", "heads"])
def test_past_32_bit_offsets(bits, layout):
    """The last pages of a cache of more than 2^31 bytes per tensor, also of scales."""
    hk, D, page = 8, 128, 64
    num_pages = (1 << 15) * (1 if bits == 8 else 2) + 40
    pager = jfa.Pager(max_seqs=2, max_pages=12, num_pages=num_pages, page_size=page, H=16, Hkv=hk, D=D, bits=bits)
    held = []
    for n in (D * bits // 8, coded_ref.scale_bytes(bits, D)):
        for _ in range(2):
            if n < 16:  # pages of scales far apart
                t = torch.zeros((num_pages, 1 << 17), dtype=U8, device="cuda")[:, :page * hk * n].view(num_pages, page, hk, n)
            else:
                t = torch.zeros((num_pages, hk, page, n) if layout == "heads" else (num_pages, page, hk, n), dtype=U8, device="cuda")
                t = t.transpose(1, 2) if layout == "heads" else t
            held.append(t)
    assert held[0].stride(0) * (num_pages - 13) > 2**31 and held[2].stride(0) * (num_pages - 13) > 2**31
    n = 700
    table = _ints(np.stack([num_pages - 1 - np.arange(12), np.arange(12)]))
    t = torch.arange(n, device="cuda")
    at = table[0, t // page].long(), t % page
    k, v = _draw((n, hk, D), 1), _draw((n, hk, D), 2)
    jfa.paged_append(pager, k, v, (at[0] * page + at[1]).to(I32), *held[:2], **_scales(held))
    codes, scales = (torch.from_numpy(x).cuda() for x in coded_ref.quantise(k, bits))
    assert torch.equal(held[0][at], codes) and torch.equal(held[2][at], scales)
    assert not held[0][:num_pages - 12].any() and not held[2][:num_pages - 12].any()
    got = jfa.paged_gather(pager, *held[:2], table, _ints([0, n, n]), rows=n, **_scales(held))
    assert torch.equal(got[0].cpu().double(), coded_ref.values(codes, scales, bits))
    # decode against the rows read back, from a cache of 16 bits
    plain = jfa.Pager(max_seqs=2, max_pages=11, num_pages=12, page_size=page, H=16, Hkv=hk, D=D)
    kp, vp, _, _ = plain.pages()
    jfa.paged_append(plain, *got, t.to(I32), kp, vp)
    lens, q = _ints([n, 0]), _draw((2, 16, D), 3)
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, lens, 0.09, **_scales(held))
    ref, ref_lse, off, off_lse = coded_ref.decode(q, kp.cpu().double(), vp.cpu().double(), _ints(np.stack([np.arange(11)] * 2)), lens, 0.09)
    assert ((out.cpu().double() - ref).abs() <= off).all() and ((lse.cpu().double() - ref_lse).abs()[:, 0] <= off_lse[:, 0]).all()


def _check_on_the_gpu(pager, held, table, lens, q, scale):
    """decode against 64 bits over the rows that gather reads back, a request at a time, within coded_ref's bounds."""
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, lens, scale, **_scales(held))
    again = jfa.paged_decode(pager, q, *held[:2], table, lens, scale, **_scales(held))
    assert pager.status() == 0 and torch.equal(out, again[0]) and torch.equal(lse, again[1])
    group, D, step = pager.H // pager.Hkv, pager.D, torch.finfo(BF16).eps / 2
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            assert not out[b].any() and (lse[:, b] == -math.inf).all()
            continue
        k, v = jfa.paged_gather(pager, *held[:2], table[b:b + 1], _ints([0, n]), rows=n, **_scales(held))
        for g in range(pager.Hkv):
            heads = slice(g * group, (g + 1) * group)
            kd, vd, qd = k[:, g].double(), v[:, g].double(), q[b, heads].double()
            s = scale * qd @ kd.T
            w, ref = torch.softmax(s, 1), torch.logsumexp(s, 1)
            size = (abs(scale) * qd.abs() @ kd.abs().T).amax(1)
            delta = 2 * D * 2.0 ** -24 * size + 2.0 ** -17 + 2 * n * 2.0 ** -24
            want = w @ vd
            off = (2 * delta + coded_ref.FP16_HALF_STEP)[:, None] * (w @ vd.abs()) + n * 2.0 ** -39 * vd.abs().amax()
            assert ((out[b, heads].double() - want).abs() <= off * (1 + step) + step * want.abs()).all()
            assert ((lse[heads, b].double() - ref).abs() <= delta + 2.0 ** -23 * ref.abs()).all()


@pytest.mark.parametrize("bits,D,hk,group,mb", [
    (4, 128, 8, 2, 100), (4, 128, 2, 12, 100), (4, 128, 4, 8, 530), (4, 64, 4, 3, 100), (4, 64, 8, 16, 540),
    (8, 64, 2, 4, 100), (8, 64, 4, 9, 100), (8, 128, 2, 8, 270), (8, 128, 4, 11, 270), (4, 128, 3, 4, 120),
    (8, 128, 1, 8, 270)])
@pytest.mark.parametrize("few", [True, False])
def test_decode_heads_side_by_side(bits, D, hk, group, mb, few):
    """As much to read as makes neighbouring heads go side by side, and stay in L2; few long requests and many."""
    page, row = 16, D * bits // 8
    rows = (mb << 20) // (2 * hk * row)
    rng = np.random.default_rng(rows)
    B = 5 if few else 70
    lens = rng.dirichlet(np.full(B, 0.7)) * rows
    lens = np.maximum(lens.astype(np.int64), 0)
    lens[0], lens[-1] = 0, rows - lens[1:-1].sum()
    count = -(-lens // page)
    width, num_pages = int(count.max()), int(count.sum())
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=hk * group, Hkv=hk, D=D, bits=bits)
    held = pager.pages()
    table, order, at = np.full((B, width), -1), rng.permutation(num_pages), 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    slots = torch.arange(num_pages * page, device="cuda", dtype=I32)
    for i in range(0, len(slots), 1 << 17):
        part = slots[i:i + (1 << 17)]
        jfa.paged_append(pager, _draw((len(part), hk, D), i), _draw((len(part), hk, D), i + 1), part, *held[:2], **_scales(held))
    _check_on_the_gpu(pager, held, _ints(table), _ints(lens), _draw((B, hk * group, D), 5), D ** -0.5)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hk,D", [(16, 8, 64), (32, 2, 64), (40, 2, 64), (10, 2, 128), (32, 2, 128), (70, 2, 128)])
def test_decode_tables_wide_enough_for_64_bit_counts(bits, hq, hk, D):
    """A table of which full rows would hold more tiles than 32 bits count."""
    pager, held, table, lens = _case([300, 5000, 0, 17], hq, hk, D, 1024, "rows", bits, 12)
    q = _draw((4, hq, D), 1)
    pages = (1 << 21) - 2
    wide = torch.full((130, pages), -1, dtype=I32, device="cuda")  # 1.1 GB; only the rows of 130 requests count
    wide[:4, :table.shape[1]] = table
    big = jfa.Pager(max_seqs=130, max_pages=pages, num_pages=pager.num_pages, page_size=1024, H=hq, Hkv=hk, D=D, bits=bits)
    assert 130 * (pages * 1024 // 64) > 2**32 // hk
    many, some = torch.zeros((130, hq, D), dtype=BF16, device="cuda"), torch.zeros(130, dtype=I32, device="cuda")
    many[:4], some[:4] = q, lens
    out, lse = jfa.paged_decode(big, many, *held[:2], wide, some, 0.1, **_scales(held))
    assert big.status() == 0 and not out[4:].any() and (lse[:, 4:] == -math.inf).all()
    ref, ref_lse, off, off_lse = coded_ref.decode(q, *_values(held, bits), table, lens, 0.1)
    assert ((out[:4].cpu().double() - ref).abs() <= off).all()
    fine = ~torch.isinf(ref_lse)
    assert ((lse[:, :4].cpu().double() - ref_lse).abs()[fine] <= off_lse[fine]).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2)])
def test_decode_the_most_requests(bits, hq, hk):
    """16384 requests of 0 to 40 rows, a page of 40 each, in the bounds of coded_ref, all at once."""
    B, page, D = 16384, 40, 64
    rng = np.random.default_rng(1)
    lens, order = rng.integers(0, page + 1, B), rng.permutation(B)
    pager = jfa.Pager(max_seqs=B, max_pages=1, num_pages=B, page_size=page, H=hq, Hkv=hk, D=D, bits=bits)
    held = pager.pages()
    slots = torch.arange(B * page, device="cuda", dtype=I32)
    jfa.paged_append(pager, _draw((B * page, hk, D), 1), _draw((B * page, hk, D), 2), slots, *held[:2], **_scales(held))
    q, table, dl = _draw((B, hq, D), 3), _ints(order[:, None]), _ints(lens)
    out, lse = jfa.paged_decode(pager, q, *held[:2], table, dl, 0.125, **_scales(held))
    k, v = jfa.paged_gather(pager, *held[:2], table, _ints(np.arange(B + 1) * page), rows=B * page, **_scales(held))
    assert pager.status() == 0
    k, v = (x.view(B, page, hk, D).double().repeat_interleave(hq // hk, 2) for x in (k, v))
    s = 0.125 * torch.einsum("bhd,bthd->bht", q.double(), k)
    size = 0.125 * torch.einsum("bhd,bthd->bht", q.double().abs(), k.abs()).amax(-1)
    dead = torch.arange(page, device="cuda")[None, None] >= dl[:, None, None]
    w = torch.softmax(s.masked_fill(dead, -math.inf), -1).nan_to_num(0.0)
    want, mass = torch.einsum("bht,bthd->bhd", w, v), torch.einsum("bht,bthd->bhd", w, v.abs())
    delta = (2 * D * 2.0 ** -24 * size + 2.0 ** -17 + 2 * page * 2.0 ** -24)[..., None]
    step = torch.finfo(BF16).eps / 2
    off = (2 * delta + coded_ref.FP16_HALF_STEP) * mass + page * 2.0 ** -39 * v.abs().amax((1, 3))[..., None]
    assert ((out.double() - want).abs() <= off * (1 + step) + step * want.abs()).all()
    ref = torch.logsumexp(s.masked_fill(dead, -math.inf), -1)
    some = (dl > 0)[:, None].expand_as(ref)
    assert ((lse.T.double() - ref).abs()[some] <= (delta[..., 0] + 2.0 ** -23 * ref.abs())[some]).all()
    assert (lse.T[~some] == -math.inf).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_two_pagers_on_two_streams(bits):
    pager, held, table, lens = _case([2000, 300, 64, 5], 8, 2, 128, 16, "rows", bits, 9)
    other = jfa.Pager(max_seqs=4, max_pages=pager.max_pages, num_pages=pager.num_pages, page_size=16, H=8, Hkv=2, D=128, bits=bits)
    q = _draw((4, 8, 128), 1)
    want, _ = jfa.paged_decode(pager, q, *held[:2], table, lens, 0.1, **_scales(held))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(30):
        for s, p, o in zip(streams, (pager, other), outs):
            with torch.cuda.stream(s):
                o.append(jfa.paged_decode(p, q, *held[:2], table, lens, 0.1, **_scales(held))[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for o in outs for x in o)


@pytest.mark.parametrize("bits", [8, 4])
def test_decode_captured_with_changing_lengths(bits):
    pager, held, table, lens = _case([2000, 300, 64, 5], 8, 2, 128, 16, "rows", bits, 9)
    q = _draw((4, 8, 128), 1)
    out, lse = torch.empty_like(q), torch.empty((8, 4), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jfa.paged_decode(pager, q, *held[:2], table, lens, 0.1, **_scales(held), out=out, lse=lse)
    for new in ([2000, 300, 64, 5], [1, 0, 60, 4], [1999, 299, 1, 0], [0, 0, 0, 0]):
        lens.copy_(_ints(new))
        graph.replay()
        a, b = jfa.paged_decode(pager, q, *held[:2], table, lens, 0.1, **_scales(held))
        assert torch.equal(a, out) and torch.equal(b, lse)
        _check_decode(pager, held, table, lens)


# ------------------------------------------------------------------ refusals
def test_refusals_of_the_binding():
    with pytest.raises(ValueError):
        jfa.Pager(max_seqs=1, max_pages=1, num_pages=1, page_size=1, H=1, Hkv=1, D=64, bits=2)
    for bits in (16, 8, 4):
        pager, held, table, lens = _case([40, 20], 4, 2, 64, 16, "rows", bits, 5)
        q, k = _draw((2, 4, 64), 1), _draw((2, 2, 64), 1)
        slots = _ints([0, 1])
        calls = [lambda kp, vp, **kw: jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1, **kw),
                 lambda kp, vp, **kw: jfa.paged_append(pager, k, k, _ints([-1, -1]), kp, vp, **kw),
                 lambda kp, vp, **kw: jfa.paged_gather(pager, kp, vp, table, _ints([0, 40, 60]), rows=60, **kw)]
        for call in calls:
            call(*held[:2], **_scales(held))
            if bits == 16:
                some = torch.zeros((pager.num_pages, 16, 2, 1), dtype=U8, device="cuda")
                with pytest.raises(ValueError):
                    call(*held[:2], k_scales=some, v_scales=some)
                continue
            ks, vs = held[2:]
            for bad in (dict(), dict(k_scales=ks), dict(k_scales=ks, v_scales=vs[1:]), dict(k_scales=ks[..., :0], v_scales=vs),
                        dict(k_scales=ks, v_scales=vs.transpose(1, 2).contiguous().transpose(1, 2))):
                with pytest.raises(ValueError):
                    call(*held[:2], **bad)
            for bad in (dict(k_scales=ks.cpu(), v_scales=vs), dict(k_scales=ks, v_scales=vs.to(torch.int8))):
                with pytest.raises(TypeError):
                    call(*held[:2], **bad)
            with pytest.raises(TypeError):
                call(held[0].to(BF16), held[1], **_scales(held))
            with pytest.raises(ValueError):
                call(held[0][..., :16], held[1][..., :16], **_scales(held))
        gather = lambda **kw: jfa.paged_gather(**{**dict(pager=pager, k_pages=held[0], v_pages=held[1], table=table,  # noqa: E731
                                                         offsets=_ints([0, 40, 60]), rows=60, **_scales(held)), **kw})
        for bad in (dict(table=table[:, :1]), dict(offsets=_ints([0, 4])), dict(starts=_ints([0])),
                    dict(k_out=torch.empty((60, 2, 32), dtype=BF16, device="cuda"))):
            with pytest.raises(ValueError):
                gather(**bad)
        for bad in (dict(table=table.long()), dict(offsets=torch.tensor([0, 1, 2]).cuda()), dict(starts=torch.zeros(2, dtype=I32)),
                    dict(v_out=torch.empty((60, 2, 64), device="cuda"))):
            with pytest.raises(TypeError):
                gather(**bad)
        with pytest.raises(jfa.JfaError):  # more requests than the pager holds
            gather(offsets=_ints([0, 1, 2, 3]), table=table[[0, 1, 0]])
        with pytest.raises(jfa.JfaError):
            gather(offsets=_ints([0]), table=table[:0])
        got = gather(rows=0)
        assert got[0].shape == (0, 2, 64)


def test_host_refusals_with_a_pager():
    """Argument checks of the C entries that need a handle; nothing launches."""
    L = jfa.lib()
    for bits in (8, 4):
        pager, held, table, lens = _case([40, 20], 4, 2, 64, 16, "rows", bits, 5)
        h, st, ss = pager.handle, held[0].stride(), held[2].stride()

        def pages(**kw):
            return ctypes.byref(jfa._Pages(**{**dict(k=held[0].data_ptr(), v=held[1].data_ptr(), page=st[0], row=st[1], head=st[2]), **kw}))

        def scales(**kw):
            return ctypes.byref(jfa._Scales(**{**dict(k=held[2].data_ptr(), v=held[3].data_ptr(), page=ss[0], row=ss[1], head=ss[2]), **kw}))

        q, out, lse = _draw((2, 4, 64), 1), torch.empty((2, 4, 64), dtype=BF16, device="cuda"), torch.empty((4, 2), device="cuda")
        bad_cache = [(pages(row=st[1] + 8), scales(), 4), (pages(page=st[0] + 8), scales(), 4), (pages(), None, 1),
                     (pages(), scales(k=None), 1), (pages(), scales(head=-1), 1), (pages(), scales(row=-4), 1)]
        if bits == 4:
            bad_cache += [(pages(), scales(k=held[2].data_ptr() + 2), 4), (pages(), scales(page=ss[0] + 2), 4)]
        k = _draw((2, 2, 64), 1)
        s, off = _ints([0, 1]), _ints([0, 1, 2])
        o = torch.empty((2, 2, 64), dtype=BF16, device="cuda")
        decode = lambda p, c: L.jfa_paged_decode_ex(h, 2, q.data_ptr(), 256, p, c, table.data_ptr(), table.stride(0),  # noqa: E731
                                                    lens.data_ptr(), 0.1, out.data_ptr(), lse.data_ptr(), None)
        append = lambda p, c: L.jfa_paged_append_ex(h, 2, k.data_ptr(), 128, k.data_ptr(), 128, s.data_ptr(), p, c, None,  # noqa: E731
                                                    None, 0, 0, None, 0, None, 0, None)
        gather = lambda p, c: L.jfa_paged_gather(h, 2, p, c, table.data_ptr(), table.stride(0), None, off.data_ptr(), 2,  # noqa: E731
                                                 o.data_ptr(), 128, k.data_ptr(), 128, None)
        for p, c, code in bad_cache:
            for call in (decode, append, gather):
                assert call(p, c) == code
        good = [h, 2, pages(), scales(), table.data_ptr(), table.stride(0), None, off.data_ptr(), 2, o.data_ptr(), 128, k.data_ptr(), 128, None]
        for at, value, code in [(1, 0, 1), (1, 3, 1), (4, None, 1), (4, table.data_ptr() + 2, 4), (5, pager.max_pages - 1, 1),
                                (6, off.data_ptr() + 1, 4), (7, None, 1), (7, off.data_ptr() + 2, 4), (8, -1, 1), (8, 2**31, 1),
                                (9, None, 1), (9, o.data_ptr() + 2, 4), (10, 120, 1), (10, 132, 4), (11, None, 1), (12, 64, 1)]:
            args = list(good)
            args[at] = value
            assert L.jfa_paged_gather(*args) == code, (at, value)
        # the calls of 16 bits do not take such a pager
        assert L.jfa_paged_decode(h, 2, q.data_ptr(), 256, pages(), table.data_ptr(), table.stride(0), lens.data_ptr(), 0.1,
                                  out.data_ptr(), lse.data_ptr(), None) == 1
        assert L.jfa_paged_append(h, 2, k.data_ptr(), 128, k.data_ptr(), 128, s.data_ptr(), pages(), None, None, 0, 0, None, 0,
                                  None, 0, None) == 1
    torch.cuda.synchronize()


# ------------------------------------------------- a serving run of them all
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(bits, captured):
    """Requests enter with a prompt, decode a token a step, drop their last tokens and leave:
    tables, append with rotation, gather of what each request has, the forward of its new
    rows over it, and decode of its last.  The forward and decode are checked against
    attention in 64 bits over the rows read back, and those against the rows that went in."""
    H, hk, D, page, width, num_pages, B, rows = 8, 2, 128, 8, 12, 60, 6, 64
    freq, axis = jfa.rotary_pairs(D, (32, 16, 16))
    rot = jfa.Rotary(freq, axis, D=D)
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=H, Hkv=hk, D=D, bits=bits)
    held = pager.pages()
    lens, delta, n_free = _ints(np.zeros(B)), _ints(np.zeros(B)), _ints([num_pages])
    table, free = _ints(np.full((B, width), -1)), _ints(np.random.default_rng(0).permutation(num_pages))
    slots, positions, offsets = (torch.empty(n, dtype=I32, device="cuda") for n in (rows, rows, B + 1))
    qkv = torch.zeros((rows, H + 2 * hk, D), dtype=BF16, device="cuda")
    turned = torch.empty((rows, H, D), dtype=BF16, device="cuda")
    most = B * width * page
    kv_offsets = torch.zeros(B + 1, dtype=I32, device="cuda")
    k_all, v_all = (torch.zeros((most, hk, D), dtype=BF16, device="cuda") for _ in range(2))
    out, lse = torch.empty((B, H, D), dtype=BF16, device="cuda"), torch.empty((H, B), device="cuda")

    def step():
        jfa.paged_tables(pager, lens, delta, table, free, n_free, rows=rows, lens_out=lens, n_free_out=n_free,
                         slots=slots, positions=positions, row_offsets=offsets)
        jfa.paged_append(pager, qkv[:, H:H + hk], qkv[:, H + hk:], slots, *held[:2], **_scales(held), rotary=rot,
                         positions=positions, q=qkv[:, :H], q_out=turned)
        kv_offsets[1:] = torch.cumsum(lens, 0).to(I32)
        jfa.paged_gather(pager, *held[:2], table, kv_offsets, rows=most, **_scales(held), k_out=k_all, v_out=v_all)
        newest = (offsets[1:] - 1).clamp(min=0).long()
        jfa.paged_decode(pager, turned[newest], *held[:2], table, lens, 0.09, **_scales(held), out=out, lse=lse)

    if captured:
        step()  # warm up, with nothing to do
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    rng = np.random.default_rng(1)
    kept = [[] for _ in range(B)]  # (k, v) of each request's rows, as they went in
    for i in range(12):
        d = np.ones(B, int)
        for b in range(B):
            n = len(kept[b])
            if n == 0:
                d[b] = rng.integers(0, 20)
            elif n > 70 or rng.random() < 0.1:
                d[b] = -n if rng.random() < 0.5 else -rng.integers(0, n + 1)
        while np.maximum(d, 0).sum() > rows:
            d[d.argmax()] = 1
        delta.copy_(_ints(d))
        qkv.copy_(_draw(qkv.shape, 100 + i))
        graph.replay() if captured else step()
        assert pager.status() == 0
        k_new = jfa.rotate(rot, positions, qkv[:, H:H + hk])
        at = 0
        for b in range(B):
            kept[b] = kept[b][:len(kept[b]) + d[b]] if d[b] < 0 else kept[b] + [(k_new[at + j].cpu(), qkv[at + j, H + hk:].cpu()) for j in range(d[b])]
            at += max(d[b], 0)
        ends = kv_offsets.cpu().numpy()
        assert lens.cpu().tolist() == [len(x) for x in kept] == np.diff(ends).tolist()
        for z, got in ((0, k_all), (1, v_all)):
            rows_in = [r[z] for x in kept for r in x]
            if rows_in:
                want = torch.stack(rows_in)
                want = want.double() if bits == 16 else coded_ref.values(*coded_ref.quantise(want, bits), bits)
                assert torch.equal(got[:ends[-1]].cpu().double(), want)
        # the forward of the new rows, query heads of a group as rows of their own
        G, n = H // hk, int(offsets[-1])
        if n:
            q = turned[:n].view(n, hk, G, D).transpose(1, 2).reshape(n * G, hk, D).contiguous()
            new = np.diff(offsets.cpu().numpy())
            o, l = jfa.fwd_simple(q, k_all[:ends[-1]], v_all[:ends[-1]], ends, G * offsets.cpu().numpy(), scale=0.09)
            o = o.view(n, G, hk, D).transpose(1, 2).reshape(n, H, D)
            at = 0
            for b in range(B):
                if new[b] == 0:
                    continue
                kb, vb = (x[ends[b]:ends[b + 1]].double() for x in (k_all, v_all))
                for h in range(H):
                    s = 0.09 * turned[at:at + new[b], h].double() @ kb[:, h // G].T
                    want = torch.softmax(s, 1) @ vb[:, h // G]
                    mass = torch.softmax(s, 1) @ vb[:, h // G].abs()
                    # the forward's weights are bf16 (2^-8 of the mass), and so is its output (2^-8)
                    assert ((o[at:at + new[b], h].double() - want).abs() <= 2.0 ** -8 * (mass + want.abs()) * 1.01 + 1e-6).all()
                at += new[b]
        newest = (offsets[1:] - 1).clamp(min=0).long()
        full = [torch.zeros((B, width * page, hk, D), dtype=torch.float64) for _ in range(2)]  # a page for each request
        for b in range(B):
            for x, got in zip(full, (k_all, v_all)):
                x[b, :ends[b + 1] - ends[b]] = got[ends[b]:ends[b + 1]].cpu().double()
        ref, ref_lse, off, off_lse = coded_ref.decode(turned[newest], *full, _ints(np.arange(B)[:, None]), lens, 0.09)
        some = ~torch.isinf(ref_lse)
        assert ((out.cpu().double() - ref).abs() <= off).all()
        assert torch.equal(torch.isinf(lse.cpu()), ~some) and ((lse.cpu().double() - ref_lse).abs()[some] <= off_lse[some]).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_a_stream_of_its_own(bits):
    """stream= runs a call there, and makes its outputs there; the block of a dropped pager stays until its call is done."""
    pager, held, table, lens = _case([700, 33], 4, 2, 64, 16, "rows", bits, 14)
    q, off = _draw((2, 4, 64), 1), _ints([0, 700, 733])
    want = jfa.paged_decode(pager, q, *held[:2], table, lens, 0.125, **_scales(held))
    rows = jfa.paged_gather(pager, *held[:2], table, off, rows=733, **_scales(held))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = jfa.paged_decode(pager, q, *held[:2], table, lens, 0.125, **_scales(held), stream=stream)
        back = jfa.paged_gather(pager, *held[:2], table, off, rows=733, **_scales(held), stream=stream)
        jfa.paged_append(pager, back[0][:2], back[1][:2], _ints([-1, -1]), *held[:2], **_scales(held), stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *rows)))
        assert pager.status(stream=stream) == 0
    at, size = pager.block.data_ptr(), pager.block.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(600_000_000)
    jfa.paged_gather(pager, *held[:2], table, off, rows=733, **_scales(held), stream=side)
    del pager
    others = [torch.empty(size, dtype=U8, device="cuda") for _ in range(4)]
    assert not side.query()
    assert all(not at <= x.data_ptr() < at + size and not x.data_ptr() <= at < x.data_ptr() + size for x in others)
    side.synchronize()
