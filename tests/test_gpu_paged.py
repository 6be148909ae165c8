"""GPU tests of the paged-cache operators against their 64-bit plain forms.
Bounds on floating outputs are derived in paged_ref; whole numbers are equal."""
import ctypes
import math

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import paged_ref, parity

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


def _draw(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(BF16)


# ------------------------------------------------------------------ tables
def _tables_case(B, page, width, num_pages, most, seed, free_short=0):
    """A sound state: pages dealt out at random, some requests empty."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, B)
    lens[rng.random(B) < 0.2] = 0
    held = -(-lens // page)
    order = rng.permutation(num_pages)
    table = rng.integers(-5, num_pages + 5, (B, width))  # stale entries behind
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = rng.integers(0, num_pages, num_pages)
    n_free = num_pages - at
    free[:n_free] = order[at:]
    return rng, lens, table, free, n_free - free_short


def _run_tables(lens, delta, table, free, n_free, rows, page, num_pages, in_place=False, row_pad=0):
    B, width = table.shape
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=1, Hkv=1, D=64)
    wide = torch.full((B, width + row_pad), -77, dtype=I32, device="cuda")
    wide[:, :width] = _ints(table)
    dl, dd, df, dn = _ints(lens), _ints(delta), _ints(free), _ints([n_free])
    # outputs inside larger buffers, which stay as they were around them
    bufs = [torch.full((n + 64,), -99, dtype=I32, device="cuda") for n in (rows, rows, B + 1)]
    slots, positions, offsets = (t[32:32 + n] for t, n in zip(bufs, (rows, rows, B + 1)))
    got = jfa.paged_tables(pager, dl, dd, wide[:, :width], df, dn, rows=rows, slots=slots, positions=positions,
                           row_offsets=offsets, lens_out=dl if in_place else None,
                           n_free_out=dn if in_place else None)
    status = pager.status()
    assert pager.status() == 0
    for t, n in zip(bufs, (rows, rows, B + 1)):
        assert (t[:32] == -99).all() and (t[32 + n:] == -99).all()
    assert (wide[:, width:] == -77).all()
    want = paged_ref.tables(np.asarray(lens), np.asarray(delta), np.asarray(table), np.asarray(free), n_free, rows,
                            page, num_pages)
    names = ("lens", "n_free", "slots", "positions", "offsets", "table", "free_list")
    have = [got[0], got[1][0], got[2], got[3], got[4], wide[:, :width], df]
    for name, a, b in zip(names, have, want):
        assert np.array_equal(a.cpu().numpy().astype(np.int64), np.asarray(b)), name
    assert status == want[-1]
    return want


@pytest.mark.parametrize("B,page,width,most", [(1, 16, 8, 100), (3, 1, 40, 30), (33, 16, 12, 150), (200, 24, 9, 180),
                                               (1025, 8, 20, 130), (2500, 128, 3, 300)])
@pytest.mark.parametrize("seed", range(3))
def test_tables(B, page, width, most, seed):
    num_pages = B * width + 3
    rng, lens, table, free, n_free = _tables_case(B, page, width, num_pages, most, 10 * B + seed)
    room = width * page - lens
    delta = np.where(rng.random(B) < 0.3, -rng.integers(0, lens + 1), np.minimum(room, rng.integers(0, 2 * page + 3, B)))
    delta[rng.random(B) < 0.1] = 0
    rows = int(np.maximum(delta, 0).sum()) + int(rng.integers(0, 70))
    want = _run_tables(lens, delta, table, free, n_free, rows, page, num_pages, in_place=seed == 1, row_pad=seed)
    assert want[-1] == 0


def test_tables_of_single_tokens_and_of_nothing():
    rng, lens, table, free, n_free = _tables_case(64, 16, 10, 700, 150, 5)
    _run_tables(lens, np.ones(64, int), table, free, n_free, 64, 16, 700)
    _run_tables(lens, np.zeros(64, int), table, free, n_free, 0, 16, 700)
    _run_tables(lens, -lens, table, free, n_free, 3, 16, 700)


def test_tables_of_one_long_prompt():
    table, free = np.full((2, 9000), -1), np.random.default_rng(1).permutation(9000)
    _run_tables([0, 0], [1, 140001], table, free, 9000, 140002, 16, 9000)


@pytest.mark.parametrize("seed", range(4))
def test_tables_without_enough_pages(seed):
    """Requests that find no page stay as they were; those that need none go on."""
    B, page, width, num_pages = 40, 8, 12, 500
    rng, lens, table, free, n_free = _tables_case(B, page, width, num_pages, 70, seed)
    delta = np.where(rng.random(B) < 0.2, -rng.integers(0, lens + 1), rng.integers(0, 20, B))
    want = _run_tables(lens, delta, table, free, int(rng.integers(0, 12)), int(np.maximum(delta, 0).sum()), page, num_pages)
    assert want[-1] & paged_ref.NO_PAGES


def test_tables_leave_bad_requests_as_they_were():
    rng, lens, table, free, n_free = _tables_case(12, 4, 5, 80, 18, 9)
    delta = np.ones(12, int)
    lens[1], lens[2], delta[3], delta[4] = -3, 21, 30, -40
    delta[5], lens[6], delta[7] = 2**31 - 1, 2**31 - 1, -2**31
    want = _run_tables(lens, delta, table, free, n_free, 9, 4, 80)
    assert want[-1] & paged_ref.BAD_LENGTH
    # rows that do not hold all new tokens
    rng, lens, table, free, n_free = _tables_case(12, 4, 5, 80, 8, 9)
    want = _run_tables(lens, np.full(12, 3), table, free, n_free, 20, 4, 80)
    assert want[-1] == paged_ref.BAD_LENGTH
    # a free count outside the cache: nothing changes
    for bad in (-1, 81, 2**31 - 1, 79):
        d = np.where(np.arange(12) % 2, -lens, 2)
        want = _run_tables(lens, d, table, free, bad, 30, 4, 80)
        assert want[-1] & paged_ref.BAD_PAGE and want[1] == bad and np.array_equal(want[0], lens)
    # pages outside the cache on the free list: their rows get no slot
    free = free.copy()
    free[:n_free] = -7
    want = _run_tables(lens, np.full(12, 5), table, free, n_free, 60, 4, 80)
    assert want[-1] & paged_ref.BAD_PAGE


def test_tables_over_many_steps_in_place_and_captured():
    """One captured step replayed while requests come, grow and leave."""
    B, page, width, num_pages, rows = 16, 8, 10, 120, 100
    rng = np.random.default_rng(3)
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=1, Hkv=1, D=64)
    lens, delta, n_free = _ints(np.zeros(B)), _ints(np.zeros(B)), _ints([num_pages])
    table, free = _ints(np.full((B, width), -1)), _ints(rng.permutation(num_pages))
    slots, positions, offsets = (torch.empty(n, dtype=I32, device="cuda") for n in (rows, rows, B + 1))
    state = [x.cpu().numpy().astype(np.int64) for x in (lens, table, free)] + [num_pages]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jfa.paged_tables(pager, lens, delta, table, free, n_free, rows=rows, lens_out=lens, n_free_out=n_free,
                         slots=slots, positions=positions, row_offsets=offsets)
    for _ in range(40):
        d = np.where(rng.random(B) < 0.25, -rng.integers(0, state[0] + 1), rng.integers(0, 7, B))
        d = np.minimum(d, width * page - state[0])
        delta.copy_(_ints(d))
        graph.replay()
        out = paged_ref.tables(state[0], d, state[1], state[2], state[3], rows, page, num_pages)
        assert pager.status() == out[-1]
        for a, b in zip((lens, n_free, slots, positions, offsets, table, free),
                        (out[0], [out[1]], out[2], out[3], out[4], out[5], out[6])):
            assert np.array_equal(a.cpu().numpy().astype(np.int64), np.asarray(b))
        state = [out[0], out[5], out[6], out[1]]


# ------------------------------------------------------------------ append
def _cache(num_pages, page, hk, D, heads_first, seed):
    shape = (num_pages, hk, page, D) if heads_first else (num_pages, page, hk, D)
    k, v = _draw(shape, seed), _draw(shape, seed + 1)
    return (k.transpose(1, 2), v.transpose(1, 2)) if heads_first else (k, v)


@pytest.mark.parametrize("rows,hq,hk,D,page,heads_first", [
    (1, 4, 4, 128, 16, False), (37, 12, 3, 64, 24, True), (300, 8, 1, 128, 1, False), (129, 16, 8, 64, 128, True),
    (1000, 2, 2, 128, 7, False)])
@pytest.mark.parametrize("rotary", [None, "half", "interleaved"])
def test_append(rows, hq, hk, D, page, heads_first, rotary):
    num_pages = -(-2 * rows // page) + 2
    pager = jfa.Pager(max_seqs=4, max_pages=4, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D)
    kp, vp = _cache(num_pages, page, hk, D, heads_first, 1)
    want_k, want_v = kp.clone(), vp.clone()
    x = _draw((rows, hq + 2 * hk, D), 3)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    rng = np.random.default_rng(rows)
    slots = rng.permutation(num_pages * page)[:rows]
    slots[rng.random(rows) < 0.2] = -1
    if rows > 5:
        slots[1], slots[2] = -2**31, -5
    else:
        slots[0] = num_pages * page - 1
    half = D // 2 - 8
    freq, axis = jfa.rotary_pairs(2 * half, (half - 9, 9))
    rot = None if rotary is None else jfa.Rotary(freq, axis, D=D, interleaved=rotary == "interleaved")
    pos = None if rot is None else torch.randint(0, 10**6, (rows, 2), device="cuda", dtype=I32)
    gq = None if rot is None else parity.guarded((rows, hq, D), BF16)
    got = jfa.paged_append(pager, k, v, _ints(slots), kp, vp, rotary=rot, positions=pos,
                           q=None if rot is None else q, q_out=None if rot is None else gq.t)
    assert pager.status() == 0
    live = np.flatnonzero(slots >= 0)
    page_of, row_of = torch.as_tensor(slots[live] // page).cuda(), torch.as_tensor(slots[live] % page).cuda()
    written = kp[page_of, row_of]
    if rot is None:
        assert got is None and torch.equal(written, k[live])
    else:
        for a, b in ((written, k[live]), (gq.t, q)):
            at = pos if b is q else pos[live]
            ref = paged_ref.rotate(b, at, freq, axis, rot.interleaved)
            bound = paged_ref.rotate_bound(b, ref, half, rot.interleaved, BF16)
            assert ((a.cpu().double() - ref).abs() <= bound).all()
        gq.check("q")
        assert got is gq.t
    want_k[page_of, row_of], want_v[page_of, row_of] = written, v[live]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)  # all other rows as they were


def test_append_leaves_out_slots_outside_the_cache():
    """The row kernel compares a slot with the cache's size before it uses it."""
    pager = jfa.Pager(max_seqs=1, max_pages=1, num_pages=3, page_size=5, H=2, Hkv=2, D=64)
    kp, vp = _cache(3, 5, 2, 64, False, 1)
    k, v = _draw((4, 2, 64), 3), _draw((4, 2, 64), 4)
    want = kp.clone()
    jfa.paged_append(pager, k, v, _ints([15, 14, 2**31 - 1, -1]), kp, vp)
    want[2, 4] = k[1]
    assert torch.equal(kp, want) and torch.equal(vp[2, 4], v[1])
    assert pager.status() == jfa.PAGER_BAD_PAGE and pager.status() == 0


# ------------------------------------------------------------------ decode
def _decode_case(lens, hq, hk, D, page, heads_first, seed, spread=1.0, width=None):
    lens = np.asarray(lens)
    count = -(-lens // page)
    width = max(1, int(count.max())) if width is None else width
    rng = np.random.default_rng(seed)
    num_pages = int(count.sum()) + 3
    order = rng.permutation(num_pages)
    table = rng.integers(-2**31, 2**31, (len(lens), width))  # nothing behind the length is looked at
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    kp, vp = _cache(num_pages, page, hk, D, heads_first, seed)
    if spread != 1.0:
        kp.mul_(spread)
    # what lies behind a sequence's last row, and on pages of nobody
    dead = torch.ones((num_pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            dead[table[b, t // page], t % page] = False
    dead = dead.cuda()
    for x, bad in ((kp, float("nan")), (vp, float("inf"))):
        x[dead] = bad
    q = _draw((len(lens), hq, D), seed + 7)
    pager = jfa.Pager(max_seqs=len(lens), max_pages=width, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D)
    return pager, q, kp, vp, _ints(table), _ints(lens)


def _check_decode(pager, q, kp, vp, table, lens, scale=None, status=0):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    go, gl = parity.guarded((*q.shape[:2], q.shape[2]), BF16), parity.guarded((q.shape[1], q.shape[0]), F32)
    out, lse = jfa.paged_decode(pager, q, kp, vp, table, lens, scale, out=go.t, lse=gl.t)
    assert pager.status() == status
    go.check("out")
    gl.check("lse")
    ref, ref_lse, off, off_lse = paged_ref.decode(q, kp, vp, table, lens, scale)
    o, l = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(o).all()
    err = (o - ref).abs()
    assert (err <= off).all(), float((err / off.clamp(min=1e-300)).max())
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(l), empty) and (l[empty] < 0).all()
    assert ((l - ref_lse).abs()[~empty] <= off_lse[~empty]).all(), float((l - ref_lse).abs()[~empty].max())
    return out, lse


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 511, 1000]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 4), (6, 2), (4, 1), (15, 3), (6, 1), (14, 2), (8, 1), (9, 1),
                                   (24, 2), (16, 1), (17, 1), (40, 1), (48, 1), (66, 2), (128, 1), (130, 1),
                                   (300, 1)])
def test_decode_head_groups(D, hq, hk):
    _check_decode(*_decode_case(EDGES, hq, hk, D, 16, False, hq * 100 + hk))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 3, 8, 24, 32, 64, 100, 128, 1024])
@pytest.mark.parametrize("heads_first", [False, True])
def test_decode_pages(D, page, heads_first):
    _check_decode(*_decode_case(EDGES, 4, 2, D, page, heads_first, page))


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [1] * 700, [5000], [3, 20000], [20000, 0, 1], [129] * 152,
                                  list(range(300)), [0] * 300 + [4000]], ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1)])
def test_decode_splits(lens, hq, hk):
    """Few long rows, many short ones, and both: every way a row is cut and joined."""
    _check_decode(*_decode_case(lens, hq, hk, 128, 16, False, len(lens)))


def test_decode_wide_table_and_long_scores():
    """Entries behind the length are never followed; peaked softmax; scale 0 and below."""
    case = _decode_case([40, 700, 3], 4, 2, 128, 16, False, 3, spread=30.0, width=500)
    _check_decode(*case)
    _check_decode(*case, scale=0.0)
    _check_decode(*case, scale=-0.3)


def test_decode_scores_of_minus_infinity_and_huge_keys():
    """A key whose score overflows downwards takes no weight, also where it is the first of its part."""
    pager, q, kp, vp, table, lens = _decode_case([300], 2, 2, 64, 16, False, 4)
    q.fill_(1.0)
    for t in (0, 1, 2, 3, 16, 17, 200, 299):
        kp[table[0, t // 16], t % 16] = -3e38  # q . k = -inf in fp32
    keep = [t for t in range(300) if t not in (0, 1, 2, 3, 16, 17, 200, 299)]
    out, lse = jfa.paged_decode(pager, q, kp, vp, table, lens, 1.0)
    t = torch.tensor(keep).cuda()
    page = table[0, t // 16].long()
    k, v = (x[page, t % 16].double().cpu() for x in (kp, vp))
    for h in range(2):
        s = k[:, h].sum(1)
        want = torch.softmax(s, 0) @ v[:, h]
        assert (out[0, h].cpu().double() - want).abs().max() <= 2.0 ** -8 * v.abs().max()
        assert abs(float(lse[h, 0]) - float(torch.logsumexp(s, 0))) < 1e-3


def test_decode_bad_lengths_and_pages():
    """Lengths outside the table are empty rows, pages outside the cache are left out."""
    pager, q, kp, vp, table, lens = _decode_case([40, 100, 64, 33, 16], 4, 2, 64, 16, True, 5)
    lens[0], lens[3] = -1, 2**31 - 1
    _check_decode(pager, q, kp, vp, table, lens, status=jfa.PAGER_BAD_LENGTH)
    lens[0], lens[3] = 40, 33
    num = kp.shape[0]
    table[1, 2], table[2, 0], table[3, 0], table[3, 1], table[3, 2], table[4, 0] = num, -1, num, 2**31 - 1, -2**31, num
    _check_decode(pager, q, kp, vp, table, lens, status=jfa.PAGER_BAD_PAGE)


def test_decode_strided_q_is_the_same_and_runs_repeat_bit_for_bit():
    lens = [3000, 17, 0, 900]
    pager, q, kp, vp, table, lens = _decode_case(lens, 8, 2, 128, 16, False, 6)
    out, lse = _check_decode(pager, q, kp, vp, table, lens)
    wide = torch.zeros((4, 13, 128), dtype=BF16, device="cuda")
    wide[:, 2:10] = q
    for _ in range(20):
        o, l = jfa.paged_decode(pager, wide[:, 2:10], kp, vp, table, lens, 1 / math.sqrt(128))
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_decode_fewer_requests_than_the_pager_holds():
    pager, q, kp, vp, table, lens = _decode_case([500, 20, 1500], 8, 2, 128, 16, False, 8)
    big = jfa.Pager(max_seqs=100, max_pages=pager.max_pages, num_pages=kp.shape[0], page_size=16, H=8, Hkv=2, D=128)
    for n in (3, 1, 2):
        _check_decode(big, q[:n], kp, vp, table[:n], lens[:n])


def test_decode_captured_with_changing_lengths_and_streams():
    """A graph replayed with other lengths, eager calls in between, and two
    pagers decoding at once on two streams."""
    case = _decode_case([2000, 300, 64, 5], 8, 2, 128, 16, False, 9)
    pager, q, kp, vp, table, lens = case
    other = jfa.Pager(max_seqs=4, max_pages=pager.max_pages, num_pages=kp.shape[0], page_size=16, H=8, Hkv=2, D=128)
    out, lse = torch.empty_like(q), torch.empty((8, 4), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1, out=out, lse=lse)
    for new in ([2000, 300, 64, 5], [1, 0, 60, 4], [1999, 299, 1, 0], [0, 0, 0, 0]):
        lens.copy_(_ints(new))
        graph.replay()
        a, b = jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1)
        assert torch.equal(a, out) and torch.equal(b, lse)
        _check_decode(*case)
    lens.copy_(_ints([2000, 300, 64, 5]))
    want, _ = jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(30):
        for s, p, o in zip(streams, (pager, other), outs):
            with torch.cuda.stream(s):
                o.append(jfa.paged_decode(p, q, kp, vp, table, lens, 0.1)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for o in outs for x in o)


@pytest.mark.parametrize("heads_first", [False, True])
def test_decode_and_append_past_32_bit_offsets(heads_first):
    """The last pages of a cache of more than 2^31 values per tensor."""
    hk, D, page, num_pages = 8, 128, 64, (1 << 15) + 40
    shape = (num_pages, hk, page, D) if heads_first else (num_pages, page, hk, D)
    kp, vp = (torch.zeros(shape, dtype=BF16, device="cuda") for _ in range(2))
    if heads_first:
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    pager = jfa.Pager(max_seqs=2, max_pages=12, num_pages=num_pages, page_size=page, H=16, Hkv=hk, D=D)
    n = 700
    table = _ints(np.stack([num_pages - 1 - np.arange(12), np.arange(12)]))
    t = torch.arange(n, device="cuda")
    slots = (table[0, t // page] * page + t % page).to(I32)
    k, v = _draw((n, hk, D), 1), _draw((n, hk, D), 2)
    jfa.paged_append(pager, k, v, slots, kp, vp)
    assert torch.equal(kp[table[0, t // page].long(), t % page], k)
    assert not kp[:num_pages - 12].any() and not vp[:num_pages - 12].any()
    _check_decode(pager, _draw((2, 16, D), 3), kp, vp, table, _ints([n, 70]))


def test_refusals_of_the_binding():
    pager, q, kp, vp, table, lens = _decode_case([40, 20], 4, 2, 64, 16, False, 5)
    call = lambda **kw: jfa.paged_decode(**{**dict(pager=pager, q=q, k_pages=kp, v_pages=vp, table=table, lens=lens,  # noqa: E731
                                                   scale=0.1), **kw})
    call()
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(k_pages=kp.half()), dict(lens=lens.long()),
                dict(table=table.long()), dict(lens=lens.cpu())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=q[:, :2]), dict(k_pages=kp[1:], v_pages=vp[1:]), dict(table=table[:, :1]), dict(table=table[:1]),
                dict(lens=lens[:1]), dict(v_pages=vp.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(lse=torch.empty(2, 4, device="cuda")), dict(out=torch.empty(2, 8, 64, dtype=BF16, device="cuda")[:, :4])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(jfa.JfaError):
        call(scale=float("nan"))
    with pytest.raises(jfa.JfaError) as e:  # more requests than the pager holds
        call(q=q[[0, 1, 0]], table=table[[0, 1, 0]], lens=lens[[0, 1, 0]])
    assert e.value.code == 1
    k = _draw((2, 2, 64), 1)
    slots = _ints([0, 1])
    with pytest.raises(ValueError):
        jfa.paged_append(pager, k, k, slots, kp, vp, q=q)
    with pytest.raises(ValueError):
        jfa.paged_append(pager, k, k, slots, kp, vp, rotary=jfa.Rotary(*jfa.rotary_pairs(64), D=64))
    with pytest.raises(ValueError):
        jfa.paged_append(pager, k, k[:1], slots, kp, vp)
    with pytest.raises(jfa.JfaError):  # a rotary of another head dimension
        jfa.paged_append(pager, k, k, slots, kp, vp, rotary=jfa.Rotary(*jfa.rotary_pairs(64), D=128), positions=slots)
    with pytest.raises(TypeError):
        jfa.paged_append(pager, k, k, slots.long(), kp, vp)
    with pytest.raises(ValueError):
        jfa.paged_tables(pager, lens, lens, table, _ints([0]), _ints([0]), rows=4)
    pager.close()
    with pytest.raises(RuntimeError):
        call()


def test_host_refusals_with_a_pager():
    """Argument checks of the C entries that need a handle; nothing launches."""
    pager, q, kp, vp, table, lens = _decode_case([40, 20], 4, 2, 64, 16, False, 5)
    L, h = jfa.lib(), pager.handle
    st = kp.stride()

    def pages(**kw):
        a = dict(k=kp.data_ptr(), v=vp.data_ptr(), page=st[0], row=st[1], head=st[2])
        a.update(kw)
        return ctypes.byref(jfa._Pages(**a))

    out, lse = torch.empty_like(q), torch.empty((4, 2), device="cuda")
    good = [h, 2, q.data_ptr(), 256, pages(), table.data_ptr(), table.stride(0), lens.data_ptr(), 0.1, out.data_ptr(),
            lse.data_ptr(), None]
    for at, value, code in [(1, 0, 1), (1, 3, 1), (2, None, 1), (2, q.data_ptr() + 2, 4), (3, 255, 1), (3, 260, 4),
                            (4, None, 1), (4, pages(k=None), 1), (4, pages(v=vp.data_ptr() + 8), 4),
                            (4, pages(row=st[1] + 4), 4), (4, pages(page=-8), 1), (5, None, 1),
                            (6, pager.max_pages - 1, 1), (7, None, 1), (8, math.inf, 1), (9, None, 1),
                            (9, out.data_ptr() + 8, 4), (10, None, 1)]:
        args = list(good)
        args[at] = value
        assert L.jfa_paged_decode(*args) == code, (at, value)
    k = _draw((2, 2, 64), 1)
    s = _ints([0, 1])
    rot = jfa.Rotary(*jfa.rotary_pairs(64), D=64)
    good = [h, 2, k.data_ptr(), 128, k.data_ptr(), 128, s.data_ptr(), pages(), rot.handle, s.data_ptr(), 1, 0,
            q.data_ptr(), 256, out.data_ptr(), 256, None]
    for at, value, code in [(1, -1, 1), (2, None, 1), (3, 120, 1), (4, k.data_ptr() + 2, 4), (5, 132, 4), (6, None, 1),
                            (7, None, 1), (8, None, 1), (9, None, 1), (10, -1, 1), (12, None, 1), (14, None, 1),
                            (15, 264 - 4, 4)]:
        args = list(good)
        args[at] = value
        assert L.jfa_paged_append(*args) == code, (at, value)
    free = _ints(np.zeros(pager.num_pages))
    one, off = _ints([0]), _ints([0, 0, 0])
    good = [h, 2, lens.data_ptr(), s.data_ptr(), lens.data_ptr(), table.data_ptr(), table.stride(0), free.data_ptr(),
            one.data_ptr(), one.data_ptr(), 2, s.data_ptr(), s.data_ptr(), off.data_ptr(), None]
    for at, value, code in [(1, 0, 1), (1, 3, 1), (2, None, 1), (3, None, 1), (4, None, 1), (5, None, 1),
                            (5, table.data_ptr() + 2, 4), (6, pager.max_pages - 1, 1), (7, None, 1), (8, None, 1),
                            (3, lens.data_ptr(), 1), (9, None, 1), (9, lens.data_ptr(), 1), (10, -1, 1), (10, 2**31, 1), (11, None, 1), (12, None, 1), (13, None, 1)]:
        args = list(good)
        args[at] = value
        assert L.jfa_paged_tables(*args) == code, (at, value)


# ------------------------------------------------- a serving run of them all
@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(captured):
    """Requests enter with a prompt, decode a token a step, drop their last tokens
    and leave; every step is tables, append with rotation and decode, and every
    output is checked against attention in 64 bits over the rows a request kept."""
    H, hk, D, page, width, num_pages, B, rows = 8, 2, 128, 8, 12, 60, 6, 64
    freq, axis = jfa.rotary_pairs(D, (32, 16, 16))
    rot = jfa.Rotary(freq, axis, D=D)
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=H, Hkv=hk, D=D)
    kp, vp = (torch.full((num_pages, page, hk, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    lens, delta, n_free = _ints(np.zeros(B)), _ints(np.zeros(B)), _ints([num_pages])
    table, free = _ints(np.full((B, width), -1)), _ints(np.random.default_rng(0).permutation(num_pages))
    slots, positions, offsets = (torch.empty(n, dtype=I32, device="cuda") for n in (rows, rows, B + 1))
    qkv = torch.zeros((rows, H + 2 * hk, D), dtype=BF16, device="cuda")
    turned = torch.empty((rows, H, D), dtype=BF16, device="cuda")
    last, out, lse = _ints(np.zeros(B)), torch.empty((B, H, D), dtype=BF16, device="cuda"), torch.empty((H, B), device="cuda")

    def step():
        jfa.paged_tables(pager, lens, delta, table, free, n_free, rows=rows, lens_out=lens, n_free_out=n_free,
                         slots=slots, positions=positions, row_offsets=offsets)
        jfa.paged_append(pager, qkv[:, H:H + hk], qkv[:, H + hk:], slots, kp, vp, rotary=rot, positions=positions,
                         q=qkv[:, :H], q_out=turned)
        newest = (offsets[1:] - 1).clamp(min=0).long()
        jfa.paged_decode(pager, turned[newest], kp, vp, table, lens, 0.09, out=out, lse=lse)

    if captured:
        step()  # warm up, with nothing to do
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    rng = np.random.default_rng(1)
    kept = [[] for _ in range(B)]  # (k, v) of each request's rows, in float64
    for i in range(25):
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
        at, x = 0, qkv.cpu().double()
        pos = torch.zeros(rows, dtype=torch.long)
        for b in range(B):
            for j in range(max(d[b], 0)):
                pos[at + j] = len(kept[b]) + j
            at += max(d[b], 0)
        # the cache holds bf16: round the rotated key and query as it does
        q64 = paged_ref.rotate(x[:, :H], pos, freq, axis)
        k64 = paged_ref.rotate(x[:, H:H + hk], pos, freq, axis)
        at = 0
        for b in range(B):
            if d[b] < 0:
                kept[b] = kept[b][:len(kept[b]) + d[b]]
                continue
            kept[b] += [(k64[at + j], x[at + j, H + hk:]) for j in range(d[b])]
            at += d[b]
            if d[b] == 0:
                continue
            k, v = (torch.stack([r[z] for r in kept[b]]) for z in range(2))
            for h in range(H):
                g, qh = h // (H // hk), q64[at - 1, h]
                s = 0.09 * (k[:, g] @ qh)
                # rounding q and k to bf16 (half a step each, and the rotation's own error, below a
                # hundredth of that) moves a score by at most 2.1 half steps of sum |q k|
                half = torch.finfo(BF16).eps / 2
                moved = 2.1 * half * 0.09 * float((k[:, g].abs() @ qh.abs()).max()) + 1e-4
                w = torch.softmax(s, 0)
                want = w @ v[:, g]
                bound = (math.exp(2 * moved) - 1) * (w @ v[:, g].abs()) + half * 1.1 * want.abs() + 1e-6
                assert ((out[b, h].cpu().double() - want).abs() <= bound).all()
                assert abs(float(lse[h, b]) - float(torch.logsumexp(s, 0))) <= moved + 1e-5
        lens_now = lens.cpu().numpy()
        assert [len(x) for x in kept] == lens_now.tolist()


@pytest.mark.parametrize("hq,hk,D", [(16, 8, 64), (32, 2, 64), (40, 2, 64), (10, 2, 128), (32, 2, 128), (70, 2, 128)])
def test_decode_tables_wide_enough_for_64_bit_counts(hq, hk, D):
    """A table of which full rows would hold more tiles than 32 bits count."""
    pager, q, kp, vp, table, lens = _decode_case([300, 5000, 0, 17], hq, hk, D, 1024, False, 12)
    pages = (1 << 21) - 2
    wide = torch.full((64, pages), -1, dtype=I32, device="cuda")  # 0.5 GB; only the rows of 64 requests count
    wide[:4, :table.shape[1]] = table
    big = jfa.Pager(max_seqs=64, max_pages=pages, num_pages=kp.shape[0], page_size=1024, H=hq, Hkv=hk, D=D)
    assert 64 * (pages * 1024 // 32) > 2**32 // hk
    many = torch.zeros((64, hq, D), dtype=BF16, device="cuda")
    many[:4] = q
    some = torch.zeros(64, dtype=I32, device="cuda")
    some[:4] = lens
    out, lse = _check_decode(big, many, kp, vp, wide, some)
    narrow = jfa.paged_decode(pager, q, kp, vp, table, lens, 1 / math.sqrt(D))
    assert torch.equal(out[:4], narrow[0]) and torch.equal(lse[:, :4], narrow[1])
    assert not out[4:].any() and torch.isinf(lse[:, 4:]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(16, 1), (12, 1), (3, 1), (40, 2), (100, 1)])
def test_decode_rows_of_many_parts(D, hq, hk):
    """Rows that all CTAs share: their parts are joined in groups first."""
    case = _decode_case([20000, 0, 7000, 9001], hq, hk, D, 24, False, 31)
    out, lse = _check_decode(*case)
    for _ in range(5):
        o, l = jfa.paged_decode(*case, 1 / math.sqrt(D))
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_a_stream_of_its_own():
    """stream= runs a call there, and makes its outputs there."""
    pager, q, kp, vp, table, lens = _decode_case([700, 33], 4, 2, 64, 16, False, 14)
    want = jfa.paged_decode(pager, q, kp, vp, table, lens, 0.125)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = jfa.paged_decode(pager, q, kp, vp, table, lens, 0.125, stream=stream)
        rot = jfa.Rotary(*jfa.rotary_pairs(64), D=64)
        turned = jfa.rotate(rot, lens, q, stream=stream)
        jfa.paged_append(pager, kp[0, :2], vp[0, :2], _ints([-1, -1]), kp, vp, stream=stream)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(turned, jfa.rotate(rot, lens, q))
        assert pager.status(stream=stream) == 0
    table2, free = _ints(np.zeros((2, pager.max_pages))), _ints(np.arange(pager.num_pages))
    got = jfa.paged_tables(pager, _ints([0, 0]), _ints([3, 5]), table2, free, _ints([pager.num_pages]), rows=8,
                           stream=side.cuda_stream)
    side.synchronize()
    assert got[0].tolist() == [3, 5]


@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2)])
def test_decode_the_most_requests(hq, hk):
    """16384 requests of 0 to 40 rows, a page of 40 each, against a batched 64-bit softmax."""
    B, page, D = 16384, 40, 64
    rng = np.random.default_rng(1)
    lens, order = rng.integers(0, page + 1, B), rng.permutation(B)
    pager = jfa.Pager(max_seqs=B, max_pages=1, num_pages=B, page_size=page, H=hq, Hkv=hk, D=D)
    kp, vp, q = _draw((B, page, hk, D), 1), _draw((B, page, hk, D), 2), _draw((B, hq, D), 3)
    table, dl = _ints(order[:, None]), _ints(lens)
    out, lse = jfa.paged_decode(pager, q, kp, vp, table, dl, 0.125)
    assert pager.status() == 0
    k, v = (x[table[:, 0].long()].double().repeat_interleave(hq // hk, 2) for x in (kp, vp))
    s = 0.125 * torch.einsum("bhd,bthd->bht", q.double(), k)
    size = 0.125 * torch.einsum("bhd,bthd->bht", q.double().abs(), k.abs()).amax(-1)
    dead = torch.arange(page, device="cuda")[None, None] >= dl[:, None, None]
    w = torch.softmax(s.masked_fill(dead, -math.inf), -1).nan_to_num(0.0)
    want, mass = torch.einsum("bht,bthd->bhd", w, v), torch.einsum("bht,bthd->bhd", w, v.abs())
    # the bounds of paged_ref.decode
    delta = 2 * D * 2.0 ** -24 * size + 2.0 ** -15 + 2 * page * 2.0 ** -24
    step = torch.finfo(BF16).eps / 2
    assert ((out.double() - want).abs() <= 2 * delta[..., None] * mass * (1 + step) + step * want.abs()).all()
    ref = torch.logsumexp(s.masked_fill(dead, -math.inf), -1)
    some = (dl > 0)[:, None].expand_as(ref)
    assert ((lse.T.double() - ref).abs()[some] <= (delta + 2.0 ** -23 * ref.abs())[some]).all()
    assert (lse.T[~some] == -math.inf).all()


def test_tables_of_the_most_requests():
    B, page, width = 16384, 4, 3
    rng, lens, table, free, n_free = _tables_case(B, page, width, B * width, page * width - 3, 21)
    delta = np.where(rng.random(B) < 0.4, -rng.integers(0, lens + 1), rng.integers(0, 4, B))
    _run_tables(lens, delta, table, free, n_free, int(np.maximum(delta, 0).sum()) + 5, page, B * width, in_place=True)


def test_tables_down_to_the_last_page():
    """A step that takes every free page, and one that wants one more."""
    table = np.array([[0, -1, -1], [1, -1, -1], [2, -1, -1]])
    free = np.array([5, 4, 3, 0, 0, 0])
    want = _run_tables([4, 4, 4], [1, 1, 1], table, free, 3, 3, 4, 6)
    assert want[1] == 0 and want[-1] == 0
    want = _run_tables([4, 4, 4], [1, 5, 1], table, free, 3, 7, 4, 6)
    assert want[-1] == paged_ref.NO_PAGES and want[1] == 0
    want = _run_tables([4, 4, 4], [1, -4, 5], table, free, 2, 6, 4, 6)  # served from what the second gives back
    assert want[-1] == 0 and want[1] == 0


@pytest.mark.parametrize("B", [2, 31, 32, 33, 63, 255, 256, 257, 512, 513])
@pytest.mark.parametrize("most", [50, 700])
def test_decode_request_counts(B, most):
    """As many requests as lanes, threads and slabs of threads have, and one more or less; some empty at either end."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most, B)
    lens[rng.random(B) < 0.3] = 0
    lens[-1] = 0 if B % 2 else most
    _check_decode(*_decode_case(lens, 2, 1, 64, 16, False, B))


def test_strides_of_dimensions_of_one_do_not_matter():
    """A single head or page, and pages of one row, whose strides torch leaves at anything."""
    def odd(x, dim, stride):
        st = list(x.stride())
        st[dim] = stride
        return x.as_strided(x.shape, st)

    for page, hk, lens, dim in ((1, 2, [30, 5], 1), (16, 1, [30, 5], 2), (64, 2, [50], 0)):
        pager, q, kp, vp, table, n = _decode_case(lens, 2, hk, 64, page, False, 3)
        if dim == 0:  # one page
            pager = jfa.Pager(max_seqs=1, max_pages=1, num_pages=1, page_size=64, H=2, Hkv=2, D=64)
            kp, vp, table = kp[table[0].long()], vp[table[0].long()], torch.zeros_like(table)
        want = jfa.paged_decode(pager, q, kp, vp, table, n, 0.125)
        for a, b in ((3, 3), (3, 5), (1 << 40, 7)):
            got = jfa.paged_decode(pager, q, odd(kp, dim, a), odd(vp, dim, b), table, n, 0.125)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        _check_decode(pager, q, odd(kp, dim, 3), odd(vp, dim, 3), table, n)
