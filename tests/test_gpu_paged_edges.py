"""GPU tests of the paged-cache operators at values and sizes where they can go
wrong, against their 64-bit plain forms."""
import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import paged_ref

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


def _case(lens, hq, hk, D, page, seed):
    """(pager, q, k_pages, v_pages, table, lens): pages dealt out at random."""
    lens = np.asarray(lens)
    count = -(-lens // page)
    width, num_pages = max(1, int(count.max())), max(1, int(count.sum()))
    order, at = np.random.default_rng(seed).permutation(num_pages), 0
    table = np.full((len(lens), width), -1)
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    kp, vp = _draw((num_pages, page, hk, D), seed), _draw((num_pages, page, hk, D), seed + 1)
    pager = jfa.Pager(max_seqs=len(lens), max_pages=width, num_pages=num_pages, page_size=page, H=hq, Hkv=hk, D=D)
    return pager, _draw((len(lens), hq, D), seed + 2), kp, vp, _ints(table), _ints(lens)


def _same_class(a, b):
    """NaN, +inf and -inf in the same places."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a == np.inf, b == np.inf) and \
        torch.equal(a == -np.inf, b == -np.inf)


@pytest.mark.parametrize("lens", [[1], [2, 0, 31], [300, 17], [9000, 40, 1]], ids=str)
@pytest.mark.parametrize("hq,hk,D", [(1, 1, 64), (4, 2, 128), (16, 1, 128), (24, 1, 64)])
def test_decode_infinite_values(lens, hq, hk, D):
    """An infinite value of V among the rows of a request makes its output infinite, as
    its weight is above 0; infinities of both signs make a NaN; all else is as before."""
    pager, q, kp, vp, table, dl = _case(lens, hq, hk, D, 16, 3)
    flat = vp.view(-1, hk, D)
    for b, n in enumerate(lens):
        for t in range(0, n, 7):  # one value of a row each, the two signs in columns of their own
            at = int(table[b, t // 16]) * 16 + t % 16
            flat[at, t % hk, 2 * (t % (D // 4))] = np.inf
            flat[at, t % hk, 1 + 2 * (t % (D // 4))] = -np.inf
        if n > 20:
            for t, sign in ((3, np.inf), (19, -np.inf)):
                flat[int(table[b, t // 16]) * 16 + t % 16, 0, D - 3] = sign
    out, lse = jfa.paged_decode(pager, q, kp, vp, table, dl, D ** -0.5)
    assert pager.status() == 0
    ref, ref_lse, off, off_lse = paged_ref.decode(q, kp, vp, table, dl, D ** -0.5)
    o, finite = out.cpu().double(), torch.isfinite(ref)
    assert _same_class(o, ref) and torch.isinf(ref).any() and finite.any()
    assert ((o - ref).abs()[finite] <= off[finite]).all()
    some = torch.isfinite(ref_lse)
    assert ((lse.cpu().double() - ref_lse).abs()[some] <= off_lse[some]).all()


def _us(call, n=10):
    """Microseconds of a captured call, the fastest of five replays of n."""
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    best = np.inf
    for _ in range(6):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3 / n)
    return best


@pytest.mark.parametrize("B,each", [(256, 1500), (5000, 3000), (16384, 1500), (16384, 100000)])
def test_tables_of_a_few_growing_requests_among_many(B, each):
    """New rows in the first, a middle and the last request alone: right, and in no more
    than three times the time that they take next to one another."""
    page = 16
    width = -(-each // page)
    num_pages = 3 * width + 1
    pager = jfa.Pager(max_seqs=B, max_pages=width, num_pages=num_pages, page_size=page, H=1, Hkv=1, D=64)
    free = np.random.default_rng(B).permutation(num_pages)
    lens, n_free = _ints(np.zeros(B)), _ints([num_pages])
    rows, table = 3 * each + 5, torch.full((B, width), -1, dtype=I32, device="cuda")
    took = {}
    for where in ((0, B // 2, B - 1), (0, 1, 2)):
        delta = np.zeros(B, int)
        delta[list(where)] = each
        args, dfree = (lens, _ints(delta), table), _ints(free)
        slots, positions, offsets = (torch.empty(n, dtype=I32, device="cuda") for n in (rows, rows, B + 1))

        def call():
            return jfa.paged_tables(pager, *args, dfree, n_free, rows=rows, slots=slots, positions=positions,
                                    row_offsets=offsets)

        got, new = call(), np.arange(each)
        assert pager.status() == 0
        pages = [free[num_pages - 1 - i * width - np.arange(width)] for i in range(3)]
        want = np.concatenate([p[new // page] * page + new % page for p in pages] + [np.full(5, -1)])
        assert np.array_equal(got[2].cpu().numpy(), want)
        assert np.array_equal(got[3].cpu().numpy(), np.concatenate([new, new, new, np.zeros(5, int)]))
        assert np.array_equal(got[4].cpu().numpy(), np.concatenate([[0], np.cumsum(delta)]))
        assert np.array_equal(got[0].cpu().numpy(), delta) and int(got[1]) == num_pages - 3 * width
        for b, p in zip(where, pages):
            assert np.array_equal(table[b].cpu().numpy(), p)
        took[where[1]] = _us(call)
    assert took[B // 2] <= 3 * took[1], took


@pytest.mark.parametrize("B,hq,hk", [(2048, 8, 2), (2048, 24, 1), (16384, 8, 2)])
def test_decode_of_a_few_requests_among_many(B, hq, hk):
    """Three requests with rows, far apart and next to one another: the same bits, and
    in no more than three times the time."""
    n, page, D, scale = 20000, 16, 128, 128 ** -0.5
    pager, q3, kp, vp, table3, lens3 = _case([n] * 3, hq, hk, D, page, B)
    want = jfa.paged_decode(pager, q3, kp, vp, table3, lens3, scale)
    ref, ref_lse, off, off_lse = paged_ref.decode(q3, kp, vp, table3, lens3, scale)
    assert ((want[0].cpu().double() - ref).abs() <= off).all()
    assert ((want[1].cpu().double() - ref_lse).abs() <= off_lse).all()
    big = jfa.Pager(max_seqs=B, max_pages=pager.max_pages, num_pages=pager.num_pages, page_size=page, H=hq, Hkv=hk, D=D)
    took, q = {}, _draw((B, hq, D), 1)
    for where in ([0, B // 2, B - 1], [0, 1, 2], [B - 3, B - 2, B - 1]):
        table, lens = torch.full((B, pager.max_pages), -1, dtype=I32, device="cuda"), _ints(np.zeros(B))
        table[where], lens[where], q[where] = table3, lens3, q3
        out, lse = jfa.paged_decode(big, q, kp, vp, table, lens, scale)
        assert big.status() == 0
        assert torch.equal(out[where], want[0]) and torch.equal(lse[:, where], want[1])
        none = lens == 0
        assert not out[none].any() and (lse[:, none] == -np.inf).all()
        took[where[1]] = _us(lambda: jfa.paged_decode(big, q, kp, vp, table, lens, scale))
    assert took[B // 2] <= 3 * took[1], took


def test_decode_refuses_an_output_over_its_queries():
    """q in place, by a part of it, and by the gaps between strided rows; next to it is fine."""
    pager, q, kp, vp, table, lens = _case([40, 300, 7], 4, 2, 64, 16, 5)
    want = jfa.paged_decode(pager, q, kp, vp, table, lens, 0.1)
    buf = torch.zeros((9, 4, 64), dtype=BF16, device="cuda")
    buf[3:6] = q
    was = buf.clone()
    for at in (3, 1, 2, 4, 5):
        with pytest.raises(jfa.JfaError) as e:
            jfa.paged_decode(pager, buf[3:6], kp, vp, table, lens, 0.1, out=buf[at:at + 3])
        assert e.value.code == 1
    wide = torch.zeros((3, 9, 4, 64), dtype=BF16, device="cuda")
    with pytest.raises(jfa.JfaError):
        jfa.paged_decode(pager, wide[:, 2], kp, vp, table, lens, 0.1, out=wide[0, 4:7])
    assert torch.equal(buf, was)
    for at in (0, 6):
        out, lse = jfa.paged_decode(pager, buf[3:6], kp, vp, table, lens, 0.1, out=buf[at:at + 3])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_decode_with_the_largest_scales():
    """Scales from 2^127 on, which times log2 e may be infinite, are refused; below they count."""
    pager, q, kp, vp, table, lens = _case([40, 1], 2, 1, 64, 16, 6)
    for scale in (2.0 ** 127, -3.4e38, 3e38, float("inf"), float("nan")):
        with pytest.raises(jfa.JfaError) as e:
            jfa.paged_decode(pager, q, kp, vp, table, lens, scale)
        assert e.value.code == 1
    zero = torch.zeros_like(q)  # all scores 0, whatever the scale
    want = jfa.paged_decode(pager, zero, kp, vp, table, lens, 1.0)
    for scale in (1.7e38, -1.7e38, 1e-45, 0.0):
        got = jfa.paged_decode(pager, zero, kp, vp, table, lens, scale)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_step_without_requests_is_refused_and_one_without_rows_is_not():
    pager, q, kp, vp, table, lens = _case([40, 1], 2, 1, 64, 16, 6)
    free = _ints(np.arange(pager.num_pages))
    with pytest.raises(jfa.JfaError) as e:
        jfa.paged_decode(pager, q[:0], kp, vp, table[:0], lens[:0], 0.1)
    assert e.value.code == 1
    with pytest.raises(jfa.JfaError) as e:
        jfa.paged_tables(pager, lens[:0], lens[:0], table[:0], free, _ints([0]), rows=4)
    assert e.value.code == 1
    got = jfa.paged_tables(pager, lens, torch.zeros_like(lens), table, free, _ints([0]), rows=0)
    assert torch.equal(got[0], lens) and got[4].tolist() == [0, 0, 0] and got[2].numel() == 0
    assert jfa.paged_append(pager, kp[0, :0], vp[0, :0], lens[:0], kp, vp) is None
    assert pager.status() == 0


def _check(case, scale):
    """One call against the 64-bit form, within its bounds; twice, with the same bits."""
    pager, q, kp, vp, table, lens = case
    out, lse = jfa.paged_decode(pager, q, kp, vp, table, lens, scale)
    again = jfa.paged_decode(pager, q, kp, vp, table, lens, scale)
    assert pager.status() == 0 and torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ref, ref_lse, off, off_lse = paged_ref.decode(q, kp, vp, table, lens, scale)
    assert ((out.cpu().double() - ref).abs() <= off).all()
    l, some = lse.cpu().double(), torch.isfinite(ref_lse)
    assert torch.equal(torch.isfinite(l), some) and ((l - ref_lse).abs()[some] <= off_lse[some]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,hq,hk", [
    ([180, 33, 64, 1, 0, 192], 17, 1), ([180, 33, 64, 1, 0, 192], 34, 2), ([1, 96, 0, 17, 32], 40, 1),
    ([1, 30, 0, 17, 32], 100, 1), ([1, 30, 0, 17, 32], 130, 1), ([7], 300, 1), ([32] * 20, 260, 2)])
def test_decode_short_rows_with_parts_side_by_side(D, lens, hq, hk):
    """A CTA for each row, whose query heads several warps hold, also in two and three passes."""
    _check(_case(lens, hq, hk, D, 16, hq), D ** -0.5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq", [130, 300])
def test_decode_rows_of_many_parts_in_passes(D, hq):
    """Parts joined in groups first, of more query heads than one pass takes."""
    _check(_case([20000, 0, 7000, 9001], hq, 1, D, 24, hq), D ** -0.5)


@pytest.mark.parametrize("B,hq,hk", [(33, 130, 1), (257, 40, 1), (257, 34, 2), (513, 17, 1)])
@pytest.mark.parametrize("most", [60, 400])
def test_decode_many_requests_with_parts_side_by_side(B, hq, hk, most):
    """More requests than a warp has lanes, and than a CTA has threads, some of them empty."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, most, B)
    lens[rng.random(B) < 0.2] = 0
    _check(_case(lens, hq, hk, 64, 16, B), 0.125)


@pytest.mark.parametrize("hq,hk,D", [(1, 1, 64), (8, 2, 128), (20, 1, 64)])
def test_decode_lse_of_rows_of_one_tile(hq, hk, D):
    """Log-sum-exp sums the weights in fp32.  q and k are small whole numbers, so that
    scores are exact but for the scale: of up to 32 rows in one tile, with S the largest
    |score|, in steps of 2^-24: a score times scale log2 e is off by three roundings, 3 S,
    less the maximum by one of at most 2 S; its exponential by 4 (ex2.approx: 2^-22), the
    sum of n by n; log2 by 4 (of itself, or absolute below 2), the maximum added to it and
    the factor ln 2 by three roundings of the result."""
    B = 400
    lens = np.random.default_rng(1).integers(1, 33, B)
    lens[:120] = np.arange(120) % 6 + 1
    pager, q, kp, vp, table, dl = _case(lens, hq, hk, D, 16, 4)
    q.copy_((q.float() * 1.5).round())
    kp.copy_((kp.float() * 1.5).round())
    scale = 2.0 ** -4
    _, lse = jfa.paged_decode(pager, q, kp, vp, table, dl, scale)
    worst = 0.0
    for b in range(B):
        n, t = int(lens[b]), torch.arange(int(lens[b]), device="cuda")
        k = kp[table[b, t // 16].long(), t % 16].double().repeat_interleave(hq // hk, 1)  # [n, hq, D]
        s = scale * torch.einsum("hd,thd->ht", q[b].double(), k)
        ref = torch.logsumexp(s, 1)
        log2 = (ref - s.amax(1)).clamp(min=0) / np.log(2)
        steps = 5 * s.abs().amax(1) + 4 + n + 4 * log2.clamp(min=1) * np.log(2) + 3 * ref.abs()
        worst = max(worst, float(((lse[:, b].double() - ref).abs() / (1.01 * steps * 2.0 ** -24)).max()))
    assert worst <= 1, worst
