"""GPU tests of the rotary operator against its 64-bit plain form, within
bounds derived in paged_ref.rotate_bound."""
import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
import workloads
from tests import paged_ref, parity

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _draw(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(dtype)


def _check(got, x, pos, freq, axis, interleaved, inverse):
    ref = paged_ref.rotate(x, pos, freq, axis, interleaved, inverse)
    bound = paged_ref.rotate_bound(x, ref, len(freq), interleaved, x.dtype)
    err = (got.detach().cpu().double() - ref).abs()
    assert torch.isfinite(got).all() and (err <= bound).all(), float((err - bound).max())


def _axes(half, n):
    return np.sort(np.arange(half) % n).astype(np.int32)


# D, rotary width, axes, rows, heads of q, heads of k
SHAPES = [(128, 128, 3, 1, 1, 0), (128, 128, 1, 33, 4, 4), (128, 96, 2, 257, 3, 1), (64, 64, 4, 100, 5, 2),
          (64, 16, 1, 7, 32, 8), (128, 16, 3, 1000, 2, 0), (64, 48, 2, 4099, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse,types", [(False, (BF16, BF16)), (True, (F32, BF16)), (True, (BF16, F32))])
def test_rotate(shape, interleaved, inverse, types):
    D, R, axes, rows, hq, hk = shape
    freq, _ = jfa.rotary_pairs(R)
    axis = _axes(R // 2, axes)
    rot = jfa.Rotary(freq, axis, D=D, interleaved=interleaved)
    g = torch.Generator(device="cuda").manual_seed(rows)
    pos = torch.randint(-5, 100000, (rows, axes), generator=g, device="cuda").to(torch.int32)
    pos[0] = 2**31 - 1
    pos[-1, 0] = -2**31
    q = _draw((rows, hq, D), types[0], 1)
    gq = parity.guarded(q.shape, types[0])
    if not hk:
        assert jfa.rotate(rot, pos, q, inverse=inverse, q_out=gq.t) is gq.t
        gq.check("q")
        return _check(gq.t, q, pos, freq, axis, interleaved, inverse)
    k = _draw((rows, hk, D), types[1], 2)
    gk = parity.guarded(k.shape, types[1])
    jfa.rotate(rot, pos, q, k, inverse=inverse, q_out=gq.t, k_out=gk.t)
    gq.check("q")
    gk.check("k")
    _check(gq.t, q, pos, freq, axis, interleaved, inverse)
    _check(gk.t, k, pos, freq, axis, interleaved, inverse)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_and_one_position_for_all_axes(interleaved):
    """q and k as slices of a fused projection, turned where they lie; v stays."""
    rows, hq, hk, D = 131, 4, 2, 128
    freq, axis = jfa.rotary_pairs(D, (16, 24, 24))
    rot = jfa.Rotary(freq, axis, D=D, interleaved=interleaved)
    x = _draw((rows, hq + 2 * hk, D), BF16, 3)
    was = x.clone()
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) * 37
    q, k = x[:, :hq], x[:, hq:hq + hk]
    jfa.rotate(rot, pos, q, k, q_out=q, k_out=k)
    _check(q, was[:, :hq], pos, freq, axis, interleaved, False)
    _check(k, was[:, hq:hq + hk], pos, freq, axis, interleaved, False)
    assert torch.equal(x[:, hq + hk:], was[:, hq + hk:])
    # positions laid out axis by axis, and a row of padding between the rows
    wide = torch.randint(0, 5000, (3, rows), device="cuda", dtype=torch.int32)
    out = torch.full((rows, hq + 1, D), 7.0, dtype=BF16, device="cuda")
    jfa.rotate(rot, wide.T, was[:, :hq], q_out=out[:, :hq])
    _check(out[:, :hq], was[:, :hq], wide.T, freq, axis, interleaved, False)
    assert (out[:, hq:] == 7.0).all()


def test_position_zero_and_copied_values_are_exact():
    rot = jfa.Rotary(*jfa.rotary_pairs(32), D=128)
    x = _draw((50, 3, 128), BF16, 4)
    assert torch.equal(jfa.rotate(rot, torch.zeros(50, dtype=torch.int32, device="cuda"), x), x)
    y = jfa.rotate(rot, torch.full((50,), 12345, dtype=torch.int32, device="cuda"), x)
    assert torch.equal(y[:, :, 32:], x[:, :, 32:]) and not torch.equal(y[:, :, :32], x[:, :, :32])


def test_no_rows():
    rot = jfa.Rotary(*jfa.rotary_pairs(64), D=64)
    q, k = (torch.empty((0, h, 64), dtype=BF16, device="cuda") for h in (4, 2))
    a, b = jfa.rotate(rot, torch.empty((0,), dtype=torch.int32, device="cuda"), q, k)
    assert a.shape == q.shape and b.shape == k.shape


def test_offsets_past_32_bits():
    """The last rows of a tensor of more than 2^31 values."""
    rows, heads, D = (1 << 21) + 37, 8, 128
    freq, axis = jfa.rotary_pairs(D)
    rot = jfa.Rotary(freq, axis, D=D)
    x = torch.zeros((rows, heads, D), dtype=BF16, device="cuda")
    tail = _draw((50, heads, D), BF16, 5)
    x[-50:] = tail
    pos = torch.arange(rows, device="cuda", dtype=torch.int32)
    y = jfa.rotate(rot, pos, x, q_out=x)
    _check(y[-50:], tail, pos[-50:], freq, axis, False, False)
    assert not x[:-50].any()


def test_another_stream_and_a_captured_graph():
    freq, axis = jfa.rotary_pairs(128)
    rot = jfa.Rotary(freq, axis, D=128)
    x, pos = _draw((77, 4, 128), BF16, 6), torch.arange(77, device="cuda", dtype=torch.int32)
    want = jfa.rotate(rot, pos, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    with torch.cuda.stream(side):
        jfa.rotate(rot, pos, x, q_out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jfa.rotate(rot, pos, x, q_out=out)
    out.zero_()
    rot.close()  # the graph holds what it needs
    for shift in (0, 1000):
        pos += shift
        graph.replay()
        torch.cuda.synchronize()
        _check(out, x, pos, freq, axis, False, False)


def test_refusals_of_the_binding():
    rot = jfa.Rotary(*jfa.rotary_pairs(128, (32, 32)), D=128)
    q = _draw((10, 2, 128), BF16, 7)
    pos = torch.zeros((10, 2), dtype=torch.int32, device="cuda")
    for bad in (pos.long(), pos.cpu()):
        with pytest.raises(TypeError):
            jfa.rotate(rot, bad, q)
    for bad in (pos[:9], pos[:, :1], torch.zeros(9, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            jfa.rotate(rot, bad, q)
    with pytest.raises(TypeError):
        jfa.rotate(rot, pos, q.half())
    with pytest.raises(TypeError):
        jfa.rotate(rot, pos, q, q_out=torch.empty_like(q, dtype=F32))
    with pytest.raises(ValueError):
        jfa.rotate(rot, pos, q, q[:5])
    with pytest.raises(ValueError):
        jfa.rotate(rot, pos, q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError):
        jfa.rotate(rot, pos, q, k_out=q)
    with pytest.raises(jfa.JfaError):  # one row repeated by a stride of 0
        jfa.rotate(rot, pos, q[:1].expand(10, 2, 128))


@pytest.mark.parametrize("mode", ["self", "broadcast"])
def test_training_step_with_positions(mode):
    """rotate, forward, backward, rotate back: gradients of the unrotated q, k and
    of v against autograd in 64 bits through the whole composition, at the
    relative L2 error the backward is held to."""
    H, D = 2, 128
    freq, axis = jfa.rotary_pairs(D, (16, 24, 24))
    rot = jfa.Rotary(freq, axis, D=D)
    p = parity.to_cuda(workloads.make_problem(4, H, D, mode, [70, 1, 200, 33], Lq=40, seed=11))
    g = torch.Generator(device="cuda").manual_seed(1)
    pos_k = torch.randint(0, 3000, (p.k.shape[0], 3), generator=g, device="cuda").to(torch.int32)
    pos_q = pos_k if mode == "self" else torch.randint(0, 3000, (40, 3), generator=g, device="cuda").to(torch.int32)
    rq, rk = jfa.rotate(rot, pos_q, p.q), jfa.rotate(rot, pos_k, p.k)
    plan = jfa.Plan(p.kv_offsets, p.q_offsets, H=H, D=D, Lq=p.Lq)
    out, lse = jfa.fwd(plan, rq, rk, p.v, p.scale)
    dq, dk, dv = jfa.bwd(plan, rq, rk, p.v, out, p.dout, lse, p.scale)
    dq = jfa.rotate(rot, pos_q, dq, inverse=True, q_out=dq)
    dk = jfa.rotate(rot, pos_k, dk, inverse=True)

    leaves = [t.cpu().double().requires_grad_(True) for t in (p.q, p.k, p.v)]

    def turn(x, pos):
        angle = pos.cpu().double()[:, axis] * torch.from_numpy(freq)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    tq, tk, total = turn(leaves[0], pos_q), turn(leaves[1], pos_k), 0.0
    for b in range(p.B):
        lo, hi = int(p.kv_offsets[b]), int(p.kv_offsets[b + 1])
        qb = tq if mode == "broadcast" else tq[lo:hi]
        do = p.dout[b * 40:(b + 1) * 40] if mode == "broadcast" else p.dout[lo:hi]
        s = torch.einsum("qhd,khd->hqk", qb, tk[lo:hi]) * p.scale
        o = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), leaves[2][lo:hi])
        total = total + (o * do.cpu().double()).sum()
    total.backward()
    for name, got, leaf in (("dq", dq, leaves[0]), ("dk", dk, leaves[1]), ("dv", dv, leaves[2])):
        assert parity.rel_l2(got, leaf.grad) <= parity.TOL_GRAD, name
