"""Host side of the rotary operator (no GPU): the fixed-point turn fractions
against exact integer arithmetic, and refusals before any launch."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import paged_ref

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _pi(bits=2400):
    one = 1 << bits

    def arctan_inv(x):
        t = s = one // x
        n, sign = 3, -1
        while t:
            t //= x * x
            s += sign * (t // n)
            n, sign = n + 2, -sign
        return s
    return Fraction(4 * (4 * arctan_inv(5) - arctan_inv(239)), one)


def _turn(x: float, pi) -> int:
    """floor(x / (2 pi) 2^64 + 1/2) mod 2^64, away from zero for negative halves."""
    t = abs(Fraction(x)) / (2 * pi) * 2**64
    n = (2 * t.numerator + t.denominator) // (2 * t.denominator)
    return (-n if x < 0 else n) % 2**64


@pytest.mark.parametrize("rotary_dim,base", [(128, 1e4), (64, 5e5), (96, 123.0)])
def test_turn_fractions_of_usual_frequencies(rotary_dim, base):
    pi = _pi(400)
    freq, _ = jfa.rotary_pairs(rotary_dim, base=base)
    assert [int(v) for v in jfa.rotary_turns(freq)] == [_turn(float(f), pi) for f in freq]


def test_turn_fractions_over_the_whole_range():
    pi = _pi()
    rng = np.random.default_rng(3)
    x = np.concatenate([np.ldexp(rng.uniform(1, 2, 400), rng.integers(-140, 31, 400)),
                        [0.0, 1.0, 2.0**30, np.nextafter(2.0**31, 0), 5e-324, 1e-300, 2.0**-64, 0.5]])
    x = np.concatenate([x, -x])
    assert [int(v) for v in jfa.rotary_turns(x)] == [_turn(float(f), pi) for f in x]


def test_fixed_point_angles_of_far_positions():
    """position * turn mod 2^64, the kernel's angle, against exact angles."""
    pi = _pi(400)
    freq, _ = jfa.rotary_pairs(128)
    turns = jfa.rotary_turns(freq)
    for pos in (0, 1, -1, 12345, 2**31 - 1, -2**31):
        for f, t in zip(freq, turns):
            got = Fraction((pos * int(t)) % 2**64, 2**64)
            want = (pos * Fraction(float(f)) / (2 * pi)) % 1
            off = abs(got - want)
            assert min(off, 1 - off) <= Fraction(abs(pos) + 1, 2**65)


def test_rotary_pairs():
    freq, axis = jfa.rotary_pairs(128, (16, 24, 24))
    assert freq.shape == (64,) and axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    assert freq[0] == 1.0 and abs(freq[32] - 1e-2) < 1e-15
    with pytest.raises(ValueError):
        jfa.rotary_pairs(128, (16, 24))
    with pytest.raises(ValueError):
        jfa.Rotary([1.0, 2.0], [0], D=128)


@pytest.mark.parametrize("change,code", [
    (dict(D=96), UNSUPPORTED), (dict(pairs=7), INVALID), (dict(pairs=72), INVALID), (dict(pairs=0), INVALID),
    (dict(axis=4), INVALID), (dict(axis=-1), INVALID), (dict(freq=float("nan")), INVALID),
    (dict(freq=float("inf")), INVALID), (dict(freq=2.0**31), INVALID), (dict(flags=2), INVALID)])
def test_create_refuses(change, code):
    L = jfa.lib()
    pairs = change.get("pairs", 32)
    f = np.ones(80)
    a = np.zeros(80, np.int32)
    f[3] = change.get("freq", 1.0)
    a[5] = change.get("axis", 0)
    h = ctypes.c_void_p()
    rc = L.jfa_rotary_create(f.ctypes.data_as(jfa._f64p), jfa._i32ptr(a), pairs, change.get("D", 128),
                             change.get("flags", 0), ctypes.byref(h))
    assert rc == code and h.value is None


def test_rotate_refuses_before_any_launch():
    """Addresses here are never read: every call is refused on the host."""
    L = jfa.lib()
    r = jfa.Rotary(*jfa.rotary_pairs(64), D=128)
    good = [r.handle, 4096, 1, 0, 10, 0, 4096, 256, 8192, 256, 2, 4096, 256, 8192, 256, 2, None]
    for at, value, code in [(0, None, INVALID), (1, None, INVALID), (1, 4098, ALIGNMENT), (2, -1, INVALID),
                            (3, -1, INVALID), (4, -1, INVALID), (4, 1 << 33, INVALID), (5, 8, INVALID),
                            (6, None, INVALID), (6, 4104, ALIGNMENT), (7, 255, INVALID), (7, 260, ALIGNMENT),
                            (8, None, INVALID), (8, 8200, ALIGNMENT), (9, 128, INVALID), (10, 0, INVALID),
                            (10, 2**31 - 1, INVALID), (11, None, INVALID), (15, 0, INVALID), (15, -1, INVALID),
                            (13, None, INVALID), (14, 260, ALIGNMENT)]:
        args = list(good)
        args[at] = value
        assert L.jfa_rotate(*args) == code, (at, value)
    args = list(good)
    args[4] = 0  # no rows: nothing to do
    assert L.jfa_rotate(*args) == 0
    r.close()
    with pytest.raises(RuntimeError):
        r.handle
    assert L.jfa_rotary_destroy(None) == INVALID


def test_binding_refuses_cpu_tensors():
    r = jfa.Rotary(*jfa.rotary_pairs(64), D=128)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        jfa.rotate(r, torch.zeros(3, dtype=torch.int32), x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_inverse_is_the_gradient(interleaved):
    """The plain form's inverse against differences of its forward."""
    g = torch.Generator().manual_seed(5)
    freq, axis = jfa.rotary_pairs(32, (6, 10))
    x = torch.randn(3, 2, 64, generator=g, dtype=torch.float64)
    up = torch.randn(3, 2, 64, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1000, (3, 2), generator=g)
    grad = paged_ref.rotate(up, pos, freq, axis, interleaved, inverse=True)
    h = 1e-3
    for i in range(0, 64, 5):
        d = torch.zeros_like(x)
        d[1, 1, i] = h
        diff = ((paged_ref.rotate(x + d, pos, freq, axis, interleaved)
                 - paged_ref.rotate(x - d, pos, freq, axis, interleaved)) * up).sum() / (2 * h)
        assert abs(diff - grad[1, 1, i]) < 1e-9
