"""Host side of the cache in 8 or 4 bits (no GPU): refusals before any launch, and the
plain form of the codes that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import coded_ref

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def test_flags_match_the_header():
    import re
    flags = {m[0]: int(m[1]) for m in re.findall(r"#define JFA_PAGER_(\w+) (\d+)u", jfa.HEADER.read_text())}
    assert flags == {"8BIT": jfa.PAGER_8BIT, "4BIT": jfa.PAGER_4BIT}


@pytest.mark.parametrize("flags,change,code", [
    (3, {}, INVALID), (4, {}, INVALID), (1, dict(D=96), UNSUPPORTED), (2, dict(H=3), INVALID),
    (2, dict(max_seqs=16385), UNSUPPORTED), (1, dict(num_pages=0), INVALID)])
def test_create_refuses(flags, change, code):
    a = dict(max_seqs=8, max_pages=4, num_pages=100, page_size=16, H=4, Hkv=2, D=128)
    a.update(change)
    h = ctypes.c_void_p()
    rc = jfa.lib().jfa_pager_create_ex(*(a[x] for x in ("max_seqs", "max_pages", "num_pages", "page_size", "H", "Hkv", "D")),
                                       flags, 4096, 1 << 30, None, ctypes.byref(h))
    assert rc == code and h.value is None


def test_null_handles_are_refused():
    L = jfa.lib()
    assert L.jfa_paged_append_ex(None, 1, None, 0, None, 0, None, None, None, None, None, 0, 0, None, 0, None, 0,
                                 None) == INVALID
    assert L.jfa_paged_gather(None, 1, None, None, None, 0, None, None, 0, None, 0, None, 0, None) == INVALID
    assert L.jfa_paged_decode_ex(None, 1, None, 0, None, None, None, 0, None, 1.0, None, None, None) == INVALID


def test_reference_tables_are_those_of_the_formats():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), coded_ref.E4M3)
    assert np.array_equal((torch.arange(248, dtype=torch.int16) << 7).view(torch.float16).double().numpy(), coded_ref.SCALES)


@pytest.mark.parametrize("bits", [8, 4])
def test_reference_codes_are_the_nearest(bits):
    """No other code is nearer; values of codes are their own; zeros, and what is not finite."""
    g = torch.Generator().manual_seed(bits)
    x = (torch.randn((50, 64), generator=g) * torch.exp(3 * torch.randn((50, 1), generator=g))).to(torch.bfloat16)
    x[3] = 0
    codes, scales = coded_ref.quantise(x, bits)
    v = coded_ref.values(codes, scales, bits)
    again = coded_ref.quantise(v, bits)
    assert np.array_equal(coded_ref.values(*again, bits), v)  # (4 bits: a scale may become another one of the same values)
    assert not v[3].any()
    if bits == 8:
        unit = torch.from_numpy(2.0 ** (scales.astype(float) - 127))
        grid = torch.from_numpy(np.concatenate((-coded_ref.E4M3, coded_ref.E4M3)))
        best = (x.double()[..., None] / unit[..., None] - grid).abs().amin(-1) * unit
        assert (x.double().abs().amax(-1) > 224 * unit[:, 0])[unit[:, 0] > 2.0 ** -48].all()  # no smaller power fits
    else:
        unit = torch.from_numpy(np.repeat(coded_ref.SCALES[scales], 16, -1))
        grid = torch.from_numpy(np.concatenate((-coded_ref.E2M1, coded_ref.E2M1)))
        best = (x.double()[..., None] - unit[..., None] * grid).abs().amin(-1)
    assert torch.equal((v - x.double()).abs(), best)
    for bad in (np.nan, np.inf, -np.inf):
        x[7, 20] = bad
        v = coded_ref.values(*coded_ref.quantise(x, bits), bits)
        assert torch.isnan(v[7, 16:32]).all() and torch.isnan(v[7]).sum() == (64 if bits == 8 else 16)
        assert torch.isfinite(v[8]).all()


def test_reference_codes_by_hand():
    """8 bits: 449 takes the next power; halves to even.  4 bits: largest 12 takes scale 2."""
    x = torch.zeros(1, 16)
    x[0, :5] = torch.tensor([448.0, 17.0, 19.0, -1.0, 2.0 ** -10])
    codes, c = coded_ref.quantise(x, 8)
    assert c[0, 0] == 127 and coded_ref.values(codes, c, 8)[0, :5].tolist() == [448.0, 16.0, 20.0, -1.0, 0.0]
    x[0, 0] = 450.0
    assert coded_ref.quantise(x, 8)[1][0, 0] == 128
    x[0, :8] = torch.tensor([12.0, 0.5, 1.5, 2.5, 3.5, 5.0, 7.0, -10.0])
    codes, s = coded_ref.quantise(x, 4)
    assert coded_ref.SCALES[s[0, 0]] == 2
    assert coded_ref.values(codes, s, 4)[0, :8].tolist() == [12.0, 0.0, 2.0, 2.0, 4.0, 4.0, 8.0, -8.0]
    assert codes[0, 0] == 7 | 0 << 4 and codes[0, 1] == 2 | 2 << 4
