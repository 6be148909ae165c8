"""GPU tests of a pager's block: as many bytes as its calls use, whatever its number of bits."""
import ctypes

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa

pytestmark = pytest.mark.gpu
BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
FLAGS = {16: 0, 8: jfa.PAGER_8BIT, 4: jfa.PAGER_4BIT}


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(8, 8), (64, 8), (16, 1), (48, 2), (64, 1), (128, 1), (300, 1)])
def test_bytes_of_a_bf16_pager(D, hq, hk):
    """Status word, three counters a CTA, and for each CTA two places for each part of a group: maximum, sum and D values of its heads."""
    group, together = hq // hk, 1
    while together < 8 and together * 16 < group:
        together *= 2
    passes = -(-group // (16 * together))
    heads = 8 if -(-group // (passes * together)) <= 8 else 16
    ctas = torch.cuda.get_device_properties(0).multi_processor_count * (2 if D == 64 else 1)
    places = 2 * ctas * together * heads
    want = _up(_up(_up(256 + 3 * ctas * 4) + places * 2 * 4) + places * D * 4)
    L = jfa.lib()
    assert L.jfa_pager_block_bytes_ex(hq, hk, D, 0) == want
    assert jfa.Pager(max_seqs=1, max_pages=1, num_pages=1, page_size=1, H=hq, Hkv=hk, D=D).block.numel() == want
    sizes = [L.jfa_pager_block_bytes_ex(hq, hk, D, f) for f in FLAGS.values()]
    assert L.jfa_pager_block_bytes(hq, hk, D) == max(sizes) and min(sizes) > 0
    for bad in (3, 4, 1 << 31):
        assert L.jfa_pager_block_bytes_ex(hq, hk, D, bad) == 0


def _tight(bits, spare=0, **sizes):
    """(pager whose block has just its bytes, less `spare`, those behind it)."""
    pager = jfa.Pager(**sizes, bits=bits)
    n = jfa.lib().jfa_pager_block_bytes_ex(sizes["H"], sizes["Hkv"], sizes["D"], FLAGS[bits])
    whole = torch.full((n + 65536,), 0xA5, dtype=U8, device="cuda")
    handle = ctypes.c_void_p()
    order = ("max_seqs", "max_pages", "num_pages", "page_size", "H", "Hkv", "D")
    rc = jfa.lib().jfa_pager_create_ex(*(sizes[x] for x in order), FLAGS[bits], whole.data_ptr(), n - spare,
                                       torch.cuda.current_stream().cuda_stream, ctypes.byref(handle))
    if rc:
        return rc
    torch.cuda.synchronize()
    jfa.lib().jfa_pager_destroy(pager.handle)
    pager._h, pager.block = handle, whole
    return pager, whole[n:]


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_a_smaller_block_is_refused(bits):
    sizes = dict(max_seqs=1, max_pages=1, num_pages=1, page_size=1, H=8, Hkv=2, D=128)
    assert _tight(bits, spare=1, **sizes) == 5
    assert isinstance(_tight(bits, **sizes), tuple)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 4), (8, 1), (32, 2), (48, 1), (128, 1), (12, 3)])
@pytest.mark.parametrize("mb", [1, 300])
def test_calls_stay_within_the_block(bits, D, hq, hk, mb):
    """Rows cut into as many parts as there are, heads one after the other and side by side."""
    page = 64
    pages = max(8, (mb << 20) // (2 * hk * page * D * bits // 8))
    sizes = dict(max_seqs=3, max_pages=pages, num_pages=pages, page_size=page, H=hq, Hkv=hk, D=D)
    pager, behind = _tight(bits, **sizes)
    plain = jfa.Pager(**sizes, bits=bits)
    k, v, k_scales, v_scales = pager.pages()
    held = {} if bits == 16 else dict(k_scales=k_scales, v_scales=v_scales)
    g = torch.Generator(device="cuda").manual_seed(pages)
    new = torch.randn((page, 2 * hk, D), generator=g, device="cuda").to(BF16)
    jfa.paged_append(pager, new[:, :hk], new[:, hk:], torch.arange(page, dtype=I32, device="cuda"), k, v, **held)
    for t in (k, v, *held.values()):
        t[1:] = t[:1]  # all pages alike
    table = torch.arange(pages, dtype=I32, device="cuda").repeat(3, 1)
    for lens in ([pages * page, 0, 0], [pages * page - 1, 130, 1], [1, 2, 65]):
        q = torch.randn((3, hq, D), generator=g, device="cuda").to(BF16)
        dl = torch.as_tensor(np.asarray(lens), dtype=I32).cuda()
        got = jfa.paged_decode(pager, q, k, v, table, dl, D ** -0.5, **held)
        want = jfa.paged_decode(plain, q, k, v, table, dl, D ** -0.5, **held)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (behind == 0xA5).all() and pager.status() == 0
