"""GPU tests of gather at its edges: no rows at all."""
import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("offsets,status", [([0, 0, 0], 0), ([0, 5, 5], jfa.PAGER_BAD_LENGTH), ([0, 0, 1], jfa.PAGER_BAD_LENGTH),
                                            ([-7, -3, 0], 0), ([-9, -8, -1], 0), ([3, 3, 2**31 - 1], jfa.PAGER_BAD_LENGTH)])
@pytest.mark.parametrize("captured", [False, True])
def test_no_rows(bits, offsets, status, captured):
    """Offsets beyond no rows say so, as they do beyond some; nothing is written."""
    pager = jfa.Pager(max_seqs=2, max_pages=3, num_pages=6, page_size=8, H=4, Hkv=2, D=64, bits=bits)
    k, v, ks, vs = pager.pages()
    held = {} if bits == 16 else dict(k_scales=ks, v_scales=vs)
    table, at = _ints([[0, 1, 2], [3, 4, 5]]), _ints(offsets)
    around = torch.full((2, 4, 2, 64), 7.0, dtype=BF16, device="cuda")
    outs = around[0, 1:1], around[1, 1:1]

    def call():
        return jfa.paged_gather(pager, k, v, table, at, rows=0, **held, k_out=outs[0], v_out=outs[1])

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        assert pager.status() == 0
        graph.replay()
    else:
        got = call()
        assert got[0].shape == (0, 2, 64)
    assert pager.status() == status and pager.status() == 0 and (around == 7.0).all()
    jfa.paged_gather(pager, k, v, table, at, rows=0, **held)
    assert pager.status() == status
