"""GPU tests of the rotary operator at the ends of its sizes."""
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import paged_ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


@pytest.mark.parametrize("heads,dtype", [(65535 * 12 + 1, BF16), (65535 * 6 + 7, F32)])
def test_more_heads_than_a_grid_has_rows_for(heads, dtype):
    """Rows of so many heads that one block for each 12 (fp32: 6) would outgrow the grid."""
    D = 64
    freq, axis = jfa.rotary_pairs(D)
    rot = jfa.Rotary(freq, axis, D=D)
    g = torch.Generator(device="cuda").manual_seed(heads)
    x = torch.randn((2, heads, D), generator=g, device="cuda", dtype=F32).to(dtype)
    pos = torch.tensor([3, 70000], device="cuda", dtype=torch.int32)
    y = jfa.rotate(rot, pos, x)
    some = torch.cat([torch.arange(20), torch.arange(heads // 2, heads // 2 + 20), torch.arange(heads - 20, heads)])
    ref = paged_ref.rotate(x[:, some], pos, freq, axis)
    bound = paged_ref.rotate_bound(x[:, some], ref, D // 2, False, dtype)
    assert ((y[:, some].cpu().double() - ref).abs() <= bound).all()
    # every head: the rotation keeps the length of a pair, whatever the head
    a, b = x.double().square(), y.double().square()
    near = 2.0 ** -6 if dtype == BF16 else 2.0 ** -18  # twice the bound on a value, relative to |a| + |b|, and a margin
    pair = (a[..., :D // 2] + a[..., D // 2:], b[..., :D // 2] + b[..., D // 2:])
    assert ((pair[0] - pair[1]).abs() <= 2 * near * pair[0]).all()
