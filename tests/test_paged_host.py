"""Host side of the paged-cache operators (no GPU): refusals before any launch,
and the plain form of the block tables that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import jagged_attention_gb300 as jfa
from tests import paged_ref

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    jfa.build()


@pytest.mark.parametrize("change,code", [
    (dict(max_seqs=0), INVALID), (dict(max_seqs=16385), UNSUPPORTED), (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID), (dict(H=3), INVALID),
    (dict(H=1), INVALID), (dict(D=96), UNSUPPORTED), (dict(H=2 * 40000), UNSUPPORTED),
    (dict(max_pages=2**31 - 1), UNSUPPORTED), (dict(num_pages=2**27), UNSUPPORTED),
    (dict(num_pages=2**40), UNSUPPORTED), (dict(max_pages=2**27 - 1), UNSUPPORTED)])
def test_create_refuses(change, code):
    a = dict(max_seqs=8, max_pages=4, num_pages=100, page_size=16, H=4, Hkv=2, D=128)
    a.update(change)
    h = ctypes.c_void_p()
    rc = jfa.lib().jfa_pager_create(a["max_seqs"], a["max_pages"], a["num_pages"], a["page_size"], a["H"], a["Hkv"],
                                    a["D"], 4096, 1 << 30, None, ctypes.byref(h))
    assert rc == code and h.value is None


def test_null_handles_are_refused():
    L = jfa.lib()
    assert L.jfa_pager_destroy(None) == INVALID
    assert L.jfa_pager_status(None, None, None) == INVALID
    assert L.jfa_paged_tables(None, 1, *[None] * 4, 1, None, None, None, 0, None, None, None, None) == INVALID
    assert L.jfa_paged_append(None, 1, None, 0, None, 0, None, None, None, None, 0, 0, None, 0, None, 0,
                              None) == INVALID
    assert L.jfa_paged_decode(None, 1, None, 0, None, None, 0, None, 1.0, None, None, None) == INVALID


def test_status_bits_match_the_header():
    import re
    bits = {m[0]: int(m[1]) for m in re.findall(r"#define JFA_PAGER_(\w+) +(\d+) +/\* status", jfa.HEADER.read_text())}
    assert bits == {"NO_PAGES": jfa.PAGER_NO_PAGES, "BAD_LENGTH": jfa.PAGER_BAD_LENGTH,
                    "BAD_PAGE": jfa.PAGER_BAD_PAGE}
    assert (paged_ref.NO_PAGES, paged_ref.BAD_LENGTH, paged_ref.BAD_PAGE) == (
        jfa.PAGER_NO_PAGES, jfa.PAGER_BAD_LENGTH, jfa.PAGER_BAD_PAGE)


def test_reference_tables_by_hand():
    """Page size 4: request 0 grows from 3 to 6 rows, 1 ends (pages 7, 8 go back), 2 starts with 5 rows."""
    table = np.array([[5, -9, -9], [7, 8, -9], [-9, -9, -9]])
    free = np.array([1, 2, 3, 0, 0, 0, 0, 0, 0, 0])
    lens, n_free, slots, pos, off, t, f, status = paged_ref.tables(
        np.array([3, 6, 0]), np.array([3, -6, 5]), table, free, 3, 9, 4, 10)
    assert status == 0 and lens.tolist() == [6, 0, 5] and off.tolist() == [0, 3, 3, 8]
    assert f[:5].tolist() == [1, 2, 3, 7, 8] and n_free == 2
    assert t.tolist() == [[5, 8, -9], [7, 8, -9], [7, 3, -9]]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 0]
    assert slots.tolist() == [23, 32, 33, 28, 29, 30, 31, 12, -1]


@pytest.mark.parametrize("seed", range(4))
def test_reference_tables_never_share_a_page(seed):
    rng = np.random.default_rng(seed)
    B, width, page, num_pages = 7, 6, int(rng.integers(1, 9)), 25
    lens, table = np.zeros(B, np.int64), np.full((B, width), -1)
    free, n_free = rng.permutation(num_pages), num_pages
    for _ in range(60):
        delta = np.where(rng.random(B) < 0.3, -rng.integers(0, lens + 1), rng.integers(0, 2 * page + 2, B))
        lens, n_free, slots, *_, table, free, status = paged_ref.tables(
            lens, delta, table, free, n_free, int(np.maximum(delta, 0).sum()) + 2, page, num_pages)
        owned = [p for b in range(B) for p in table[b, :-(-lens[b] // page)]]
        assert sorted(owned + free[:n_free].tolist()) == list(range(num_pages))
        live = slots[slots >= 0]
        assert len(set(live.tolist())) == len(live)
