"""Host side of the decode kernel (no GPU): what its source has to say for warps that meet
no barrier."""
import re

import pytest

from jagged_attention_gb300 import buildlib

SOURCE = (buildlib.CSRC / "decode_kernel.cuh").read_text()


def _slots(expression, warp, line):
    """Places in sh.part that an index expression names for a warp, over its lanes and for both of its parts."""
    return {eval(expression, {}, dict(warp=warp, line=line, lane=x, slot=2 * line + x)) for x in range(2)}


@pytest.mark.parametrize("together", [1, 2, 4, 8])
def test_a_warp_clears_the_slots_it_writes_and_no_others(together):
    """Up to 32 requests no barrier stands between a warp that clears and one that writes: a
    slot has one warp for both, whatever number of warps goes side by side."""
    clears = re.findall(r"sh\.part\[([^\]]+)\]\.n = 0", SOURCE)
    writes = re.findall(r"sh\.part\[(\w+)\] = \{", SOURCE)
    assert len(clears) == 1 and writes == ["slot"]
    assert re.search(r"const int slot = 2 \* line \+ \(parked \? 0 : 1\);", SOURCE)
    warps = 8
    assert re.search(r"kWarps = 8;", SOURCE)
    sub_bits = (warps // together).bit_length() - 1
    cleared = []
    for warp in range(warps):
        part, sub = warp & (together - 1), warp // together
        line = (part << sub_bits) + sub
        assert re.search(r"const int line = \(part << sub_bits\) \+ sub;", SOURCE)
        assert _slots(clears[0], warp, line) == _slots("slot", warp, line)
        cleared += _slots(clears[0], warp, line)
    assert sorted(cleared) == list(range(2 * warps))  # every slot is cleared
