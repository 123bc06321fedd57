"""Waits with a time limit that depend on the kernel before: a warp takes them only after it has
waited for that kernel itself, whose time would count else. The down kernel of the 4-bit floating point layer
starts beside the up kernel; its warps are stepped through here by the conditions in the source."""
import os
import re

import pytest

from int4_weight_quantized_w4_gb300 import _build


def role(name):
    with open(os.path.join(_build.CSRC, "moe_decode_fp4.cu")) as f:
        text = re.sub(r"//.*", "", f.read())
    at = text.index(f"void {name}(")
    return text[at:text.index("\n}\n", at)]


def conditions(text):
    """When a role waits for the kernel before, of the waits that stand in this part of it."""
    return [c.replace("||", " or ").replace("&&", " and ") for c in re.findall(r"if \(!waited && (.*)\) \{", text)]


@pytest.mark.parametrize("words", [2, 4])
@pytest.mark.parametrize("tma", [True, False])
@pytest.mark.parametrize("stages", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("KS", [1, 2, 3, 4, 5, 6, 7, 8])
def test_the_turning_warp_waits_first(words, tma, stages, KS):
    every, raws, tiles = 8 // words, 2, 24
    # slots of scales that the copying warp fills before it has waited
    late = conditions(role("load_scales"))
    assert len(late) == 1
    early, rs, rph = 0, 0, 1
    while not eval(late[0], {"rph": rph}):
        early += 1
        rs += 1
        if rs == raws:
            rs, rph = 0, rph ^ 1
    turn = role("turn_scales")
    first = conditions(turn[:turn.index("wait_warp(&bar.raw_full")])
    st, ph, rs, rph, taken, waited = 0, 1, 0, 0, 0, False
    for _ in range(tiles):
        for ks in range(KS):
            waited = waited or any(eval(c, {"ph": ph, "rph": rph}) for c in first)
            if ks == 0 or (tma and ks % every == 0):
                assert waited or taken < early, "waits for a copy that starts only after the kernel before"
                taken += 1
            waited = waited or ph == 0      # at the latest before a stage that is emptied only then
            if ks == KS - 1 or (tma and ks % every == every - 1):
                rs += 1
                if rs == raws:
                    rs, rph = 0, rph ^ 1
            st += 1
            if st == stages:
                st, ph = 0, ph ^ 1
