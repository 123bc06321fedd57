"""A slot of shared memory that an asynchronous copy fills is given back to it only behind a
proxy fence: the fence stands between the reads of the slot and the arrival that lets the next
copy start. Checked in the kernels' sources, without a GPU."""
import glob
import os
import re

import pytest

from int4_weight_quantized_w4_gb300 import _build

ARRIVAL = re.compile(r"mbar_arrive\(&(?:\w+\.)*(?:raw_)?empty\[")
UNITS = sorted(os.path.basename(f) for f in glob.glob(os.path.join(_build.CSRC, "*.cu*")))


def hand_backs(unit):
    """Lines that give a slot back, each with the statements before it in its block and the blocks around it."""
    with open(os.path.join(_build.CSRC, unit)) as f:
        lines = [re.sub(r"//.*", "", line) for line in f]
    return [(n + 1, "".join(lines[max(0, n - 12):n])) for n, line in enumerate(lines) if ARRIVAL.search(line)]


def test_there_are_such_slots():
    assert {u for u in UNITS if hand_backs(u)} >= {"fp4_gemm.cu", "moe_decode.cuh", "w4a8.cu"}


@pytest.mark.parametrize("unit", UNITS)
def test_a_fence_stands_before_the_hand_back(unit):
    for line, before in hand_backs(unit):
        assert "fence_proxy_async_smem()" in before, f"{unit}:{line}"
        assert not re.search(r"wait_warp\(&\w*\.?(raw_)?full", before.split("fence_proxy_async_smem()")[-1]), f"{unit}:{line}"
