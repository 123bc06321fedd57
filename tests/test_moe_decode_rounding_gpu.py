"""The few-token expert layer rounds once: its outputs are the bf16 numbers next to the exact ones,
but where these lie so near a border that fp32 sums may cross it.

x is exact, activations in between keep 22 bits and sums are fp32, in chains of some 32
additions a warp: an output is off by some 2^-19 of a typical one before it is rounded. Borders lie 2^-8 to
2^-7 of a number apart, so that one number in 2^10 of typical size, and of numbers of all sizes one in two hundred at most,
is within that of one. (With activations of 11 bits, 2^-13 off on average, it is one in twenty.)"""
import numpy as np
import pytest
import torch

import oracle as O
import synthetic as S
from _gpu import requires_cuda
from test_moe_decode_gpu import Experts, inputs

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.mark.parametrize("fmt", ["int4", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,E,H,I,group", [(1, 8, 2048, 1408, 128), (4, 16, 1024, 704, 64), (5, 4, 512, 320, 32), (8, 24, 1088, 320, 64),
                                           (9, 16, 512, 2112, 64), (16, 6, 512, 320, 64)])
def test_outputs_are_the_nearest_numbers(fmt, T, E, H, I, group):
    ex = Experts(E, H, I, fmt, group)
    xb, logits = inputs(T, H, E, seed=T)
    y = ex.call(xb, logits, 4)
    torch.cuda.synchronize()
    r, _ = O.moe_decode(xb, logits, lambda e: ex.values(0, e), lambda e: ex.values(1, e), 4)
    same = np.asarray(S.to_bf16_bits(r)) == y.cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.mean(~same) <= 1 / 200
