"""The few-token expert layer on rows with one number far above the others: what the others add up
to has to come out as exactly as without it, where the weights make nothing of the large one.

Bounds as in the layer's other tests: the output's rounding to bf16 and 2^-10 of the sum of
magnitudes. x is exact down to 2^-29 of a row's largest number."""
import numpy as np
import pytest

import oracle as O
import synthetic as S
from _gpu import requires_cuda
from test_moe_decode_gpu import Experts

pytestmark = [pytest.mark.gpu, requires_cuda]

FORMATS = ["int4", "mxfp4", "nvfp4"]


def without(parts, column, fmt):
    """The weights of a column become zero."""
    q, s, g = parts
    q = q.copy()
    if fmt == "int4":
        w = q.view(np.uint32)
        at = np.uint32(4 * (column % 8))
        w[..., column // 8] = (w[..., column // 8] & ~(np.uint32(15) << at)) | (np.uint32(8) << at)
    else:
        q[..., column // 2] &= 0x0F if column % 2 else 0xF0
    return q, s, g


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("large", [64.0, 4096.0, 65536.0, 2.0 ** 20])
def test_a_column_that_counts_for_nothing(fmt, T, large):
    H, c = 1024, 133
    ex = Experts(12, H, 320, fmt)
    ex.parts[0] = without(ex.parts[0], c, fmt)
    assert all((ex.values(0, e)[:, c] == 0).all() for e in range(12))
    x = S.normal(1, T, T * H).reshape(T, H)
    x[:, c] = large
    ex.check(S.to_bf16_bits(x), S.router_logits(T, 12, seed=5), 3, scoring="softmax")


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("I", [320, 288 * 2])
def test_power_of_two_scales_at_the_low_end(T, I):
    """Bytes 0 to 4, the first of which is not a normal number, on activations of 2^110."""
    ex = Experts(6, 512, I, "mxfp4")
    q, s, g = ex.parts[0]
    ex.parts[0] = q, (s % 5).astype(np.uint8), g
    assert (ex.parts[0][1] == 0).any()
    x = S.normal(7, T, T * 512).reshape(T, 512) * 2.0 ** 110
    ex.check(S.to_bf16_bits(x), S.router_logits(T, 6, seed=5), 2, scoring="softmax")


def test_a_scale_that_is_no_number():
    """Byte 255 in one expert: tokens that choose it get no finite number in that output, others are as they were."""
    ex = Experts(6, 512, 320, "mxfp4")
    xb, logits = S.activations_bf16(4, 512, seed=1), S.router_logits(4, 6, seed=5)
    logits[:, 3] = -30.0
    logits[2, 3] = 30.0
    clean = ex.call(xb, logits, 2).float().cpu().numpy()
    del ex._dev
    q, s, g = ex.parts[1]
    s = s.copy()
    s[3, 200, 5] = 255
    ex.parts[1] = q, s, g
    y = ex.call(xb, logits, 2).float().cpu().numpy()
    assert np.isnan(y[2, 200])
    y[2, 200] = clean[2, 200]
    np.testing.assert_array_equal(y, clean)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 9])
def test_an_activation_that_counts_for_nothing(fmt, T):
    """One gate and up row of far larger weights, and none in that column of the down weights: its
    neighbours lie up to 2^-30 below it, and have an exponent of their own."""
    H, I, c = 512, 320, 77
    ex = Experts(8, H, I, fmt)
    q, s, g = ex.parts[0]
    s = s.copy()
    s[:, [c, I + c]] = {"int4": 8.0, "mxfp4": 118 + 16, "nvfp4": 0x7E}[fmt]          # 2^7, 448
    ex.parts[0] = q, s, g
    ex.parts[1] = without(ex.parts[1], c, fmt)
    x = S.normal(3, T, T * H).reshape(T, H)
    h = ex.values(0, 0) @ x[0]
    assert np.abs(h[[c, I + c]]).min() > 10 * np.median(np.abs(h))
    ex.check(S.to_bf16_bits(x), S.router_logits(T, 8, seed=5), 3, scoring="softmax")


@pytest.mark.parametrize("T", [6, 16])
def test_an_activation_past_the_largest_number(T):
    """It is infinite in fp32, and so are the outputs that it counts for, with their sign; the others of the same token are none
    the worse."""
    H, I, c, E = 512, 320, 77, 2
    ex = Experts(E, H, I, "mxfp4")
    q, s, g = ex.parts[0]
    s = s.copy()
    s[:, [c, I + c]] = 127 + 60
    ex.parts[0] = q, s, g
    q, s, g = ex.parts[1]
    q = q.copy()
    q[:, :100, c // 2] = 0x55          # 3 in the first 100 rows
    q[:, 100:, c // 2] = 0xDD          # -3 in the others
    ex.parts[1] = q, s, g
    xb, logits = S.activations_bf16(T, H, seed=2), S.router_logits(T, E, seed=5)
    logits[:, 0], logits[:, 1] = 5.0, -5.0
    y = ex.call(xb, logits, 1).float().cpu().numpy()
    h = O.bf16_to_f64(xb) @ ex.values(0, 0).T
    with np.errstate(over="ignore"):
        a = h[:, c] / (1 + np.exp(-h[:, c])) * h[:, I + c]
    large, small = np.abs(a) > 4e38, np.abs(a) < 3e38      # fp32 ends at 3.4e38
    assert large.any() and small.any()
    for t in range(T):
        if large[t]:
            assert (y[t, :100] == np.sign(a[t]) * np.inf).all() and (y[t, 100:] == -np.sign(a[t]) * np.inf).all()
        elif small[t]:
            assert np.isfinite(y[t]).all()
