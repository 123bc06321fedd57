"""Pins of the fp8 block-scaled oracle and the grouped-routing oracle against worked
values, closed forms and PyTorch on the CPU."""
import numpy as np
import torch

import oracle as O
import synthetic as S


def test_block_quant_of_one_block_is_the_per_token_quant():
    x = S.activations_bf16(5, 128, seed=1)
    q, s = O.quant_fp8_per_block(x)
    rq, rs = O.quant_fp8_per_token(x)
    np.testing.assert_array_equal(q, rq)
    np.testing.assert_array_equal(s[:, 0], rs)


def test_block_quant_worked_values():
    """Scales from the blocks' own maxima; a block of zeros has scale 1; the last,
    short block has its own."""
    x = np.zeros((1, 300), np.float32)
    x[0, 0], x[0, 1] = 448.0, -17.0            # scale 1: -17 rounds to -16 (spacing 2, tie to even)
    x[0, 299] = 2.0                            # scale 2 / 448
    q, s = O.quant_fp8_per_block(S.to_bf16_bits(x))
    np.testing.assert_array_equal(s, np.array([[1.0, 1.0, np.float32(2.0) / np.float32(448.0)]], np.float32))
    v = O.e4m3_decode(q)
    assert v[0, 0] == 448 and v[0, 1] == -16 and v[0, 299] == 448 and not v[0, 2:299].any()


def test_block_quant_matches_torch_cast():
    x = S.activations_bf16(40, 512, seed=3, outlier_frac=0.02)
    q, s = O.quant_fp8_per_block(x)
    t = torch.from_numpy(S.bf16_bits_to_f32(x)) / torch.from_numpy(s).repeat_interleave(128, 1)
    np.testing.assert_array_equal(q, t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_block_linear_against_dequantized_matmul():
    M, N, K = 5, 200, 300
    qx, qw = S.fp8_codes((M, K), seed=1), S.fp8_codes((N, K), seed=2)
    sx = S.scales_f16((M, 3), seed=3).astype(np.float32)
    sw = S.scales_f16((2, 3), seed=4).astype(np.float32)
    b = S.bias_bf16(N)
    x = O.e4m3_decode(qx) * np.repeat(sx.astype(np.float64), 128, 1)[:, :K]
    w = O.e4m3_decode(qw) * np.repeat(np.repeat(sw.astype(np.float64), 128, 0), 128, 1)[:N, :K]
    np.testing.assert_allclose(O.fp8_block_linear(qx, sx, qw, sw, b), x @ w.T + O.bf16_to_f64(b), rtol=1e-6, atol=1e-6)


def test_block_linear_closed_form():
    """All codes 1.0: y is the sum over blocks of sx sw times the block's width."""
    one = np.uint8(0x38)
    qx, qw = np.full((1, 144), one), np.full((8, 144), one)
    y = O.fp8_block_linear(qx, np.array([[2.0, 4.0]], np.float32), qw, np.array([[0.5, 0.25]], np.float32))
    np.testing.assert_array_equal(y, np.full((1, 8), 2 * 0.5 * 128 + 4 * 0.25 * 16, np.float32))


def test_grouped_linear_is_the_linear_of_each_segment():
    off = np.array([0, 2, 2, 5], np.int32)
    qx, qw = S.fp8_codes((5, 128), seed=1), S.fp8_codes((3, 16, 128), seed=2)
    sx, sw = np.ones((5, 1), np.float32), np.ones((3, 1, 1), np.float32)
    y = O.fp8_block_grouped_linear(qx, sx, off, qw, sw)
    np.testing.assert_array_equal(y[:2], O.fp8_block_linear(qx[:2], sx[:2], qw[0], sw[0]))
    np.testing.assert_array_equal(y[2:], O.fp8_block_linear(qx[2:], sx[2:], qw[2], sw[2]))


def test_route_grouped_without_groups_is_the_plain_route():
    lg = S.router_logits(50, 24, seed=1)
    ids, w, _ = O.moe_route_grouped(lg, 5, scoring="softmax", renormalize=False)
    r_ids, r_w, off, rt, ro = O.moe_route(lg, 5, False)
    np.testing.assert_array_equal(ids, r_ids)
    np.testing.assert_allclose(w, r_w, rtol=1e-6)
    for a, b in zip(O.row_order(ids, 24), (off, rt, ro)):
        np.testing.assert_array_equal(a, b)


def test_route_grouped_worked_example():
    """Eight experts in four groups of two. By the largest key the groups rank 2, 0,
    3, 1; by the sum of two (with a bias) the bias on expert 3 lifts group 1."""
    lg = np.array([[2.0, -1.0, 0.5, 0.4, 3.0, -3.0, 1.0, 0.9]], np.float32)
    ids, w, _ = O.moe_route_grouped(lg, 3, n_group=4, topk_group=2, renormalize=False)
    np.testing.assert_array_equal(ids, [[4, 0, 1]])
    np.testing.assert_allclose(w[0], 1 / (1 + np.exp(-lg[0, [4, 0, 1]].astype(np.float64))), rtol=1e-12)
    bias = np.zeros(8, np.float32)
    bias[3] = 1.0
    ids, w, _ = O.moe_route_grouped(lg, 2, bias=bias, n_group=4, topk_group=1, renormalize=True, scale=2.0)
    np.testing.assert_array_equal(ids, [[3, 2]])     # keys 1.60 and 0.62: the best sum
    s = 1 / (1 + np.exp(-lg[0, [3, 2]].astype(np.float64)))
    np.testing.assert_allclose(w[0], 2 * s / s.sum(), rtol=1e-12)


def test_route_grouped_masked_row():
    lg = np.full((1, 4), -np.inf, np.float32)
    for scoring in ("sigmoid", "softmax"):
        ids, w, _ = O.moe_route_grouped(lg, 2, scoring=scoring)
        np.testing.assert_array_equal(ids, [[0, 1]])
        np.testing.assert_array_equal(w, [[0, 0]])
