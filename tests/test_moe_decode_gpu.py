"""The few-token expert layer against the float64 oracle.

An output is off by its rounding to bf16 (2^-8 of it at most), by the activations'
rounding, in int4 to 11 bits (2^-11 of each, so of the sum of magnitudes `size`), in the 4-bit
floating point formats to 2^-13 of the largest of 16 or 32 neighbours, for x and for the activations
in between: with signs and sizes at random, 2^-13 of a few typical magnitudes each, of which a sum
of K terms keeps a share of about K^-1/2; and by fp32 sums: a chain of at most 2^10 additions a warp,
2^-23 each of what is summed, for gate, up and output, which silu enlarges by less than twice.
2^-10 of `size` covers either."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from tests._gpu import bf16, dev, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]

FORMATS = ["int4", "mxfp4", "nvfp4"]


class Experts:
    """Random experts in a format: tensors of the call, and values for the oracle."""

    def __init__(self, E, H, I, fmt, group=64, seed=1):
        self.fmt, self.E, self.H, self.I = fmt, E, H, I
        self.parts = [self._part(E, 2 * I, H, group, seed), self._part(E, H, I, group, seed + 10)]

    def _part(self, E, N, K, group, seed):
        if self.fmt == "int4":
            g = K if group == -1 else group
            q = S.random_words((E, N, K // 8), seed=seed)
            s = S.scales_f16((E, N, K // g), seed=seed + 1)
            return q, s, None
        q = S.fp8_codes((E, N, K // 2), seed=seed)
        raw = S.fp8_codes((E, N, K // O.FP4_BLOCK[self.fmt]), seed=seed + 1)
        if self.fmt == "mxfp4":
            return q, (118 + raw % 5).astype(np.uint8), None
        return q, (0x20 + raw % 0x30).astype(np.uint8), np.linspace(0.01, 0.02, E).astype(np.float32)

    def values(self, i, e):
        q, s, g = self.parts[i]
        if self.fmt == "int4":
            return (O.unpack_ct(q[e:e + 1])[0].astype(np.float64) - 8) * np.repeat(s[e].astype(np.float64), q.shape[2] * 8 // s.shape[2], axis=1)
        v = O.dequant_fp4(q[e], s[e], self.fmt)
        return v if g is None else v * np.float64(g[e])

    def call(self, xb, logits, top_k, **kw):
        (u, us, ug), (d, ds, dg) = self.parts
        dv = lambda a: None if a is None else to_dev(a)  # noqa: E731
        if not hasattr(self, "_dev"):
            self._dev = [dv(a) for a in (u, us, d, ds, ug, dg)]
        u, us, d, ds, ug, dg = self._dev
        return w4.w4_moe_decode(bf16(xb), to_dev(logits), u, us, d, ds, top_k, self.fmt, gate_up_global=ug, down_global=dg, **kw)

    def check(self, xb, logits, top_k, bias=None, **route):
        y = self.call(xb, logits, top_k, bias=None if bias is None else to_dev(bias), **route)
        torch.cuda.synchronize()
        assert w4.w4_device_status() == w4.W4_OK
        r, size = O.moe_decode(xb, logits, lambda e: self.values(0, e), lambda e: self.values(1, e), top_k, bias=bias, **route)
        err = np.abs(y.float().cpu().numpy() - r)
        over = err / (2.0 ** -8 * np.abs(r) + 2.0 ** -10 * size + 1e-37)
        assert over.max() <= 1.0, (over.max(), np.unravel_index(over.argmax(), over.shape))
        assert np.sqrt(np.mean(err ** 2)) <= 2.5e-3 * np.sqrt(np.mean(r ** 2)) + 1e-37
        return y


def inputs(T, H, E, seed=0):
    return S.activations_bf16(T, H, seed=seed, outlier_frac=0.01), S.router_logits(T, E, seed=seed + 3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16])
def test_any_number_of_tokens(fmt, T):
    Experts(24, 512, 320, fmt).check(*inputs(T, 512, 24, seed=T), 4, scoring="softmax")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,I,group", [(64, 64, 32), (128, 64, 64), (1024, 128, 128), (1088, 1408, 32), (2048, 704, 64), (2048, 1408, -1), (4096, 64, 64)])
def test_sizes(fmt, H, I, group):
    if fmt == "int4" and group > 0 and (H % group or I % group):
        group = 64
    Experts(5, H, I, fmt, group).check(*inputs(3, H, 5, seed=H), 2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_all_tokens_choose_the_same_experts(fmt):
    """Sixteen tokens an expert, in two blocks of eight columns."""
    xb, logits = inputs(16, 256, 4)
    logits[:, 2] += 50
    logits[:13, 0] += 40
    Experts(4, 256, 192, fmt).check(xb, logits, 2, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,k,n_group,topk_group,scoring", [(1, 1, 1, 1, "softmax"), (256, 32, 1, 1, "sigmoid"), (65, 8, 5, 2, "sigmoid"), (64, 8, 8, 3, "softmax"), (200, 6, 8, 4, "sigmoid")])
def test_routing_arguments(E, k, n_group, topk_group, scoring):
    xb, logits = inputs(6, 128, E, seed=E)
    bias = S.zeros_bf16((1, E), std=0.1)
    bias = O.bf16_to_f64(bias)[0].astype(np.float32)
    _, _, gap = O.moe_route_grouped(logits, k, bias=bias, n_group=n_group, topk_group=topk_group, scoring=scoring)
    assert gap.min() > 2.0 ** -22      # the choice is the same in fp32
    Experts(E, 128, 64, "mxfp4").check(xb, logits, k, bias=bias, n_group=n_group, topk_group=topk_group, scoring=scoring)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e8])
def test_activations_of_any_size(fmt, size):
    """Powers of two leave fp16's range to the exponents kept beside it."""
    xb, logits = inputs(4, 256, 6)
    x = O.bf16_to_f64(xb) * size
    x[1] *= 1e-4
    Experts(6, 256, 128, fmt).check(S.to_bf16_bits(x), logits, 2)


def test_a_token_with_nan_or_infinity_leaves_the_others_alone():
    ex = Experts(4, 128, 64, "int4")
    xb, logits = inputs(4, 128, 4)
    clean = ex.call(xb, logits, 3)
    x = O.bf16_to_f64(xb).astype(np.float32)
    x[1, 5], x[3, 100] = np.nan, np.inf
    y = ex.call(S.to_bf16_bits(x), logits, 3)
    assert torch.isnan(y[1].float()).all() and not torch.isfinite(y[3].float()).any()
    assert torch.equal(y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_token_of_zeros_gives_zeros(fmt):
    xb, logits = inputs(3, 128, 4)
    xb[1] = 0
    y = Experts(4, 128, 64, fmt).call(xb, logits, 2)
    assert (y[1] == 0).all() and (y[0] != 0).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_do_not_depend_on_the_batch(fmt):
    """A token's output is the same alone as among others (its sums have the same order)
    where its experts share no more than eight tokens."""
    ex = Experts(16, 256, 192, fmt)
    xb, logits = inputs(6, 256, 16, seed=9)
    all_of = ex.call(xb, logits, 4)
    one = ex.call(xb[2:3], logits[2:3], 4)
    assert np.allclose(all_of[2].float().cpu().numpy(), one[0].float().cpu().numpy(), rtol=2.0 ** -7, atol=1e-3 * float(one.float().abs().max()))


@pytest.mark.parametrize("fmt", FORMATS)
def test_repeated_and_captured_calls_are_the_same(fmt):
    ex = Experts(32, 512, 256, fmt)
    xb, logits = inputs(5, 512, 32)
    x, lg = bf16(xb), to_dev(logits)
    ex.call(xb, logits, 4)
    u, us, d, ds, ug, dg = ex._dev
    call = lambda **kw: w4.w4_moe_decode(x, lg, u, us, d, ds, 4, fmt, gate_up_global=ug, down_global=dg, **kw)  # noqa: E731
    first = call()
    outs = [call() for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    y = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y=y)
        call(y=y)
    x2, l2 = inputs(5, 512, 32, seed=7)
    x.copy_(bf16(x2)), lg.copy_(to_dev(l2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, call())


def test_no_tokens():
    ex = Experts(4, 128, 64, "mxfp4")
    assert ex.call(np.zeros((0, 128), np.uint16), np.zeros((0, 4), np.float32), 2).shape == (0, 128)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_token_with_nan_or_infinity_leaves_the_others_alone_in_fp4(fmt):
    ex = Experts(4, 128, 64, fmt)
    xb, logits = inputs(4, 128, 4)
    clean = ex.call(xb, logits, 3)
    x = O.bf16_to_f64(xb).astype(np.float32)
    x[1, 5], x[3, 100] = np.nan, np.inf
    y = ex.call(S.to_bf16_bits(x), logits, 3)
    assert torch.isnan(y[1].float()).all() and not torch.isfinite(y[3].float()).any()
    assert torch.equal(y[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("H,I,group", [(384, 192, 96), (2048, 1408, 128), (192, 576, 192), (1088, 320, 64)])
@pytest.mark.parametrize("T", [2, 16])
def test_groups_of_an_int4_scale(H, I, group, T):
    """Scales that end inside a warp's columns, and numbers of columns that are no power of two."""
    Experts(6, H, I, "int4", group).check(*inputs(T, H, 6, seed=H + T), 3)


@pytest.mark.parametrize("fmt,T,H,I", [("mxfp4", 3, 128, 2112), ("nvfp4", 9, 128, 2112), ("nvfp4", 2, 320, 4096), ("mxfp4", 1, 8256, 64)])
def test_sizes_past_the_block_scaled_form(fmt, T, H, I):
    Experts(5, H, I, fmt).check(*inputs(T, H, 5, seed=I), 2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bf16_logits(fmt):
    """Choices among rounded logits: as with the same numbers in fp32."""
    ex = Experts(24, 128, 64, fmt)
    xb, logits = inputs(7, 128, 24)
    lb = S.to_bf16_bits(logits)
    want = ex.call(xb, O.bf16_to_f64(lb).astype(np.float32), 5)
    u, us, d, ds, ug, dg = ex._dev
    got = w4.w4_moe_decode(bf16(xb), bf16(lb), u, us, d, ds, 5, fmt, gate_up_global=ug, down_global=dg)
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_masked_logits(fmt):
    """Experts masked by -inf or the lowest number are chosen last; a token with nothing but -inf weighs nothing."""
    ex = Experts(12, 128, 64, fmt)
    xb, logits = inputs(3, 128, 12)
    logits[0, 3:] = -np.inf
    logits[1, :] = -np.inf
    logits[2, 4:] = np.finfo(np.float32).min
    y = ex.call(xb, logits, 3, scoring="softmax")
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    ids, wts, _ = O.moe_route_grouped(logits, 3, scoring="softmax")
    assert sorted(ids[0].tolist()) == [0, 1, 2]
    r, size = O.moe_decode(xb[[0, 2]], logits[[0, 2]], lambda e: ex.values(0, e), lambda e: ex.values(1, e), 3, scoring="softmax")
    err = np.abs(y[[0, 2]].float().cpu().numpy() - r)
    assert (err <= 2.0 ** -8 * np.abs(r) + 2.0 ** -10 * size).all()
    assert (y[1] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [3, 12])
def test_a_larger_call_captured_after_a_smaller_one(fmt, T):
    """Kernels whose shared memory grows with the sizes: the first larger call may be one that is captured."""
    Experts(4, 64, 64, fmt).call(*inputs(T, 64, 4), 2)
    ex = Experts(4, 2048, 1024, fmt, group=128)
    xb, logits = inputs(T, 2048, 4, seed=T)
    (u, us, ug), (d, ds, dg) = ex.parts
    u, us, d, ds, ug, dg = (None if a is None else to_dev(a) for a in (u, us, d, ds, ug, dg))
    x, lg = bf16(xb), to_dev(logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w4.w4_moe_decode(x, lg, u, us, d, ds, 2, fmt, gate_up_global=ug, down_global=dg)
    graph.replay()
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    assert torch.equal(y, ex.call(xb, logits, 2))
