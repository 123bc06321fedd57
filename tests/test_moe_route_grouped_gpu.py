"""Grouped routing (sigmoid or softmax scores, balance bias, expert groups) on
the GPU against the oracle, through the C ABI."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from _gpu import bf16, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]


def _check(logits, logits_d, k, bias=None, **kw):
    T, E = logits.shape
    ids, wts, off, rt, ro = w4.w4_moe_route_grouped(logits_d, k, bias=None if bias is None else to_dev(bias), **kw)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    ids, wts = ids.cpu().numpy(), wts.cpu().numpy()
    r_ids, r_w, gap = O.moe_route_grouped(logits, k, bias=bias, **kw)
    # without a bias the choice compares the logits themselves, exactly; with one, two keys (or sums of two)
    # closer than a few fp32 roundings of values up to 4 may come out in either order
    clear = np.ones(T, bool) if bias is None else gap > 2.0 ** -20
    assert clear.mean() >= 0.95 or T < 40
    np.testing.assert_array_equal(ids[clear], r_ids[clear])
    np.testing.assert_allclose(wts[clear], r_w[clear], rtol=2e-5, atol=1e-9)
    r_off, r_rt, r_ro = O.row_order(ids, E)
    np.testing.assert_array_equal(off.cpu().numpy(), r_off)
    np.testing.assert_array_equal(rt.cpu().numpy(), r_rt)
    np.testing.assert_array_equal(ro.cpu().numpy(), r_ro)
    return ids, wts


@pytest.mark.parametrize("T,E,k,G,keep", [
    (1, 64, 8, 1, 1), (1, 1, 1, 1, 1), (3, 256, 8, 8, 4), (37, 96, 6, 8, 3), (200, 160, 6, 8, 3), (100, 60, 5, 5, 2),
    (129, 33, 4, 3, 2), (257, 256, 8, 8, 4), (65, 1024, 64, 32, 7), (40, 512, 10, 2, 1), (50, 24, 4, 24, 5),
    (600, 40, 1, 4, 1), (31, 992, 3, 31, 30)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_grouped_matches_oracle(T, E, k, G, keep, scoring, with_bias):
    lg = S.router_logits(T, E, seed=T + E)
    bias = (S.normal(T, 80, E) * 0.1).astype(np.float32) if with_bias else None
    _check(lg, to_dev(lg), k, bias, n_group=G, topk_group=keep, scoring=scoring, renormalize=T % 2 == 0, scale=2.5)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_grouped_bf16_ties(scoring):
    """bf16 logits tie often, whole groups tie: the lower index wins. With a
    bias of equal values equal logits have equal keys."""
    b = S.to_bf16_bits(S.router_logits(300, 64, seed=4))
    lg = S.bf16_bits_to_f32(b)
    lg[0] = 0.5
    lg[1, :32], lg[1, 32:] = 0.25, 0.25
    lg[2, 8:16], lg[2, 40:48] = 3.0, 3.0
    d = bf16(S.to_bf16_bits(lg))
    _check(lg, d, 6, None, n_group=8, topk_group=2, scoring=scoring)
    ids, _ = _check(lg, d, 6, np.full(64, 0.125, np.float32), n_group=8, topk_group=2, scoring=scoring)
    np.testing.assert_array_equal(ids[0], np.arange(6))
    np.testing.assert_array_equal(ids[2], np.arange(8, 14))


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_grouped_masked_logits(scoring, with_bias):
    """-inf (masked), NaN and +inf logits, rows masked altogether among them."""
    T, E = 40, 64
    lg = S.router_logits(T, E, seed=8)
    lg[0] = -np.inf
    lg[1, 5:] = -np.inf
    lg[2, 9] = np.nan
    lg[3, 3] = np.inf
    lg[4] = np.float32(-3.4e38)
    lg[5, :] = np.float32(100.0)
    bias = (S.normal(3, 80, E) * 0.1).astype(np.float32) if with_bias else None
    for renorm in (True, False):
        ids, w = _check(lg, to_dev(lg), 8, bias, n_group=4, topk_group=2, scoring=scoring, renormalize=renorm)
        assert np.isfinite(w).all() and not w[0].any()
        assert all(len(set(r)) == 8 for r in ids.tolist())


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_grouped_equals_plain_route(scoring):
    """One group, no bias: the choice of w4_moe_route; with softmax its weights too."""
    lg = to_dev(S.router_logits(700, 128, seed=6))
    a = w4.w4_moe_route(lg, 7, True)
    b = w4.w4_moe_route_grouped(lg, 7, scoring=scoring, renormalize=True)
    torch.cuda.synchronize()
    for i in (0, 2, 3, 4):
        np.testing.assert_array_equal(a[i].cpu().numpy(), b[i].cpu().numpy())
    if scoring == "softmax":
        np.testing.assert_allclose(a[1].cpu().numpy(), b[1].cpu().numpy(), rtol=2e-6)


@pytest.mark.parametrize("T", [0, 2049, 20000])
def test_route_grouped_many_tokens(T):
    E, k = 48, 4
    lg = S.router_logits(T, E, seed=7)
    ids, wts, off, rt, ro = w4.w4_moe_route_grouped(to_dev(lg), k, n_group=4, topk_group=2)
    torch.cuda.synchronize()
    ids = ids.cpu().numpy()
    counts = np.bincount(ids.reshape(-1), minlength=E)
    np.testing.assert_array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    order = np.argsort(ids.reshape(-1), kind="stable")
    np.testing.assert_array_equal(rt.cpu().numpy(), order // k)
    np.testing.assert_array_equal(ro.cpu().numpy().reshape(-1)[order], np.arange(T * k))


@pytest.mark.parametrize("given", [False, True])
def test_routes_of_no_tokens_have_empty_segments(given):
    """T = 0: every offset is 0, in outputs of the caller's too (a reused buffer would
    otherwise keep the segments of the call before)."""
    E, k = 48, 4
    lg = torch.empty((0, E), device="cuda")
    for route in (w4.w4_moe_route_grouped, w4.w4_moe_route):
        i32 = dict(dtype=torch.int32, device="cuda")
        out = (torch.empty((0, k), **i32), torch.empty((0, k), device="cuda"), torch.full((E + 1,), 7, **i32),
               torch.empty((0,), **i32), torch.empty((0, k), **i32)) if given else None
        got = route(lg, k, out=out)
        torch.cuda.synchronize()
        assert not got[2].any() and got[2].shape == (E + 1,) and got[0].shape == (0, k)
        assert not given or got[2].data_ptr() == out[2].data_ptr()


@pytest.mark.parametrize("top_k", [65, 1 << 20, 2 ** 31 - 1])
def test_refused_top_k_asks_for_no_memory(top_k):
    """The library's refusal, not an allocation of T * top_k words that fails before it."""
    lg = torch.zeros((100000, 64), device="cuda")
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(w4.W4Error) as e:
        w4.w4_moe_route_grouped(lg, top_k)
    assert e.value.status == w4.W4_ERR_SHAPE
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_masked_experts_with_and_without_a_bias(scoring):
    """A logit of -inf is chosen last without a bias; with one its key is the bias alone. A
    bias of -inf closes an expert."""
    lg = np.full((1, 8), -2.0, np.float32)
    lg[0, 3] = -np.inf
    ids, _ = _check(lg, to_dev(lg), 8, None, scoring=scoring)
    assert ids[0, -1] == 3
    bias = np.zeros(8, np.float32)
    bias[3], bias[5] = 1.0, -np.inf
    ids, w = _check(lg, to_dev(lg), 8, bias, scoring=scoring, renormalize=False)
    assert ids[0, 0] == 3 and w[0, 0] == 0 and ids[0, -1] == 5


@pytest.mark.parametrize("T,E,k,G,keep", [(5000, 256, 8, 8, 4), (16384, 256, 8, 8, 4), (2500, 512, 10, 2, 1),
                                          (1300, 1024, 16, 32, 8), (5000, 64, 6, 1, 1), (10001, 33, 4, 3, 2)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_grouped_more_tokens_than_warps(T, E, k, G, keep, scoring, with_bias):
    """Tiles of more tokens than their CTA has warps: a warp routes several, the next one's
    logits on their way meanwhile. Ids and weights of every token against the oracle."""
    lg = S.router_logits(T, E, seed=T + k)
    bias = (S.normal(T, 80, E) * 0.1).astype(np.float32) if with_bias else None
    _check(lg, to_dev(lg), k, bias, n_group=G, topk_group=keep, scoring=scoring, renormalize=T % 2 == 0, scale=2.5)
