"""Chains of calls without a synchronization against the same calls with one, bit for bit, at sizes
whose copies go around the slots of shared memory many times: a slot that was given back before its
words were read would show as another output."""
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
from _gpu import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

FORMATS = ["int4", "mxfp4", "nvfp4"]


def random(*shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(torch.bfloat16)


def weight(E, N, K, fmt, seed, group=128):
    """Codes of every kind, scales in a small range, and (nvfp4) a scale per expert."""
    g = torch.Generator("cuda").manual_seed(seed)
    if fmt == "int4":
        q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), device="cuda", generator=g).to(torch.int32)
        return q, (0.002 + 0.003 * torch.rand((E, N, K // group), device="cuda", generator=g)).half(), None
    q = torch.randint(0, 256, (E, N, K // 2), device="cuda", generator=g).to(torch.uint8)
    low, high, block = (119, 123, 32) if fmt == "mxfp4" else (0x20, 0x40, 16)
    s = torch.randint(low, high, (E, N, K // block), device="cuda", generator=g).to(torch.uint8)
    return q, s, None if fmt == "mxfp4" else torch.full((E,), 0.013, device="cuda")


def check_chain(call, inputs, rounds=12):
    ref = []
    for i in range(len(inputs)):
        ref.append(call(inputs[i]).clone())
        torch.cuda.synchronize()
        assert torch.isfinite(ref[-1]).all() and (ref[-1] != 0).float().mean() > 0.99
    for _ in range(rounds):
        order = [i % len(inputs) for i in range(2 * len(inputs))]
        got = [call(inputs[i]) for i in order]
        torch.cuda.synchronize()
        assert all(torch.equal(y, ref[i]) for i, y in zip(order, got))
    assert w4.w4_device_status() == w4.W4_OK


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", [2, 24, 150, 1500])
def test_experts(fmt, T):
    E, k, N, K = 64, 8, 2816, 2048
    q, s, g = weight(E, N, K, fmt, 1)
    xg = torch.tensor([6.0 / (6 * 448)], device="cuda") if fmt == "nvfp4" else None

    def tokens(seed):
        ids = torch.rand((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        offsets = torch.searchsorted(ids[order], torch.arange(E + 1, device="cuda")).to(torch.int32)
        return random(T, K, seed=seed), (order // k).to(torch.int32), offsets

    check_chain(lambda v: w4.w4_fp4_moe_gemm_bf16in(*v, q, s, fmt, xg, g), [tokens(n) for n in range(3)])


def check_layer(fmt, T, E, k, H, I, group=128):
    (u, us, ug), (d, ds, dg) = weight(E, 2 * I, H, fmt, 1, group), weight(E, H, I, fmt, 2, group)

    def call(v):
        return w4.w4_moe_decode(*v, u, us, d, ds, k, fmt, gate_up_global=ug, down_global=dg, scoring="softmax")

    check_chain(call, [(random(T, H, seed=n), random(T, E, seed=n + 10).float()) for n in range(4)])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 8, 16])
def test_few_token_layer(fmt, T):
    check_layer(fmt, T, 64, 8, 2048, 1408)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k,H,I", [(7, 96, 6, 1088, 704), (16, 40, 4, 1088, 320), (3, 24, 6, 512, 2112), (11, 24, 6, 512, 4160)])
def test_few_token_layer_of_other_sizes(fmt, T, E, k, H, I):
    """Rows of scales that are no whole 16 bytes, or of several stages; more columns than the block-scaled kernels take."""
    check_layer(fmt, T, E, k, H, I, 64)
