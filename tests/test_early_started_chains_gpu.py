"""Chains of kernels that start while the kernels before them run (the fp8 block-scaled
layer, the grouped router and the W4A16 GEMM), each call reading what the one before it
writes: results equal the same calls with a synchronization between them."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import synthetic as S
from _gpu import bf16, bits, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]

G = 128


def fp8_weight(N, K, seed):
    q = S.fp8_codes((N, K), seed=seed)
    q = ((q & 0x80) | (q & 0x7F) % 0x39).astype(np.uint8)
    s = S.scales_f16((-(-N // 128), -(-K // 128)), seed=seed + 1).astype(np.float32)
    return to_dev(q).view(torch.float8_e4m3fn), to_dev(s)


def int4_weight(N, K, seed):
    return to_dev(S.random_words((K // 8, N), seed=seed)), to_dev(S.scales_f16((K // G, N), seed=seed + 1))


@pytest.mark.parametrize("M", [1, 8, 64, 300, 3000])
def test_w4a16_after_an_fp8_product(M):
    """The GEMV of the last rows starts while the product, however long, still writes them."""
    H, N, K = 2048, 1024, 4096
    wq, ws = fp8_weight(H, K, 1)
    qw, sw = int4_weight(N, H, 3)
    x = bf16(S.activations_bf16(M, K, seed=M))
    y, z = torch.empty((M, H), dtype=torch.bfloat16, device="cuda"), torch.empty((min(M, 8), N), dtype=torch.bfloat16, device="cuda")
    tail = y[M - min(M, 8):]
    w4.w4_fp8_block_gemm_bf16in(x, wq, ws, y=y)
    torch.cuda.synchronize()
    w4.w4a16_gemm(tail, qw, sw, G, y=z)
    torch.cuda.synchronize()
    ref = bits(z)
    assert np.isfinite(z.float().cpu().numpy()).all()
    for _ in range(30):
        y.fill_(float("nan"))
        z.fill_(float("nan"))
        w4.w4_fp8_block_gemm_bf16in(x, wq, ws, y=y)
        w4.w4a16_gemm(tail, qw, sw, G, y=z)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(z), ref)
    assert w4.w4_device_status() == w4.W4_OK


@pytest.mark.parametrize("M", [1, 8, 24])
def test_layers_of_both_kinds_in_turn(M):
    """int4 and fp8 layers of one width in turn, in place in two buffers, several times over
    without a synchronization: every call overwrites what the call before the last one wrote
    and the last one read."""
    H, L = 2048, 6
    a = [int4_weight(H, H, 10 * i) for i in range(L)]
    b = [fp8_weight(H, H, 10 * i + 5) for i in range(L)]
    x = bf16(S.activations_bf16(M, H, seed=1))
    bufs = [torch.empty_like(x), torch.empty_like(x)]

    def run(sync):
        bufs[0].copy_(x)
        for i in range(L):
            w4.w4a16_gemm(bufs[0], *a[i], G, y=bufs[1])
            if sync:
                torch.cuda.synchronize()
            w4.w4_fp8_block_gemm_bf16in(bufs[1], *b[i], y=bufs[0])
            if sync:
                torch.cuda.synchronize()
        return bufs[0].clone()

    # scales small enough that twelve layers stay in range
    for w in a:
        w[1].mul_(0.02)
    for w in b:
        w[1].mul_(0.05)
    last = run(True)
    assert torch.isfinite(last).all() and (last != 0).float().mean() > 0.99
    ref = bits(last)
    outs = [run(False) for _ in range(20)]
    torch.cuda.synchronize()
    for y in outs:
        np.testing.assert_array_equal(bits(y), ref)
    assert w4.w4_device_status() == w4.W4_OK


@pytest.mark.parametrize("T", [4, 40, 700, 5000])
def test_routing_into_the_same_buffers(T):
    """Router, experts from tokens, quantizer and experts from codes over and over in the same
    outputs and workspaces: each pass reads the offsets and rows of its own routing, although
    the products start while the kernels before them run. At 5000 tokens codes are copied."""
    E, k, H, I = 16, 4, 1024, 256
    lead = (E,)
    def weight(N, K, seed):
        q = S.fp8_codes(lead + (N, K), seed=seed)
        q = ((q & 0x80) | (q & 0x7F) % 0x39).astype(np.uint8)
        s = S.scales_f16(lead + (N // 128, K // 128), seed=seed + 1).astype(np.float32)
        return to_dev(q).view(torch.float8_e4m3fn), to_dev(s)
    up, down = weight(2 * I, H, 1), weight(H, I, 3)
    R, dev = T * k, "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    out = (torch.empty((T, k), **i32), torch.empty((T, k), device=dev), torch.empty(E + 1, **i32), torch.empty(R, **i32),
           torch.empty((T, k), **i32))
    ws_r = torch.empty(max(16, w4.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE_GROUPED, T, E, 1, 0)), dtype=torch.uint8, device=dev)
    ws_u = torch.empty(w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, R, 2 * I, H, E), dtype=torch.uint8, device=dev)
    h, y = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=dev), torch.empty((R, H), dtype=torch.bfloat16, device=dev)
    a, s = torch.empty((R, I), dtype=torch.float8_e4m3fn, device=dev), torch.empty((R, I // 128), device=dev)
    inputs = [(to_dev(S.router_logits(T, E, seed=n)), bf16(S.activations_bf16(T, H, seed=n + 50))) for n in range(5)]

    def one(n, sync):
        lg, x = inputs[n]
        wait = torch.cuda.synchronize if sync else (lambda: None)
        w4.w4_moe_route_grouped(lg, k, n_group=4, topk_group=2, out=out, workspace=ws_r)
        wait()
        w4.w4_fp8_block_moe_gemm_bf16in(x, out[3], out[2], *up, y=h, workspace=ws_u)
        wait()
        w4.w4_silu_mul_quant_block(h, q=a, scale=s)
        wait()
        w4.w4_fp8_block_moe_grouped_gemm(a, s, out[2], *down, y=y)
        wait()
        return w4.w4_moe_combine(y, out[1], out[4])

    ref = [bits(one(n, True)) for n in range(5)]
    order = [0, 1, 2, 3, 4, 2, 0, 4, 1, 3] * 4
    got = [one(n, False) for n in order]
    torch.cuda.synchronize()
    for n, z in zip(order, got):
        np.testing.assert_array_equal(bits(z), ref[n])
    assert w4.w4_device_status() == w4.W4_OK
