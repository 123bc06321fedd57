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
