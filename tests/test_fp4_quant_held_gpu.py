"""nvfp4 blocks far beyond what their scale can stand for: the scale is held at 448 and the codes at
6, each with the sign of its number, by the quantizer and by the product that quantizes few rows itself."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from _gpu import bf16, dev, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]

ROWS = [np.full(64, -3.3e38), np.full(64, 3.3e38), np.resize([-3.3e38, 3.3e38, -1e38, 2e-3], 64), np.resize([-5e4, 7e3, -2e3, 1.1], 64),
        np.resize([-1e30, 3e32, -2.0, -0.0], 64), np.resize([-2.6875, 2.6875, -4.1e3, 1835.0], 64)]


def host(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


@pytest.mark.parametrize("g", [1.0, 1e-3, 2.5e-13, 1e-20, 3e-38])
@pytest.mark.parametrize("f16", [False, True])
def test_codes_keep_their_sign(g, f16):
    x = np.stack(ROWS)
    t = torch.tensor([g], dtype=torch.float32, device=dev())
    if f16:
        x = np.clip(x, -65504, 65504).astype(np.float16)
        q, s = w4.w4_quant_fp4(to_dev(x), "nvfp4", t)
        rq, rs = O.quant_fp4(x, "nvfp4", g)
    else:
        xb = S.to_bf16_bits(x)
        q, s = w4.w4_quant_fp4(bf16(xb), "nvfp4", t)
        rq, rs = O.quant_fp4(xb, "nvfp4", g)
    assert np.array_equal(host(s).reshape(rs.shape), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("g", [1e-3, 2.5e-13])
def test_the_product_of_few_rows_keeps_it_too(g):
    x = bf16(S.to_bf16_bits(np.concatenate([np.stack(ROWS)] * 2, axis=1)))
    t = torch.tensor([g], dtype=torch.float32, device=dev())
    w = to_dev(np.full((8, 64), 0x22, np.uint8))           # ones
    sw = to_dev(np.full((8, 8), 0x38, np.uint8))
    y = w4.w4_fp4_gemm_bf16in(x, w, sw, "nvfp4", t)
    q, s = w4.w4_quant_fp4(x, "nvfp4", t)
    assert torch.equal(y, w4.w4_fp4_gemm(q, s, w, sw, "nvfp4", t))
    # a row of one number: 128 codes of 6 with its sign, at 448 g
    want = torch.tensor([-128 * 6 * 448 * np.float32(g), 128 * 6 * 448 * np.float32(g)]).to(torch.bfloat16)
    assert torch.equal(y[:2, 0].cpu(), want)


def test_silu_mul_keeps_it():
    h = np.zeros((2, 64), np.float32)
    h[:, :32], h[0, 32:], h[1, 32:] = 1e19, -3e18, 3e18
    q, _ = w4.w4_silu_mul_quant_fp4(bf16(S.to_bf16_bits(h)), "nvfp4", torch.tensor([1e-6], device=dev()))
    assert (O.fp4_decode(host(q))[0] == -6).all() and (O.fp4_decode(host(q))[1] == 6).all()
