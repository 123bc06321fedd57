"""The example MoE layer: every stage of one layer held to the oracle on the
previous stage's GPU output, and the layer itself against the same calls."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
from _compare import check_bf16_output
from _gpu import bits, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_moe_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("fp8_moe_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules[spec.name] = m          # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("T", [1, 7, 64, 700])
def test_layer_stage_by_stage(T):
    layer = example().random_layer(seed=T)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, layer.router.shape[1]), generator=g).to(torch.bfloat16).cuda()
    out = layer(x)

    logits = x.float() @ layer.router.T
    ids, wts, off, rt, ro = w4.w4_moe_route_grouped(logits, layer.top_k, bias=layer.balance, n_group=layer.n_group,
                                                    topk_group=layer.topk_group, scale=layer.route_scale)
    r_ids, r_w, gap = O.moe_route_grouped(logits.cpu().numpy(), layer.top_k, bias=layer.balance.cpu().numpy(),
                                          n_group=layer.n_group, topk_group=layer.topk_group, scale=layer.route_scale)
    clear = gap > 2.0 ** -20
    np.testing.assert_array_equal(ids.cpu().numpy()[clear], r_ids[clear])
    np.testing.assert_allclose(wts.cpu().numpy()[clear], r_w[clear], rtol=2e-5)
    offn = off.cpu().numpy()

    h = w4.w4_fp8_block_moe_gemm_bf16in(x, rt, off, layer.gate_up.codes, layer.gate_up.scale)
    q, s = O.quant_fp8_per_block(bits(x)[rt.cpu().numpy()])
    check_bf16_output(bits(h), O.fp8_block_grouped_linear(q, s, offn, codes(layer.gate_up.codes),
                                                          layer.gate_up.scale.cpu().numpy()), "gate_up")
    a, sa = w4.w4_silu_mul_quant_block(h)
    y = w4.w4_fp8_block_moe_grouped_gemm(a, sa, off, layer.down.codes, layer.down.scale)
    check_bf16_output(bits(y), O.fp8_block_grouped_linear(codes(a), sa.cpu().numpy(), offn, codes(layer.down.codes),
                                                          layer.down.scale.cpu().numpy()), "down")
    routed = w4.w4_moe_combine(y, wts, ro)
    hs = w4.w4_fp8_block_gemm_bf16in(x, layer.shared_gate_up.codes, layer.shared_gate_up.scale)
    b, sb = w4.w4_silu_mul_quant_block(hs)
    shared = w4.w4_fp8_block_gemm(b, sb, layer.shared_down.codes, layer.shared_down.scale)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(shared), O.fp8_block_linear(codes(b), sb.cpu().numpy(), codes(layer.shared_down.codes),
                                                       layer.shared_down.scale.cpu().numpy()), "shared down")
    np.testing.assert_array_equal(bits(out), bits(routed + shared))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 64])
def test_shared_expert_of_the_layer(T):
    """The shared expert's gate_up from 16-bit tokens, quantized in the product or before it."""
    layer = example().random_layer(seed=T + 1)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, layer.router.shape[1]), generator=g).to(torch.bfloat16).cuda()
    h = w4.w4_fp8_block_gemm_bf16in(x, layer.shared_gate_up.codes, layer.shared_gate_up.scale)
    torch.cuda.synchronize()
    q, s = O.quant_fp8_per_block(bits(x))
    check_bf16_output(bits(h), O.fp8_block_linear(q, s, codes(layer.shared_gate_up.codes),
                                                  layer.shared_gate_up.scale.cpu().numpy()), "shared gate_up")
