"""The example layer on 4-bit floating point experts goes the way that takes its sizes."""
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
from _gpu import requires_cuda
from test_fp4_moe_layer_gpu import example, tokens

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("sizes", [dict(E=300, H=128, I=128), dict(E=64, H=128, I=128, top_k=40)])
def test_few_tokens_of_sizes_that_the_few_token_call_refuses(fmt, sizes):
    layer = example().random_layer(format=fmt, **sizes)
    x = tokens(3, sizes["H"], 1)
    logits = x.float() @ layer.router.T
    with pytest.raises(w4.W4Error) as e:
        layer.decode(x, logits)
    assert e.value.status == w4.W4_ERR_UNSUPPORTED
    y = layer(x)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    assert torch.equal(y, layer.prefill(x, logits)) and (y != 0).any()


def test_other_errors_are_raised():
    layer = example().random_layer(format="mxfp4", E=8, H=128, I=128)
    layer.top_k = 9
    with pytest.raises(w4.W4Error):
        layer(tokens(3, 128, 1))


def test_the_faster_way():
    """By what the chosen experts weigh."""
    layer = example().random_layer(format="mxfp4", E=64, H=1024, I=768, top_k=2)
    size = sum(t.numel() for t in (layer.gate_up.codes, layer.gate_up.scale, layer.down.codes, layer.down.scale)) / 64
    assert layer.few(0) and layer.few(1) and 2 * size < 50e6
    assert layer.few(16) == (64 * (1 - (1 - 2 / 64) ** 16) * size <= 50e6)
    assert not layer.few(17)
    layer.top_k = 64
    assert not layer.few(1) and 64 * size > 50e6
