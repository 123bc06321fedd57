"""A routed mixture-of-experts layer on 4-bit floating point weights, for prefill and decode.

The experts' weights are e2m1 codes with block scales (``mxfp4`` or ``nvfp4``), quantized by the
library. Up to sixteen tokens take the few-token layer (16-bit activations, routing and both
products in one call) where that is the faster way and takes their sizes; others are routed, quantized to the
weights' format and multiplied on the block-scaled tensor cores. Run it on a GPU::

    python examples/fp4_moe_layer.py --tokens 64 --format nvfp4

All memory is allocated through PyTorch.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_quantized_w4_gb300 as w4

DECODE_TOKENS = 16
# Bytes of the chosen experts' weights up to which the few-token call is the faster one. On a GB300, it and the
# separate calls: 8 experts of 2048 x 1408 in mxfp4 (37 MB) 24 and 29 us, 15 of them 34 and 32; 39 of 1024 x 704 in
# nvfp4 (47 MB) 32 and 34; 8 of 4096 x 1536 (80 MB) 40 and 33.
DECODE_BYTES = 50e6


@dataclasses.dataclass
class Fp4Weight:
    """e2m1 codes ``[E, N, K/2]``, block scales ``[E, N, K/block]`` and (nvfp4) fp32 scales ``[E]``."""
    codes: torch.Tensor
    scale: torch.Tensor
    tensor_scale: torch.Tensor | None


@dataclasses.dataclass
class Fp4MoeLayer:
    router: torch.Tensor        # fp32 [E, H]
    gate_up: Fp4Weight          # [E, 2I, H], gate rows first
    down: Fp4Weight             # [E, H, I]
    x_scale: torch.Tensor | None   # nvfp4: fp32 scales of the quantized inputs of the two products
    a_scale: torch.Tensor | None
    format: str
    top_k: int

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """bf16 ``[T, H]`` -> bf16 ``[T, H]``."""
        logits = x.float() @ self.router.T
        if self.few(x.shape[0]):
            try:
                return self.decode(x, logits)
            except w4.W4Error as e:
                if e.status != w4.W4_ERR_UNSUPPORTED:
                    raise
        return self.prefill(x, logits)

    def few(self, tokens: int) -> bool:
        """Whether the few-token call is the faster one."""
        E = self.router.shape[0]
        chosen = E * (1 - (1 - self.top_k / E) ** tokens)      # experts that get a token, on average
        parts = (self.gate_up.codes, self.gate_up.scale, self.down.codes, self.down.scale)
        return tokens <= DECODE_TOKENS and chosen / E * sum(t.numel() for t in parts) <= DECODE_BYTES

    def decode(self, x, logits):
        u, d = self.gate_up, self.down
        return w4.w4_moe_decode(x, logits, u.codes, u.scale, d.codes, d.scale, self.top_k, self.format,
                                gate_up_global=u.tensor_scale, down_global=d.tensor_scale, scoring="softmax")

    def prefill(self, x, logits):
        u, d = self.gate_up, self.down
        _, weights, offsets, row_token, row_of = w4.w4_moe_route_grouped(logits, self.top_k, scoring="softmax")
        h = w4.w4_fp4_moe_gemm_bf16in(x, row_token, offsets, u.codes, u.scale, self.format, self.x_scale, u.tensor_scale)
        a, a_scale = w4.w4_silu_mul_quant_fp4(h, self.format, self.a_scale)
        y = w4.w4_fp4_moe_grouped_gemm(a, a_scale, offsets, d.codes, d.scale, self.format, self.a_scale, d.tensor_scale)
        return w4.w4_moe_combine(y, weights, row_of)


def quantize_weights(w: torch.Tensor, format: str) -> Fp4Weight:
    """bf16 ``[E, N, K]`` to 4-bit floats, expert by expert (load time)."""
    tensor_scale = None
    if format == "nvfp4":   # block scales of an expert reach up to e4m3's largest value
        tensor_scale = w.abs().amax(dim=(1, 2)).float() / (6 * 448)
    parts = [w4.w4_quant_fp4(w[e], format, None if tensor_scale is None else tensor_scale[e:e + 1]) for e in range(w.shape[0])]
    return Fp4Weight(torch.stack([q for q, _ in parts]), torch.stack([s.view(torch.uint8) for _, s in parts]), tensor_scale)


def random_layer(H=512, I=256, E=16, top_k=4, format="nvfp4", seed=0, device="cuda") -> Fp4MoeLayer:
    g = torch.Generator().manual_seed(seed)

    def weight(*shape):
        return quantize_weights((torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(torch.bfloat16).to(device), format)

    def largest(v):
        return torch.tensor([v / (6 * 448)], device=device) if format == "nvfp4" else None

    return Fp4MoeLayer(router=(torch.randn((E, H), generator=g) * H ** -0.5).to(device), gate_up=weight(E, 2 * I, H),
                       down=weight(E, H, I), x_scale=largest(6.0), a_scale=largest(12.0), format=format, top_k=top_k)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--format", choices=("mxfp4", "nvfp4"), default="nvfp4")
    a = ap.parse_args()
    layer = random_layer(format=a.format)
    x = torch.randn((a.tokens, layer.router.shape[1]), device="cuda").to(torch.bfloat16)
    y = layer(x)
    torch.cuda.synchronize()
    if w4.w4_device_status() != w4.W4_OK:
        raise SystemExit("a kernel reported an error")
    print(f"{a.tokens} tokens, {layer.router.shape[0]} experts, top {layer.top_k}: rms {y.float().square().mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
