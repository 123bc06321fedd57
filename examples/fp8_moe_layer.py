"""A routed mixture-of-experts layer on fp8 block-scaled weights.

The layer of a checkpoint that keeps its linear layers as e4m3 with one scale per
128 x 128 block: a router with sigmoid scores, a balance bias and expert groups,
gated expert projections over the routed rows, and a shared expert that every token
passes through. Run it on a GPU::

    python examples/fp8_moe_layer.py --tokens 64

All memory is allocated through PyTorch; every step of the arithmetic but the last
addition runs in the library's kernels.
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


@dataclasses.dataclass
class Fp8Weight:
    """e4m3 codes ``[..., N, K]`` with fp32 scales ``[..., ceil(N/128), ceil(K/128)]``."""
    codes: torch.Tensor
    scale: torch.Tensor


@dataclasses.dataclass
class Fp8MoeLayer:
    router: torch.Tensor        # fp32 [E, H]
    balance: torch.Tensor       # fp32 [E], moves the choice of experts only
    gate_up: Fp8Weight          # [E, 2I, H], gate rows first
    down: Fp8Weight             # [E, H, I]
    shared_gate_up: Fp8Weight   # [2S, H]
    shared_down: Fp8Weight      # [H, S]
    top_k: int
    n_group: int
    topk_group: int
    route_scale: float

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """bf16 ``[T, H]`` -> bf16 ``[T, H]``."""
        logits = x.float() @ self.router.T
        _, weights, offsets, row_token, row_of = w4.w4_moe_route_grouped(
            logits, self.top_k, bias=self.balance, n_group=self.n_group, topk_group=self.topk_group,
            scoring="sigmoid", renormalize=True, scale=self.route_scale)
        h = w4.w4_fp8_block_moe_gemm_bf16in(x, row_token, offsets, self.gate_up.codes, self.gate_up.scale)
        a, a_scale = w4.w4_silu_mul_quant_block(h)
        y = w4.w4_fp8_block_moe_grouped_gemm(a, a_scale, offsets, self.down.codes, self.down.scale)
        routed = w4.w4_moe_combine(y, weights, row_of)
        h = w4.w4_fp8_block_gemm_bf16in(x, self.shared_gate_up.codes, self.shared_gate_up.scale)
        a, a_scale = w4.w4_silu_mul_quant_block(h)
        return routed + w4.w4_fp8_block_gemm(a, a_scale, self.shared_down.codes, self.shared_down.scale)


def quantize_weight(w: torch.Tensor) -> Fp8Weight:
    """fp32 or bf16 ``[..., N, K]`` to e4m3 with one scale per 128 x 128 block (load
    time, plain PyTorch)."""
    *lead, N, K = w.shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    p = torch.zeros((*lead, nb * 128, kb * 128), dtype=torch.float32, device=w.device)
    p[..., :N, :K] = w
    p = p.view(*lead, nb, 128, kb, 128)
    s = p.abs().amax(dim=(-3, -1)) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (p / s[..., :, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).reshape(*lead, nb * 128, kb * 128)[..., :N, :K].contiguous()
    return Fp8Weight(q.view(torch.float8_e4m3fn), s)


def random_layer(H=512, I=256, S=384, E=16, top_k=4, n_group=4, topk_group=2, seed=0, device="cuda") -> Fp8MoeLayer:
    g = torch.Generator().manual_seed(seed)

    def weight(*shape):
        return quantize_weight((torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(device))

    return Fp8MoeLayer(router=(torch.randn((E, H), generator=g) * H ** -0.5).to(device),
                       balance=(0.1 * torch.randn((E,), generator=g)).to(device),
                       gate_up=weight(E, 2 * I, H), down=weight(E, H, I), shared_gate_up=weight(2 * S, H),
                       shared_down=weight(H, S), top_k=top_k, n_group=n_group, topk_group=topk_group, route_scale=2.5)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    layer = random_layer()
    x = torch.randn((a.tokens, layer.router.shape[1]), device="cuda").to(torch.bfloat16)
    y = layer(x)
    torch.cuda.synchronize()
    if w4.w4_device_status() != w4.W4_OK:
        raise SystemExit("a kernel reported an error")
    print(f"{a.tokens} tokens, {layer.router.shape[0]} experts, top {layer.top_k}: rms {y.float().square().mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
