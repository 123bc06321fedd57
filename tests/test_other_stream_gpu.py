"""Calls on a stream that is not the current one, with outputs and workspace left to the
binding: what it allocates belongs to the call's stream until its kernels are done."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import synthetic as S
from _gpu import bf16, bits, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def fp8(a):
    return to_dev(a).view(torch.float8_e4m3fn)


def weights(N, K, seed=1, E=None):
    """Random e4m3 codes of magnitude up to 1 and block scales around 0.02."""
    lead = () if E is None else (E,)
    q = S.fp8_codes(lead + (N, K), seed=seed)
    q = (q & 0x80) | (q & 0x7F) % 0x39
    s = S.scales_f16(lead + (-(-N // 128), -(-K // 128)), seed=seed + 1).astype(np.float32)
    return q.astype(np.uint8), s


def on_side_stream(call, refill, held_ms=60):
    """The outputs of ``call(stream)`` on a side stream that is busy when it is made, while the
    current stream allocates and overwrites memory of the sizes ``refill`` (bytes) meanwhile."""
    side = torch.cuda.Stream()
    torch.empty(16, dtype=torch.uint8, device="cuda").fill_(0xFF)   # a kernel's first launch waits for the device
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(held_ms * 2e6))
    out = call(side)
    kept = []
    for n in refill:
        for _ in range(4):
            kept.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
            kept[-1].fill_(0xFF)
    torch.cuda.current_stream().synchronize()
    assert not side.query()          # the call had not even begun when the memory was written
    side.synchronize()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("M,N,K", [(24, 1032, 1408), (300, 4096, 4112)])
def test_scratch_of_a_call_on_another_stream(M, N, K):
    """Codes, scales and part sums that the binding allocates for a call on another
    stream stay the call's until its kernels are done."""
    x = S.activations_bf16(M, K, seed=M)
    qw, sw = weights(N, K, seed=3)
    t, wd, sd = bf16(x), fp8(qw), to_dev(sw)
    q, s = w4.w4_quant_act_per_block(t)
    ref, ref_q = w4.w4_fp8_block_gemm_bf16in(t, wd, sd), w4.w4_fp8_block_gemm(q, s, wd, sd)
    need = w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, M, N, K, 0)
    parts = w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK, M, N, K, 0)
    y = on_side_stream(lambda st: w4.w4_fp8_block_gemm_bf16in(t, wd, sd, stream=st), [need, 2 * M * N])
    np.testing.assert_array_equal(bits(y), bits(ref))
    y = on_side_stream(lambda st: w4.w4_fp8_block_gemm(q, s, wd, sd, stream=st), [max(parts, 16), 2 * M * N])
    np.testing.assert_array_equal(bits(y), bits(ref_q))
    qs, ss = on_side_stream(lambda st: w4.w4_quant_act_per_block(t, stream=st), [M * K, 4 * s.numel()])
    np.testing.assert_array_equal(codes(qs), codes(q))
    np.testing.assert_array_equal(ss.cpu().numpy(), s.cpu().numpy())


def test_scratch_of_routing_and_experts_on_another_stream():
    T, E, k, N, K = 1000, 64, 4, 136, 400
    lg, x = to_dev(S.router_logits(T, E, seed=1)), bf16(S.activations_bf16(T, K, seed=2))
    qw, sw = weights(N, K, seed=3, E=E)
    wd, sd = fp8(qw), to_dev(sw)
    ref = w4.w4_moe_route_grouped(lg, k, n_group=4, topk_group=2)
    ref_y = w4.w4_fp8_block_moe_gemm_bf16in(x, ref[3], ref[2], wd, sd)
    table = w4.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE_GROUPED, T, E, 1, 0)
    out = on_side_stream(lambda st: w4.w4_moe_route_grouped(lg, k, n_group=4, topk_group=2, stream=st),
                         [table, 16 * T * k + 4 * (E + 1)])
    for a, b in zip(out, ref):
        np.testing.assert_array_equal(a.cpu().numpy(), b.cpu().numpy())
    need = w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, T * k, N, K, E)
    y = on_side_stream(lambda st: w4.w4_fp8_block_moe_gemm_bf16in(x, ref[3], ref[2], wd, sd, stream=st),
                       [need, 2 * T * k * N])
    np.testing.assert_array_equal(bits(y), bits(ref_y))


def test_outputs_of_a_call_on_another_stream_read_on_the_current_one():
    """An output released on the current stream, whose reader is still queued there, is not
    handed to the next call on the side stream."""
    M, N, K = 40, 520, 400
    qw, sw = weights(N, K, seed=3)
    wd, sd = fp8(qw), to_dev(sw)
    a, b = bf16(S.activations_bf16(M, K, seed=1)), bf16(S.activations_bf16(M, K, seed=2))
    ref = w4.w4_fp8_block_gemm_bf16in(a, wd, sd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = w4.w4_fp8_block_gemm_bf16in(a, wd, sd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(int(40e6))
    copy = y.clone()                 # queued behind the sleep
    del y
    for _ in range(4):
        w4.w4_fp8_block_gemm_bf16in(b, wd, sd, stream=side)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(copy), bits(ref))


def test_scratch_of_the_int4_layers_on_another_stream():
    M, N, K, g, E = 300, 520, 1024, 128, 4
    xb = S.activations_bf16(M, K, seed=1)
    x = bf16(xb)
    qw, sw = to_dev(S.random_words((K // 8, N), seed=2)), to_dev(S.scales_f16((K // g, N), seed=3))
    qe, se = to_dev(S.random_words((E, N, K // 8), seed=4)), to_dev(S.scales_f16((E, N, K // g), seed=5))
    off = to_dev(np.array([0, 100, 100, 290, M], np.int32))
    lg = to_dev(S.router_logits(5000, 64, seed=6))
    need = w4.w4_workspace_bytes(w4.W4_OP_W4A8, M, N, K, g)
    ref, ref_s = w4.w4a8_gemm_bf16in(x, qw, sw, g)
    y, s = on_side_stream(lambda st: w4.w4a8_gemm_bf16in(x, qw, sw, g, stream=st), [need, 2 * M * N, 4 * M])
    np.testing.assert_array_equal(bits(y), bits(ref))
    np.testing.assert_array_equal(s.cpu().numpy(), ref_s.cpu().numpy())
    need = w4.w4_workspace_bytes(w4.W4_OP_W4AFP8_MOE, M, N, K, g)
    ref, _ = w4.w4afp8_moe_gemm_bf16in(x, None, off, qe, se, g)
    y, _ = on_side_stream(lambda st: w4.w4afp8_moe_gemm_bf16in(x, None, off, qe, se, g, stream=st), [need, 2 * M * N, 4 * M])
    np.testing.assert_array_equal(bits(y), bits(ref))
    need = w4.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE, 5000, 64, 1, 0)
    ref = w4.w4_moe_route(lg, 6)
    out = on_side_stream(lambda st: w4.w4_moe_route(lg, 6, stream=st), [need, 4 * 5000 * 6, 4 * 65])
    for a, b in zip(out, ref):
        np.testing.assert_array_equal(a.cpu().numpy(), b.cpu().numpy())
    # a layer whose activations are a transposed view of what the side stream makes
    side = torch.cuda.Stream()
    made = torch.zeros((2, M // 2, K), dtype=torch.bfloat16, device="cuda")
    src = x.view(2, M // 2, K)
    ref = w4.apply_weights(src.transpose(0, 1).contiguous(), qw, sw, g)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(40e6))
        made.copy_(src)
    y = w4.apply_weights(made.transpose(0, 1), qw, sw, g, stream=side)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y), bits(ref))
