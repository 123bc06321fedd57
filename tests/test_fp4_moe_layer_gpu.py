"""The example layer on 4-bit floating point experts: every stage held to the oracle on the
previous stage's GPU output, and the operators in the ways they may be called side by side:
on other streams, two at once, captured, and on tensors of the least alignment."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from _compare import check_bf16_output
from _gpu import bf16, bits, dev, requires_cuda, to_dev
from test_other_stream_gpu import on_side_stream

pytestmark = [pytest.mark.gpu, requires_cuda]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_moe_layer.py")
FORMATS = ["mxfp4", "nvfp4"]


def example():
    spec = importlib.util.spec_from_file_location("fp4_moe_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m          # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def number(t):
    return None if t is None else t.cpu().numpy().astype(np.float32)


def first(t):
    return None if t is None else np.float32(t.item())


def tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [17, 64, 700])
def test_many_tokens_stage_by_stage(fmt, T):
    layer = example().random_layer(format=fmt, seed=T)
    x = tokens(T, layer.router.shape[1], T)
    out = layer(x)
    logits = x.float() @ layer.router.T
    _, wts, off, rt, ro = w4.w4_moe_route_grouped(logits, layer.top_k, scoring="softmax")
    u, d, offn = layer.gate_up, layer.down, off.cpu().numpy()
    h = w4.w4_fp4_moe_gemm_bf16in(x, rt, off, u.codes, u.scale, fmt, layer.x_scale, u.tensor_scale)
    q, s = O.quant_fp4(bits(x)[rt.cpu().numpy()], fmt, first(layer.x_scale))
    check_bf16_output(bits(h), O.fp4_grouped_linear(q, s, offn, codes(u.codes), codes(u.scale), fmt, first(layer.x_scale),
                                                    number(u.tensor_scale)), "gate_up")
    a, sa = w4.w4_silu_mul_quant_fp4(h, fmt, layer.a_scale)
    y = w4.w4_fp4_moe_grouped_gemm(a, sa, off, d.codes, d.scale, fmt, layer.a_scale, d.tensor_scale)
    check_bf16_output(bits(y), O.fp4_grouped_linear(codes(a), codes(sa), offn, codes(d.codes), codes(d.scale), fmt,
                                                    first(layer.a_scale), number(d.tensor_scale)), "down")
    routed = w4.w4_moe_combine(y, wts, ro)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    assert torch.equal(out, routed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 16])
def test_few_tokens(fmt, T):
    """Bounds of an output as in the few-token layer's own tests: its rounding to bf16, and the
    activations' to 2^-13 of their block's largest."""
    layer = example().random_layer(format=fmt, seed=T)
    x = tokens(T, layer.router.shape[1], T)
    y = layer(x)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK

    def values(w):
        g = number(w.tensor_scale)
        return lambda e: O.dequant_fp4(codes(w.codes[e]), codes(w.scale[e]), fmt) * (1.0 if g is None else np.float64(g[e]))

    logits = (x.float() @ layer.router.T).cpu().numpy()
    _, _, gap = O.moe_route_grouped(logits, layer.top_k, scoring="softmax")
    clear = gap > 2.0 ** -20
    r, size = O.moe_decode(bits(x), logits, values(layer.gate_up), values(layer.down), layer.top_k, scoring="softmax")
    err = np.abs(y.float().cpu().numpy() - r)
    assert (err <= 2.0 ** -8 * np.abs(r) + 2.0 ** -10 * size)[clear].all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_captured_layer_of_either_kind(fmt):
    """One graph of a decode and a prefill call over shared weights, replayed on new tokens."""
    layer = example().random_layer(format=fmt)
    H = layer.router.shape[1]
    few, many = tokens(4, H, 1), tokens(40, H, 2)
    lf, lm = few.float() @ layer.router.T, many.float() @ layer.router.T
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(few, lf), layer.prefill(many, lm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = layer.decode(few, lf), layer.prefill(many, lm)
    few.copy_(tokens(4, H, 3)), many.copy_(tokens(40, H, 4))
    lf.copy_(few.float() @ layer.router.T), lm.copy_(many.float() @ layer.router.T)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, layer.decode(few, lf)) and torch.equal(b, layer.prefill(many, lm))


@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_on_another_stream(fmt):
    """What the binding allocates for them is theirs until their kernels are done."""
    layer = example().random_layer(format=fmt)
    H, T, k = layer.router.shape[1], 40, layer.top_k
    I, block = layer.down.codes.shape[2] * 2, O.FP4_BLOCK[fmt]
    x = tokens(T, H, 1)
    lg = x.float() @ layer.router.T
    _, _, off, rt, _ = w4.w4_moe_route_grouped(lg, k, scoring="softmax")
    u, d = layer.gate_up, layer.down
    up = lambda **kw: w4.w4_fp4_moe_gemm_bf16in(x, rt, off, u.codes, u.scale, fmt, layer.x_scale, u.tensor_scale, **kw)  # noqa: E731
    ref = up()
    y = on_side_stream(lambda st: up(stream=st), [w4.w4_workspace_bytes(w4.W4_OP_FP4_MOE_IN, T * k, 2 * I, H, block), 4 * T * k * I])
    assert torch.equal(y, ref)
    tensor_scale = None if u.tensor_scale is None else u.tensor_scale[:1]
    dense = lambda **kw: w4.w4_fp4_gemm_bf16in(x, u.codes[0], u.scale[0], fmt, layer.x_scale, tensor_scale, **kw)  # noqa: E731
    ref = dense()
    y = on_side_stream(lambda st: dense(stream=st), [w4.w4_workspace_bytes(w4.W4_OP_FP4_IN, T, 2 * I, H, block), 4 * T * I])
    assert torch.equal(y, ref)
    rq, rs = w4.w4_quant_fp4(x, fmt, layer.x_scale)
    q, s = on_side_stream(lambda st: w4.w4_quant_fp4(x, fmt, layer.x_scale, stream=st), [rq.numel(), rs.numel()])
    np.testing.assert_array_equal(codes(q), codes(rq))
    np.testing.assert_array_equal(codes(s), codes(rs))
    few, lf = x[:9].contiguous(), lg[:9].contiguous()
    dec = lambda **kw: w4.w4_moe_decode(few, lf, u.codes, u.scale, d.codes, d.scale, k, fmt, u.tensor_scale, d.tensor_scale,  # noqa: E731
                                        scoring="softmax", **kw)
    ref = dec()
    y = on_side_stream(lambda st: dec(stream=st), [w4.w4_workspace_bytes(w4.W4_OP_MOE_DECODE, 9, k, I, 0), 2 * 9 * H])
    assert torch.equal(y, ref)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_calls_at_once(fmt):
    layer = example().random_layer(format=fmt)
    H = layer.router.shape[1]
    xs = [tokens(n, H, n) for n in (3, 16, 33, 200)]
    logits = [x.float() @ layer.router.T for x in xs]
    run = lambda i: layer.decode(xs[i], logits[i]) if i < 2 else layer.prefill(xs[i], logits[i])  # noqa: E731
    ref = [run(i) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs.append((i, run(i)))
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    assert all(torch.equal(y, ref[i]) for i, y in outs)


def shifted(a, by):
    """A copy of a CPU or device tensor ``by`` bytes behind a 256-byte boundary."""
    t = a if isinstance(a, torch.Tensor) else to_dev(a)
    n = t.numel() * t.element_size()
    room = torch.empty(n + 256, dtype=torch.uint8, device=dev())
    at = room[by:by + n].view(t.dtype).view(t.shape)
    at.copy_(t)
    assert at.data_ptr() % 256 == by
    return at


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 5, 20, 100, 150, 400])
def test_least_alignment(fmt, M):
    """Matrices at 16 bytes and no more, scales at 4: the same numbers as on aligned tensors."""
    N, K = 328, 896
    x = bf16(S.activations_bf16(M, K, seed=M))
    w = bf16(S.activations_bf16(N, K, seed=3))
    q, s = w4.w4_quant_fp4(x, fmt)
    qw, sw = w4.w4_quant_fp4(w, fmt)
    q, s, qw, sw = (t.view(torch.uint8) for t in (q, s, qw, sw))
    ref = w4.w4_fp4_gemm(q, s, qw, sw, fmt)
    check_bf16_output(bits(ref), O.fp4_linear(codes(q), codes(s), codes(qw), codes(sw), fmt), fmt)
    y = shifted(torch.zeros_like(ref), 16)
    w4.w4_fp4_gemm(shifted(q, 16), shifted(s, 4), shifted(qw, 48), shifted(sw, 12), fmt, y=y)
    assert torch.equal(y, ref)
    assert torch.equal(w4.w4_fp4_gemm_bf16in(shifted(x, 16), shifted(qw, 16), shifted(sw, 4), fmt), ref)
    q2, s2 = shifted(torch.zeros_like(q), 16), shifted(torch.zeros_like(s), 1)
    w4.w4_quant_fp4(shifted(x, 16), fmt, q=q2, scale=s2)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    off = to_dev(np.array([0, M // 3, M // 3, M], np.int32))
    qe, se = qw[None].repeat(3, 1, 1), sw[None].repeat(3, 1, 1)
    y = w4.w4_fp4_moe_grouped_gemm(shifted(q, 16), shifted(s, 8), shifted(off, 4), shifted(qe, 16), shifted(se, 4), fmt)
    assert torch.equal(y, w4.w4_fp4_moe_grouped_gemm(q, s, off, qe, se, fmt))
    check_bf16_output(bits(y), O.bf16_to_f64(bits(ref)), fmt)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK


def test_refusals():
    """Shapes and types that the binding turns away before any launch."""
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=dev())
    q, s = w4.w4_quant_fp4(x, "mxfp4")
    w, ws = torch.zeros((64, 128), dtype=torch.uint8, device=dev()), torch.zeros((64, 8), dtype=torch.uint8, device=dev())
    ok = w4.w4_fp4_gemm(q, s, w, ws, "mxfp4")
    assert ok.shape == (4, 64)
    g1 = torch.ones(1, device=dev())
    off = torch.zeros(3, dtype=torch.int32, device=dev())
    we, wse = w[None].repeat(2, 1, 1), ws[None].repeat(2, 1, 1)
    lg = torch.zeros((4, 2), device=dev())
    wd, wds = torch.zeros((2, 256, 16), dtype=torch.uint8, device=dev()), torch.zeros((2, 256, 1), dtype=torch.uint8, device=dev())
    for call in (lambda: w4.w4_quant_fp4(x.float(), "mxfp4"),
                 lambda: w4.w4_quant_fp4(x, "mxfp4", q=q[:3]),
                 lambda: w4.w4_quant_fp4(x, "mxfp4", scale=s[:, :4]),
                 lambda: w4.w4_quant_fp4(x.t(), "mxfp4"),                      # not contiguous
                 lambda: w4.w4_quant_fp4(x, "nvfp4", torch.ones(2, device=dev())),
                 lambda: w4.w4_quant_fp4(x, "nvfp4", g1.double()),
                 lambda: w4.w4_silu_mul_quant_fp4(x.to(torch.float16), "mxfp4"),
                 lambda: w4.w4_dequant_fp4(q, s, "nvfp4"),                      # scales of the other block
                 lambda: w4.w4_fp4_gemm(q, s[:3], w, ws, "mxfp4"),
                 lambda: w4.w4_fp4_gemm(q, s, w[:, :64], ws, "mxfp4"),
                 lambda: w4.w4_fp4_gemm(q, s, w, ws[:, :4], "mxfp4"),
                 lambda: w4.w4_fp4_gemm(q, s, w, ws, "mxfp4", bias=torch.zeros(8, dtype=torch.bfloat16, device=dev())),
                 lambda: w4.w4_fp4_gemm(q, s, w, ws, "mxfp4", y=ok[:, :32]),
                 lambda: w4.w4_fp4_moe_grouped_gemm(q, s, off[:2], we, wse, "mxfp4"),
                 lambda: w4.w4_fp4_moe_grouped_gemm(q, s, off, we, ws, "mxfp4"),
                 lambda: w4.w4_fp4_moe_gemm_bf16in(x, off.long(), off, we, wse, "mxfp4"),
                 lambda: w4.w4_moe_decode(x, lg[:3], we, wse, wd, wds, 1, "mxfp4"),
                 lambda: w4.w4_moe_decode(x, lg, we, wse, wd[:1], wds, 1, "mxfp4"),
                 lambda: w4.w4_moe_decode(x, lg, we, wse, wd, wds, 1, "int4"),
                 lambda: w4.w4_moe_decode(x, lg, we, wse, wd, wds, 1, "mxfp4", bias=lg[0, :1])):
        with pytest.raises(ValueError):
            call()
    room = torch.zeros(w4.w4_workspace_bytes(w4.W4_OP_FP4_IN, 40, 64, 256, 32), dtype=torch.uint8, device=dev())
    for call in (lambda: w4.w4_quant_fp4(x, "mxfp4", g1),                       # refused by the library
                 lambda: w4.w4_moe_decode(x, lg, we, wse, wd, wds, 1, "mxfp4"),  # 2I = 64: I is no multiple of 64
                 lambda: w4.w4_fp4_gemm_bf16in(x.repeat(10, 1), w, ws, "mxfp4", workspace=shifted(room, 8))):
        with pytest.raises((RuntimeError, ValueError)):
            call()
