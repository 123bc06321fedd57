"""The microscaled 4-bit floating point layer against the float64 oracle.

Quantized codes and scales are whole numbers and have to be equal, but where silu is
in between: there fp32 steps and float64 may put a value on different sides of a border.
Products of codes are exact and sums are taken in fp32, so that outputs meet the bar of
every bf16 output (tests/_compare.py: one rounding is at most 2^-8 of a value, the bar is two of
them, and the sum's error a hundredth of one)."""
import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from tests._compare import check_bf16_output
from tests._gpu import bf16, bits, dev, requires_cuda, to_dev

pytestmark = [pytest.mark.gpu, requires_cuda]

FORMATS = ["mxfp4", "nvfp4"]
STEP = {"mxfp4": 128, "nvfp4": 64}


def host(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def scalar(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device=dev())


def act(M, K, seed=0):
    return S.activations_bf16(M, K, seed=seed, outlier_frac=0.01)


def g_of(fmt, xb):
    return np.float32(np.abs(O.bf16_to_f64(xb)).max() / (6 * 448)) if fmt == "nvfp4" else None


def weights(shape, fmt, seed=1):
    """Codes of every kind, scales around 2^-6, a scale per tensor."""
    *lead, N, K = shape
    q = S.fp8_codes((*lead, N, K // 2), seed=seed)
    raw = S.fp8_codes((*lead, N, K // O.FP4_BLOCK[fmt]), seed=seed + 1)
    s = (118 + raw % 7).astype(np.uint8) if fmt == "mxfp4" else (0x20 + raw % 0x30).astype(np.uint8)
    return q, s, None if fmt == "mxfp4" else np.float32(0.013)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 1408), (129, 2048), (1, 8192), (67, 4064)])
@pytest.mark.parametrize("f16", [False, True])
def test_quant_is_bit_exact(fmt, M, K, f16):
    xb = act(M, K, seed=M + K)
    g = g_of(fmt, xb)
    if f16:
        x = O.bf16_to_f64(xb).astype(np.float16)
        q, s = w4.w4_quant_fp4(to_dev(x), fmt, scalar(g))
        rq, rs = O.quant_fp4(x, fmt, g)
    else:
        q, s = w4.w4_quant_fp4(bf16(xb), fmt, scalar(g))
        rq, rs = O.quant_fp4(xb, fmt, g)
    assert np.array_equal(host(s).reshape(rs.shape), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("g", [None, 1e-3, 3e-38, 2e30])
def test_quant_of_extreme_values(fmt, g):
    """Zeros and -0, ties, subnormals, the largest numbers, scales that vanish or hold at 448."""
    if fmt == "mxfp4" and g is not None:
        pytest.skip("mxfp4 has no scale per tensor")
    rows = [np.zeros(64), -np.zeros(64), np.resize([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 64),
            np.resize([1e-39, -3e-39, 9e-41, 2e-38], 64), np.full(64, 3.3e38), np.resize([1.0, 1e-30, -2e-7, 0.0], 64),
            np.resize([-6.0, 0.5, 7.5, 0.26], 64), np.resize([1e30, 1e28, -4e29, 0.0], 64), np.resize([2.0 ** -126, 2.0 ** -133], 64)]
    xb = S.to_bf16_bits(np.stack(rows))
    q, s = w4.w4_quant_fp4(bf16(xb), fmt, scalar(g))
    rq, rs = O.quant_fp4(xb, fmt, g)
    assert np.array_equal(host(s).reshape(rs.shape), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_with_nan_or_infinity_gets_a_nan_scale(fmt, bad):
    x = O.bf16_to_f64(act(4, 128, seed=3)).astype(np.float32)
    x[2, 40] = bad
    xb = bf16(S.to_bf16_bits(x))
    q, s = w4.w4_quant_fp4(xb, fmt)
    rq, rs = O.quant_fp4(S.to_bf16_bits(x), fmt)
    assert np.array_equal(host(s).reshape(rs.shape), rs) and np.array_equal(host(q), rq)
    out = w4.w4_dequant_fp4(q, s, fmt)
    b = O.FP4_BLOCK[fmt]
    nan = torch.isnan(out.float()).cpu().numpy()
    assert nan[2, 40 // b * b:40 // b * b + b].all() and nan.sum() == b
    qw, sw, gw = weights((16, 128), fmt)
    y = w4.w4_fp4_gemm(q, s, to_dev(qw), to_dev(sw), fmt, None, scalar(gw)).float().cpu().numpy()
    assert np.isnan(y[2]).all() and np.isfinite(y[[0, 1, 3]]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R,I", [(1, 32), (7, 1408), (130, 704)])
def test_silu_mul_quant(fmt, R, I):
    hb = S.activations_bf16(R, 2 * I, seed=R)
    g = np.float32(0.004) if fmt == "nvfp4" else None
    q, s = w4.w4_silu_mul_quant_fp4(bf16(hb), fmt, scalar(g))
    rq, rs = O.silu_mul_quant_fp4(hb, fmt, g)
    # fp32 steps are within 4 roundings (2^-22) of float64: one value in 2^18 may lie that near a border
    assert np.mean(host(s).reshape(rs.shape) != rs) <= 1e-3
    a, r = O.fp4_unpack(host(q)).astype(int), O.fp4_unpack(rq).astype(int)
    assert np.mean(a != r) <= 1e-3


def test_silu_mul_quant_of_far_gates():
    """Gates far out: the formula's zeros and infinities, NaN blocks for what is not finite."""
    h = np.zeros((1, 256), np.float32)
    h[0, :5] = [-1000.0, -90.0, 1e30, 200.0, -87.0]
    h[0, 128:133] = [3.0, 1.0, 2.0, -5.0, 1e38]
    h[0, 64], h[0, 192] = 3e38, 3e38
    q, s = w4.w4_silu_mul_quant_fp4(bf16(S.to_bf16_bits(h)), "mxfp4")
    assert host(s).tolist()[0][1:] == [0, 255, 0]
    assert O.fp4_decode(host(q))[0, 2] > 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_dequant_is_the_rounded_value(fmt, dtype):
    qw, sw, _ = weights((37, 352), fmt, seed=5)
    g = np.float32(0.37) if fmt == "nvfp4" else None
    out = w4.w4_dequant_fp4(to_dev(qw), to_dev(sw), fmt, scalar(g), dtype=dtype)
    d = O.fp4_scale_decode(sw, fmt)
    if g is not None:
        d = (d.astype(np.float32) * g).astype(np.float64)
    v = (O.fp4_decode(qw).reshape(*d.shape, -1) * d[..., None]).reshape(37, 352).astype(np.float32)
    assert torch.equal(out.cpu(), torch.from_numpy(v).to(dtype))


def check_linear(M, N, K, fmt, bias=False, seed=0):
    xb = act(M, K, seed=seed)
    gx = g_of(fmt, xb)
    qx, sx = O.quant_fp4(xb, fmt, gx)
    qw, sw, gw = weights((N, K), fmt, seed=seed + 1)
    bb = S.bias_bf16(N) if bias else None
    b = bf16(bb) if bias else None
    y = w4.w4_fp4_gemm(to_dev(qx), to_dev(sx), to_dev(qw), to_dev(sw), fmt, scalar(gx), scalar(gw), bias=b)
    again = w4.w4_fp4_gemm_bf16in(bf16(xb), to_dev(qw), to_dev(sw), fmt, scalar(gx), scalar(gw), bias=b)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(y), O.fp4_linear(qx, sx, qw, sw, fmt, gx, gw, bb), f"{fmt} {M}x{N}x{K}")
    assert torch.equal(y, again)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300])
def test_linear_of_any_number_of_rows(fmt, M):
    check_linear(M, 264, 640, fmt, seed=M)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,k", [(8, 1), (136, 2), (1000, 3), (2816, 11), (200, 16), (4096, 33)])
@pytest.mark.parametrize("M", [3, 40, 150])
def test_linear_of_ragged_sizes(fmt, M, N, k):
    check_linear(M, N, k * STEP[fmt], fmt, bias=N % 16 == 8, seed=k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_of_many_tiles(fmt):
    """More tiles than SMs: accumulators and ring go around."""
    check_linear(700, 9000, 1024, fmt, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_scale_reaches_its_block(fmt):
    """One weight block and one activation block at a time is not zero."""
    b, K, M, N = O.FP4_BLOCK[fmt], 512, 130, 200
    for form in (M, 5):
        qx = np.full((form, K // 2), 0x22, np.uint8)           # ones
        qw = np.full((N, K // 2), 0x22, np.uint8)
        one = 127 if fmt == "mxfp4" else 0x38
        r = np.arange(max(form, N))[:, None] * 7 + np.arange(K // b)[None] * 3
        sx, sw = (one + (r[:form] % 5)).astype(np.uint8), (one + (r[:N] % 4)).astype(np.uint8)
        y = w4.w4_fp4_gemm(to_dev(qx), to_dev(sx), to_dev(qw), to_dev(sw), fmt)
        check_bf16_output(bits(y), O.fp4_linear(qx, sx, qw, sw, fmt), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[7, 0, 9, 1], [0, 0, 40], [130, 1, 0, 70, 300], [1]])
def test_experts(fmt, counts):
    E, N, K = len(counts), 328, 384
    off = S.offsets_from_counts(counts)
    R = int(off[-1])
    xb = act(max(R // 2, 1), K, seed=R)
    gx = g_of(fmt, xb)
    rows = (np.arange(R) * 5 % xb.shape[0]).astype(np.int32)
    qw, sw, _ = weights((E, N, K), fmt, seed=3)
    gw = np.linspace(0.01, 0.03, E).astype(np.float32) if fmt == "nvfp4" else None
    gwd = None if gw is None else to_dev(gw)
    y = w4.w4_fp4_moe_gemm_bf16in(bf16(xb), to_dev(rows), to_dev(off), to_dev(qw), to_dev(sw), fmt, scalar(gx), gwd)
    qx, sx = O.quant_fp4(xb[rows], fmt, gx)
    z = w4.w4_fp4_moe_grouped_gemm(to_dev(qx), to_dev(sx), to_dev(off), to_dev(qw), to_dev(sw), fmt, scalar(gx), gwd)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(y), O.fp4_grouped_linear(qx, sx, off, qw, sw, fmt, gx, gw), fmt)
    assert torch.equal(y, z)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_no_expert_are_left_as_they_were(fmt):
    N, K, R = 136, 256, 50
    qw, sw, gw = weights((3, N, K), fmt)
    qx, sx = O.quant_fp4(act(R, K), fmt)
    off = np.array([4, 20, 20, 41], np.int32)
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=dev())
    w4.w4_fp4_moe_grouped_gemm(to_dev(qx), to_dev(sx), to_dev(off), to_dev(qw), to_dev(sw), fmt, y=y)
    ref = O.fp4_grouped_linear(qx, sx, off, qw, sw, fmt)
    check_bf16_output(bits(y)[4:41], ref[4:41], fmt)
    assert (y[:4] == 7).all() and (y[41:] == 7).all()


def test_token_ids_out_of_range_give_zero_rows():
    qw, sw, _ = weights((1, 64, 128), "mxfp4")
    rows = to_dev(np.array([0, 5, -1, 1], np.int32))
    y = w4.w4_fp4_moe_gemm_bf16in(bf16(act(2, 128)), rows, to_dev(np.array([0, 4], np.int32)), to_dev(qw), to_dev(sw), "mxfp4")
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_ERR_SHAPE
    assert (y[1:3] == 0).all() and (y[[0, 3]] != 0).any()


def test_no_rows():
    qw, sw, _ = weights((2, 64, 128), "mxfp4")
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=dev())
    assert w4.w4_quant_fp4(x, "mxfp4")[0].shape == (0, 64)
    assert w4.w4_fp4_gemm_bf16in(x, to_dev(qw[0]), to_dev(sw[0]), "mxfp4").shape == (0, 64)
    rows = torch.empty((0,), dtype=torch.int32, device=dev())
    off = torch.zeros((3,), dtype=torch.int32, device=dev())
    assert w4.w4_fp4_moe_gemm_bf16in(x, rows, off, to_dev(qw), to_dev(sw), "mxfp4").shape == (0, 64)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_chain_without_synchronization_equals_the_calls_with_it(fmt):
    """A weight quantized right before its products, captured into a graph and replayed on new inputs."""
    N, K, M = 512, 1024, 9
    w = bf16(S.to_bf16_bits(0.02 * S.normal(1, 1, N * K).reshape(N, K)))
    xs = [bf16(act(M, K, seed=i)) for i in range(4)]
    h = torch.empty((M, N), dtype=torch.bfloat16, device=dev())
    x = xs[0].clone()
    out = torch.empty((M, N // 2), dtype=torch.bfloat16, device=dev())

    def chain():
        q, s = w4.w4_quant_fp4(w, fmt)
        w4.w4_fp4_gemm_bf16in(x, q, s, fmt, y=h)
        qa, sa = w4.w4_silu_mul_quant_fp4(h, fmt)
        w4.w4_fp4_gemm(qa, sa, q[:N // 2, :N // 4].contiguous(), s[:N // 2, :s.shape[1] * N // (2 * K)].contiguous(), fmt, y=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for i in (1, 2, 3):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        chain()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        q, s = w4.w4_quant_fp4(w, fmt)
        torch.cuda.synchronize()
        qx, sx = w4.w4_quant_fp4(x, fmt)
        check_bf16_output(bits(h), O.fp4_linear(host(qx), host(sx), host(q), host(s), fmt), "chain")


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_quantized_once_give_the_same_rows(fmt):
    """Enough rows for the copy of the tokens' codes: as with a workspace that has no room for it."""
    T, k, E, N, K = 700, 8, 6, 64, 2048
    xb = act(T, K, seed=1)
    gx = g_of(fmt, xb)
    rows = (np.arange(T * k) * 13 % T).astype(np.int32)
    rows[5], rows[9] = T, -3
    off = S.offsets_from_counts([T * k // 2, 0, 100, T * k // 2 - 300, 200, 0])
    qw, sw, _ = weights((E, N, K), fmt)
    call = lambda **kw: w4.w4_fp4_moe_gemm_bf16in(bf16(xb), to_dev(rows), to_dev(off), to_dev(qw), to_dev(sw), fmt, scalar(gx), **kw)  # noqa: E731
    y = call()
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_ERR_SHAPE
    small = torch.empty(w4.w4_workspace_bytes(w4.W4_OP_FP4_IN, T * k, N, K, O.FP4_BLOCK[fmt]), dtype=torch.uint8, device=dev())
    z = call(workspace=small)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_ERR_SHAPE
    assert torch.equal(y, z) and (y[[5, 9]] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,k", [(257, 5000, 1), (513, 2696, 7), (900, 2056, 16), (1300, 1992, 3)])
def test_linear_of_many_rows(fmt, M, N, k):
    """Pairs of CTAs: rows and outputs that end inside a tile, a second CTA with no rows, odd numbers of stages."""
    check_linear(M, N, k * STEP[fmt], fmt, bias=M % 2 == 0, seed=M)


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_of_rows_that_fill_fewer_tiles_than_pairs(fmt):
    check_linear(517, 11008, STEP[fmt], fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,k", [(300, 264, 33), (390, 1000, 16), (200, 2048, 20)])
def test_linear_of_few_weight_tiles(fmt, M, N, k):
    """Clusters that cut k among more rows than one tile holds."""
    check_linear(M, N, k * STEP[fmt], fmt, bias=True, seed=k)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[600, 0, 3, 470], [1, 1025], [255, 257, 129, 384]])
def test_experts_of_many_rows(fmt, counts):
    test_experts(fmt, counts)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(2101, 4064), (8193, 1024)])
def test_quant_of_many_elements_is_bit_exact(fmt, M, K):
    """Several blocks a thread, and a last warp with some of its threads' second ones."""
    test_quant_is_bit_exact(fmt, M, K, False)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(4096, 11008, 4096), (700, 4096, 4096), (100, 4096, 2048), (5, 4096, 4096)])
def test_chains_of_calls_give_the_same_bits(fmt, M, N, K):
    """A product that starts while its quantizer still runs finds its first stages all there at once."""
    qw, sw, gw = weights((N, K), fmt)
    qw, sw, gw = to_dev(qw), to_dev(sw), scalar(gw)
    xs = [torch.randn((M, K), device=dev(), generator=torch.Generator(dev()).manual_seed(i)).to(torch.bfloat16) for i in range(3)]
    gx = scalar(np.float32(6.0 / (6 * 448))) if fmt == "nvfp4" else None
    ref = []
    for x in xs:
        q, s = w4.w4_quant_fp4(x, fmt, gx)
        torch.cuda.synchronize()
        ref.append(w4.w4_fp4_gemm(q, s, qw, sw, fmt, gx, gw))
        torch.cuda.synchronize()
    for _ in range(40):
        ys = [w4.w4_fp4_gemm_bf16in(xs[i % 3], qw, sw, fmt, gx, gw) for i in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, ref[i % 3]) for i, y in enumerate(ys))
    assert w4.w4_device_status() == w4.W4_OK
