"""The fp8 block-scaled layer on the GPU against the oracle, through the C ABI:
per-block quantization, silu * up requantization, the dense product in both its
forms, and the product over expert segments."""
import ctypes

import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
import synthetic as S
from _compare import check_bf16_output
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
    s = S.scales_f16(lead + (-(-N // 128), -(-K // 128)), seed=seed + 1).astype(np.float32) * np.float32(1.0001)
    return q.astype(np.uint8), s


def rows(M, K, seed=0):
    x = S.activations_bf16(M, K, seed=seed, outlier_frac=0.01)
    q, s = O.quant_fp8_per_block(x)
    return x, q, s


# ---- quantizers -------------------------------------------------------------

@pytest.mark.parametrize("M,K", [(1, 8), (3, 16), (1, 128), (2, 136), (7, 264), (5, 504), (129, 1408), (33, 4096),
                                 (1, 8200), (1031, 520)])
@pytest.mark.parametrize("f16", [False, True])
def test_quant_per_block_bit_exact(M, K, f16):
    """Codes and scales, with a zero row and a zero block among them."""
    if f16:
        x = S.bf16_bits_to_f32(S.activations_bf16(M, K, seed=K)).astype(np.float16)
        x[M // 2, :128] = 0
        t = to_dev(x)
    else:
        x = S.activations_bf16(M, K, seed=K, outlier_frac=0.02)
        x[M // 2, :128] = 0
        t = bf16(x)
    q, s = w4.w4_quant_act_per_block(t)
    torch.cuda.synchronize()
    rq, rs = O.quant_fp8_per_block(x)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes(q), rq)


def test_quant_per_block_extremes():
    """Blocks of subnormals, of the largest bf16 values, and of equal magnitudes."""
    x = np.zeros((4, 256), np.uint16)
    x[0, :128] = S.raw_u64(3, 1, 128) % 128                      # bf16 subnormals
    x[0, 128:] = 0x7F7F                                          # the largest finite value
    x[1, :] = np.where(np.arange(256) % 2, 0x8001, 0x0001)       # the smallest subnormal, both signs
    x[2, ::3] = 0x3F80
    x[3, :] = S.activations_bf16(1, 256, seed=9, std=1e-30)[0]
    q, s = w4.w4_quant_act_per_block(bf16(x))
    torch.cuda.synchronize()
    rq, rs = O.quant_fp8_per_block(x)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    keep = rs.repeat(128, axis=1) > 0                            # a scale that underflowed to 0 divides by 0
    np.testing.assert_array_equal(codes(q)[keep], rq[keep])


@pytest.mark.parametrize("R,I", [(1, 8), (3, 128), (5, 200), (64, 1408), (1000, 136)])
def test_silu_mul_quant_block(R, I):
    """fp32 silu with the fast exponential is within 2^-19 of the definition
    where it matters, so scales are within 2^-19 and a code moves by one step at
    most, on few elements."""
    h = S.activations_bf16(R, 2 * I, seed=R + I, std=3.0)
    h[R // 2] = 0
    q, s = w4.w4_silu_mul_quant_block(bf16(h))
    torch.cuda.synchronize()
    act = O.silu_mul_f64(h).astype(np.float32)
    for b in range(-(-I // 128)):
        c = slice(b * 128, min(I, (b + 1) * 128))
        amax = np.abs(act[:, c]).max(axis=1)
        rs = np.where(amax == 0, 1.0, amax.astype(np.float64) / 448)
        np.testing.assert_allclose(s.cpu().numpy()[:, b], rs, rtol=2.0 ** -19)
        ref = O.e4m3_encode(act[:, c].astype(np.float64) / rs[:, None]).astype(np.int64)
        got = codes(q)[:, c].astype(np.int64)
        same_sign = ((ref ^ got) & 0x80) == 0
        step = np.abs((ref & 0x7F) - (got & 0x7F))
        assert np.all((step <= 1) & (same_sign | (step + (ref & 0x7F) <= 1)))
        assert np.mean(step == 0) >= 0.999 or step.sum() <= 1


def test_silu_mul_quant_block_far_gates():
    """Gates far below zero give 0, however large they or `up` are; only the
    product itself overflows; NaN and infinite gates stay in their block."""
    g = torch.tensor([-90.0, -1000.0, -1e30, -3e38, 1.0, 2.0, 0.0, -0.0]).repeat(32)
    u = torch.tensor([1.0, 1e30, 3e38, 3e38, 448.0, -2.0, 5.0, 7.0]).repeat(32)
    h = torch.cat([g, u]).bfloat16().cuda().repeat(3, 1)
    h[1, 3], h[2, 129] = float("nan"), float("-inf")
    q, s = w4.w4_silu_mul_quant_block(h)
    torch.cuda.synchronize()
    act = torch.nn.functional.silu(g.double()) * u.double()
    c = codes(q).reshape(3, 32, 8)
    np.testing.assert_allclose(s.cpu().numpy()[0], float(act[4]) / 448, rtol=2.0 ** -19)
    assert (c[0][:, [0, 1, 2, 3, 6, 7]] & 0x7F == 0).all()
    ref = O.e4m3_encode((act[4:6] / act[4] * 448).numpy())
    assert (c[0][:, 4:6] == ref).all()
    assert c[1][0, 3] & 0x7F == 0x7F and c[2].reshape(-1)[129] & 0x7F == 0x7F
    np.testing.assert_array_equal(c[1][16:], c[0][16:])
    np.testing.assert_array_equal(c[2][:16], c[0][:16])


# ---- dense ------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 128, 128), (1, 136, 144), (1, 2056, 1408), (2, 264, 400), (5, 2048, 1408), (16, 520, 2064),
    (17, 384, 1024), (31, 1000, 272), (33, 136, 1552), (64, 2056, 2048), (65, 264, 640), (100, 1032, 4112),
    (128, 128, 128), (129, 8, 16), (129, 264, 144), (200, 520, 1408), (257, 1032, 272), (300, 776, 2064),
    (513, 2056, 640), (1, 4096, 8208), (640, 10240, 256),
    (64, 9736, 144), (41, 4104, 1408), (64, 1032, 2064), (16, 6144, 2064), (64, 5128, 2064), (65, 9728, 272), (65, 9736, 144), (128, 9864, 144)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gemm_matches_oracle(M, N, K, with_bias):
    _, q, s = rows(M, K, seed=M + N)
    qw, sw = weights(N, K, seed=K)
    b = S.bias_bf16(N) if with_bias else None
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4_fp8_block_gemm(fp8(q), to_dev(s), fp8(qw), to_dev(sw), bias=None if b is None else bf16(b), y=y)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(y), O.fp8_block_linear(q, s, qw, sw, b), f"fp8 block gemm {M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 15, 16, 32, 48, 64, 127, 128, 130, 383])
def test_gemm_every_token_count(M):
    """Each token-tile width and its edges, on one weight."""
    N, K = 392, 1168
    _, q, s = rows(M, K, seed=M)
    qw, sw = weights(N, K, seed=3)
    y = w4.w4_fp8_block_gemm(fp8(q), to_dev(s), fp8(qw), to_dev(sw))
    torch.cuda.synchronize()
    check_bf16_output(bits(y), O.fp8_block_linear(q, s, qw, sw), f"M={M}")


@pytest.mark.parametrize("M,N,K,f16", [(1, 2056, 1408, False), (40, 1032, 2064, True), (300, 776, 1040, False)])
def test_gemm_bf16in_equals_quant_then_gemm(M, N, K, f16):
    x = S.activations_bf16(M, K, seed=M, outlier_frac=0.01)
    t = to_dev(S.bf16_bits_to_f32(x).astype(np.float16)) if f16 else bf16(x)
    qw, sw = weights(N, K, seed=5)
    b = bf16(S.bias_bf16(N))
    q, s = w4.w4_quant_act_per_block(t)
    y2 = w4.w4_fp8_block_gemm(q, s, fp8(qw), to_dev(sw), bias=b)
    first = w4.w4_fp8_block_gemm_bf16in(t, fp8(qw), to_dev(sw), bias=b)
    for _ in range(5):     # back to back, into the same freshly freed memory: the quantizer of one call and the product of the last
        y = w4.w4_fp8_block_gemm_bf16in(t, fp8(qw), to_dev(sw), bias=b)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(first), bits(y2))
    np.testing.assert_array_equal(bits(y), bits(y2))
    r = O.fp8_block_linear(codes(q), s.cpu().numpy(), qw, sw, S.bias_bf16(N))
    check_bf16_output(bits(y), r, "bf16in")


def test_gemm_infinite_and_nan_rows_stay_in_their_rows():
    """A token whose codes are NaN gives NaN in its row only, in both forms."""
    N, K = 264, 400
    qw, sw = weights(N, K, seed=8)
    for M in (20, 200):
        _, q, s = rows(M, K, seed=M)
        q[3, 5] = 0x7F
        s[7, 1] = np.inf
        y = w4.w4_fp8_block_gemm(fp8(q), to_dev(s), fp8(qw), to_dev(sw)).float().cpu().numpy()
        assert np.isnan(y[3]).all() and not np.isfinite(y[7]).any()
        good = [m for m in range(M) if m not in (3, 7)]
        assert np.isfinite(y[good]).all()
        r = O.fp8_block_linear(q[good], s[good], qw, sw)
        np.testing.assert_allclose(y[good], r, rtol=8e-3, atol=8e-5 * np.sqrt(np.mean(r * r)) / 8e-3)


def test_gemm_on_another_stream():
    M, N, K = 24, 1032, 1408
    x = S.activations_bf16(M, K, seed=11)
    qw, sw = weights(N, K, seed=12)
    t, qd, sd = bf16(x), fp8(qw), to_dev(sw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty((w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, M, N, K, 0),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    w4.w4_fp8_block_gemm_bf16in(t, qd, sd, y=y, workspace=ws, stream=st)
    st.synchronize()
    q, s = O.quant_fp8_per_block(x)
    check_bf16_output(bits(y), O.fp8_block_linear(q, s, qw, sw), "side stream")


def test_gemm_in_a_cuda_graph():
    M, N, K = 4, 520, 1040
    x = S.activations_bf16(M, K, seed=13)
    qw, sw = weights(N, K, seed=14)
    t, qd, sd = bf16(x), fp8(qw), to_dev(sw)
    ref = w4.w4_fp8_block_gemm_bf16in(t, qd, sd)
    y = torch.zeros_like(ref)
    ws = torch.empty((w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, M, N, K, 0),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w4_fp8_block_gemm_bf16in(t, qd, sd, y=y, workspace=ws)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(y), bits(ref))


def test_gemm_empty():
    qw, sw = weights(128, 128)
    y = w4.w4_fp8_block_gemm_bf16in(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), fp8(qw), to_dev(sw))
    assert tuple(y.shape) == (0, 128)


# ---- experts ----------------------------------------------------------------

COUNTS = [
    [1], [0, 3, 0], [16, 1, 0, 17, 5], [2] * 40 + [0] * 8, [40, 0, 25, 31], [70, 1, 64, 65], [128, 127, 129, 0, 3],
    [300, 0, 1, 200], [0, 0, 700], [1000, 0, 0, 0, 0, 0, 0, 1], [56, 56], [57, 56], [0, 113], [112, 0], [0] * 100 + [5] + [0] * 899 + [260],
]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("N,K", [(264, 400), (136, 16)])
def test_grouped_matches_oracle(counts, N, K):
    if len(counts) > 500 and K > 100:
        N, K = 16, 144
    off = S.offsets_from_counts(counts)
    R, E = int(off[-1]), len(counts)
    _, q, s = rows(R, K, seed=R)
    qw, sw = weights(N, K, seed=E, E=E)
    y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4_fp8_block_moe_grouped_gemm(fp8(q), to_dev(s), to_dev(off), fp8(qw), to_dev(sw), y=y)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(y), O.fp8_block_grouped_linear(q, s, off, qw, sw), f"{counts[:8]}")


@pytest.mark.parametrize("R", [30, 700])
def test_grouped_leaves_rows_outside_the_segments(R):
    """Rows before the first and past the last offset keep what y held; offsets
    past R are clipped."""
    N, K, E = 136, 144, 2
    _, q, s = rows(R, K, seed=R)
    qw, sw = weights(N, K, seed=2, E=E)
    for off in ([5, 9, R - 4], [5, 9, R + 100]):
        off = np.array(off, np.int32)
        y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
        w4.w4_fp8_block_moe_grouped_gemm(fp8(q), to_dev(s), to_dev(off), fp8(qw), to_dev(sw), y=y)
        torch.cuda.synchronize()
        end = min(int(off[-1]), R)
        got = y.float().cpu().numpy()
        assert np.all(got[:5] == 7) and np.all(got[end:] == 7)
        off[-1] = end
        check_bf16_output(bits(y)[5:end], O.fp8_block_grouped_linear(q, s, off, qw, sw)[5:end], "clipped")


@pytest.mark.parametrize("T,E,k,N,K", [(1, 8, 2, 264, 256), (24, 64, 8, 136, 400), (300, 8, 4, 520, 272)])
def test_grouped_bf16in_equals_gather_quant_gemm(T, E, k, N, K):
    x = S.activations_bf16(T, K, seed=T)
    _, _, off, rt, _ = w4.w4_moe_route(to_dev(S.router_logits(T, E, seed=E)), k)
    qw, sw = weights(N, K, seed=7, E=E)
    y = w4.w4_fp8_block_moe_gemm_bf16in(bf16(x), rt, off, fp8(qw), to_dev(sw))
    g = bf16(x)[rt.long()].contiguous()
    q, s = w4.w4_quant_act_per_block(g)
    y2 = w4.w4_fp8_block_moe_grouped_gemm(q, s, off, fp8(qw), to_dev(sw))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(y), bits(y2))
    r = O.fp8_block_grouped_linear(codes(q), s.cpu().numpy(), off.cpu().numpy(), qw, sw)
    check_bf16_output(bits(y), r, "grouped bf16in")


def test_grouped_bf16in_bad_row():
    """A row_token entry outside [0, T) is a zero row and sets the status word."""
    T, E, N, K = 6, 2, 136, 144
    x = S.activations_bf16(T, K, seed=1)
    qw, sw = weights(N, K, seed=7, E=E)
    rt, off = np.array([0, 6, 3, -1, 5], np.int32), np.array([0, 2, 5], np.int32)
    assert w4.w4_device_status() == w4.W4_OK
    y = w4.w4_fp8_block_moe_gemm_bf16in(bf16(x), to_dev(rt), to_dev(off), fp8(qw), to_dev(sw))
    assert w4.w4_device_status() == w4.W4_ERR_SHAPE
    q, s = O.quant_fp8_per_block(x[[0, 0, 3, 0, 5]])
    r = O.fp8_block_grouped_linear(q, s, off, qw, sw)
    r[[1, 3]] = 0
    got = bits(y)
    assert not (got[[1, 3]] & 0x7FFF).any()
    check_bf16_output(got, r, "bad rows")


@pytest.mark.parametrize("R,T,bad", [(9000, 1000, False), (9000, 1000, True), (9000, 8000, False),
                                     (33000, 1000, False), (33000, 1000, True), (33000, 16501, False)])
def test_grouped_bf16in_tokens_quantized_once(R, T, bad):
    """Many rows of few tokens: at 33000 rows the codes are copied from the tokens' (the
    last case has too many tokens for that); with a workspace that only holds the rows they
    are computed again, to the same bits. Rows of bad ids are zero."""
    E, N, K = 4, 136, 528
    x = S.activations_bf16(T, K, seed=5)
    rt = (S.raw_u64(6, 1, R) % T).astype(np.int32)
    if bad:
        rt[[0, 4444, R - 1]] = [T, -1, 2 ** 31 - 1]
    off = np.array([0, 2000, 2000, 5000, R], np.int32)
    qw, sw = weights(N, K, seed=7, E=E)
    args = bf16(x), to_dev(rt), to_dev(off), fp8(qw), to_dev(sw)
    assert w4.w4_device_status() == w4.W4_OK
    y = w4.w4_fp8_block_moe_gemm_bf16in(*args)
    assert w4.w4_device_status() == (w4.W4_ERR_SHAPE if bad else w4.W4_OK)
    rows_only = (R * K + R * 5 * 4 + 15) // 16 * 16
    y2 = w4.w4_fp8_block_moe_gemm_bf16in(*args, workspace=torch.empty(rows_only, dtype=torch.uint8, device="cuda"))
    assert w4.w4_device_status() == (w4.W4_ERR_SHAPE if bad else w4.W4_OK)
    np.testing.assert_array_equal(bits(y), bits(y2))
    ok = (rt >= 0) & (rt < T)
    q, s = O.quant_fp8_per_block(x)
    r = O.fp8_block_grouped_linear(q[np.where(ok, rt, 0)], s[np.where(ok, rt, 0)], off, qw, sw)
    r[~ok] = 0
    check_bf16_output(bits(y), r, "copied codes")


@pytest.mark.parametrize("M,N,K,split", [(300, 4096, 2064, False), (700, 776, 4112, True), (2700, 2056, 1808, False),
                                         (300, 4096, 4112, True), (2700, 2056, 4112, True),
                                         (65, 9736, 4112, True), (128, 9728, 4112, False)])
def test_gemm_split_and_whole(M, N, K, split):
    """The last wave's tiles cut along K where that pays, and the same call without
    room for it."""
    x, q, s = rows(M, K, seed=M)
    qw, sw = weights(N, K, seed=4)
    b = S.bias_bf16(N)
    assert (w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK, M, N, K, 0) > 0) == split
    r = O.fp8_block_linear(q, s, qw, sw, b)
    args = fp8(q), to_dev(s), fp8(qw), to_dev(sw)
    y = w4.w4_fp8_block_gemm(*args, bias=bf16(b))
    whole = w4.w4_fp8_block_gemm(*args, bias=bf16(b), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    again = w4.w4_fp8_block_gemm(*args, bias=bf16(b))
    act = w4.w4_fp8_block_gemm_bf16in(bf16(x), fp8(qw), to_dev(sw), bias=bf16(b))
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(y), r, "split")
    check_bf16_output(bits(whole), r, "whole")
    np.testing.assert_array_equal(bits(again), bits(y))
    np.testing.assert_array_equal(bits(act), bits(y))


def test_binding_refusals():
    """Wrong shapes, types, layouts and missing tensors raise ValueError; what the
    library refuses raises W4Error with its status."""
    M, N, K, E = 4, 264, 256, 2
    x, q, s = rows(M, K)
    qw, sw = weights(N, K)
    qe, se = weights(N, K, E=E)
    X, Q, SX, W, WS = bf16(x), fp8(q), to_dev(s), fp8(qw), to_dev(sw)
    WE, WSE, off = fp8(qe), to_dev(se), to_dev(np.array([0, 1, 4], np.int32))
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [
        lambda: w4.w4_quant_act_per_block(X.float()),
        lambda: w4.w4_quant_act_per_block(X[0]),
        lambda: w4.w4_quant_act_per_block(X[:, ::2]),
        lambda: w4.w4_quant_act_per_block(X, q=torch.empty((M, K + 8), dtype=torch.uint8, device="cuda")),
        lambda: w4.w4_quant_act_per_block(X, scale=torch.empty((M, 3), device="cuda")),
        lambda: w4.w4_silu_mul_quant_block(X.half()),
        lambda: w4.w4_silu_mul_quant_block(torch.zeros((2, 17), dtype=torch.bfloat16, device="cuda")),
        lambda: w4.w4_fp8_block_gemm(X, SX, W, WS),
        lambda: w4.w4_fp8_block_gemm(Q, SX[:, :1].contiguous(), W, WS),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W[:, :128].contiguous(), WS),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, WS[:2].contiguous()),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, WS.half()),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W.t(), WS),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, WS, bias=torch.zeros(N, device="cuda")),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, WS, bias=torch.zeros(N + 8, dtype=torch.bfloat16, device="cuda")),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, WS, y=torch.empty((M, N), device="cuda")),
        lambda: w4.w4_fp8_block_gemm(Q, SX, W, None),
        lambda: w4.w4_fp8_block_gemm_bf16in(X.float(), W, WS),
        lambda: w4.w4_fp8_block_gemm_bf16in(X, W, WS, workspace=torch.empty(64, dtype=torch.uint8)),
        lambda: w4.w4_fp8_block_moe_grouped_gemm(Q, SX, off[:2].contiguous(), WE, WSE),
        lambda: w4.w4_fp8_block_moe_grouped_gemm(Q, SX, off.long(), WE, WSE),
        lambda: w4.w4_fp8_block_moe_grouped_gemm(Q, SX, off, W, WSE),
        lambda: w4.w4_fp8_block_moe_grouped_gemm(Q, SX, off, WE, WSE[:1].contiguous()),
        lambda: w4.w4_fp8_block_moe_gemm_bf16in(X.half(), None, off, WE, WSE),
        lambda: w4.w4_fp8_block_moe_gemm_bf16in(X, torch.zeros(4, dtype=torch.int64, device="cuda"), off, WE, WSE),
        lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), dtype=torch.float16, device="cuda"), 2),
        lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), device="cuda"), 2, bias=torch.zeros(7, device="cuda")),
        lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), device="cuda"), 2, out=(1, 2)),
        lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), device="cuda"), 2, out=(
            torch.empty((2, 2), **i32), torch.empty((2, 2), device="cuda"), torch.empty(8, **i32), torch.empty(4, **i32),
            torch.empty((2, 2), **i32))),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {i} did not raise")
    refused = [
        (w4.W4_ERR_UNSUPPORTED, lambda: w4.w4_fp8_block_gemm(*(fp8(np.zeros((2, 24), np.uint8)), torch.ones((2, 1), device="cuda"),
                                                               fp8(np.zeros((8, 24), np.uint8)), torch.ones((1, 1), device="cuda")))),
        (w4.W4_ERR_ALIGN, lambda: w4.w4_quant_act_per_block(torch.zeros((2, 12), dtype=torch.bfloat16, device="cuda"))),
        (w4.W4_ERR_GROUP, lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), device="cuda"), 2, n_group=3)),
        (w4.W4_ERR_SHAPE, lambda: w4.w4_moe_route_grouped(torch.zeros((2, 8), device="cuda"), 9)),
        (w4.W4_ERR_WORKSPACE, lambda: w4.w4_fp8_block_gemm_bf16in(
            X.repeat(20, 1), W, WS, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
    ]
    for status, call in refused:
        with pytest.raises(w4.W4Error) as e:
            call()
        assert e.value.status == status
    assert w4.w4_device_status() == w4.W4_OK


def test_uint8_codes_and_given_outputs():
    """Codes as uint8 tensors are the same call; outputs are written in place."""
    M, N, K = 20, 136, 272
    _, q, s = rows(M, K, seed=2)
    qw, sw = weights(N, K, seed=3)
    a = w4.w4_fp8_block_gemm(fp8(q), to_dev(s), fp8(qw), to_dev(sw))
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    b = w4.w4_fp8_block_gemm(to_dev(q), to_dev(s), to_dev(qw), to_dev(sw), y=y)
    torch.cuda.synchronize()
    assert b.data_ptr() == y.data_ptr()
    np.testing.assert_array_equal(bits(a), bits(y))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of weights, of activations and of outputs: the last
    expert, the last rows."""
    N, K, E = 8192, 16384, 34
    qw = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")       # 4.6e9 codes
    sw = torch.ones((E, N // 128, K // 128), device="cuda")
    last_q, last_s = weights(N, K, seed=1)
    qw[E - 1], sw[E - 1] = to_dev(last_q), to_dev(last_s)
    for R in (3, 130):
        _, q, s = rows(R, K, seed=R)
        off = np.array([0] * E + [R], np.int32)
        y = w4.w4_fp8_block_moe_grouped_gemm(fp8(q), to_dev(s), to_dev(off), qw, sw)
        torch.cuda.synchronize()
        pick = np.array([0, R - 1])
        check_bf16_output(bits(y)[pick], O.fp8_block_linear(q[pick], s[pick], last_q, last_s), "last expert")
    del qw, sw
    M, K = 270000, 16384                                                # 4.4e9 codes
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    xb = S.activations_bf16(2, K, seed=9)
    x[M - 2:] = bf16(xb)
    q, s = w4.w4_quant_act_per_block(x)
    rq, rs = O.quant_fp8_per_block(xb)
    np.testing.assert_array_equal(codes(q[M - 2:]), rq)
    np.testing.assert_array_equal(s[M - 2:].cpu().numpy(), rs)
    del x
    Nw = 8200                                                           # y of 2.2e9 values, 4.4e9 bytes
    w, ws = weights(Nw, 128, seed=3)
    y = w4.w4_fp8_block_gemm(q[:, :128].contiguous(), s[:, :1].contiguous(), fp8(w), to_dev(ws))
    torch.cuda.synchronize()
    check_bf16_output(bits(y[M - 2:]), O.fp8_block_linear(rq[:, :128], rs[:, :1], w, ws), "last rows")
    assert w4.w4_device_status() == w4.W4_OK


@pytest.mark.parametrize("K", [1680, 1792, 1808, 1920, 2048])
@pytest.mark.parametrize("N", [256, 1024, 1280])
def test_gemm_split_into_as_many_parts_as_blocks(N, K):
    """Few tiles and few blocks: every part holds a block. Two calls in a row share one
    workspace, so that the second one's parts meet the first one's join."""
    M = 256
    _, q, s = rows(M, K, seed=N + K)
    qw, sw = weights(N, K, seed=K)
    need = w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK, M, N, K, 0)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    args = fp8(q), to_dev(s), fp8(qw), to_dev(sw)
    torch.cuda.synchronize()
    ys = [w4.w4_fp8_block_gemm(*args, workspace=ws) for _ in range(8)]
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    check_bf16_output(bits(ys[0]), O.fp8_block_linear(q, s, qw, sw), "parts")
    for y in ys[1:]:
        np.testing.assert_array_equal(bits(y), bits(ys[0]))


@pytest.mark.parametrize("f16", [False, True])
def test_quant_per_block_zeros_keep_their_sign(f16):
    """-0 and +0 among ordinary values, alone in a block (scale 1), and beside values so
    small that their block takes the divide."""
    M, K = 6, 520
    v = S.bf16_bits_to_f32(S.activations_bf16(M, K, seed=4)).astype(np.float32)
    zero = S.raw_u64(5, 1, M * K).reshape(M, K) % 4
    v[zero == 0], v[zero == 1] = -0.0, 0.0
    v[2, 128:256] = -0.0
    v[3, :128] = np.where(zero[3, :128] < 2, v[3, :128], np.float32(2.0 ** -24) if f16 else np.float32(1e-30))
    v[4, 512:] = [-0.0, 1.0, -0.0, 0.0, -1.0, -0.0, 3.0, 0.0]
    x = v.astype(np.float16) if f16 else S.to_bf16_bits(v)
    q, s = w4.w4_quant_act_per_block(to_dev(x) if f16 else bf16(x))
    torch.cuda.synchronize()
    rq, rs = O.quant_fp8_per_block(x)
    assert (rq == 0x80).sum() > M * K // 8 and (rq == 0).sum() > M * K // 8
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes(q), rq)


def test_silu_mul_quant_block_zeros_keep_their_sign():
    """-0 and +0 as gates and as ups: the sign is the product's."""
    g = np.array([-0.0, 0.0, 1.0, -1.0, -0.0, 0.0, 2.0, 1.0], np.float32)
    u = np.array([1.0, -1.0, -0.0, 0.0, -1.0, 1.0, 0.5, 0.0], np.float32)
    for scale in (1.0, 1e-30):                       # and in a block that takes the divide
        h = np.concatenate([np.tile(g, 17), np.tile(u * np.float32(scale), 17)])[None]
        q, _ = w4.w4_silu_mul_quant_block(bf16(S.to_bf16_bits(h)))
        torch.cuda.synchronize()
        got = codes(q).reshape(17, 8)
        np.testing.assert_array_equal(got[:, [0, 1, 2, 3]], 0x80)
        np.testing.assert_array_equal(got[:, [4, 5, 7]], 0)
        np.testing.assert_array_equal(got[:, 6], 0x7E)


@pytest.mark.parametrize("up", [1e38, -3e38, 1e20])
def test_silu_mul_quant_block_far_gates_times_large_ups(up):
    """Products that fp32 holds although 1 + exp(-gate) overflows: scales within 2^-19 of the
    definition's, codes at most a step off and almost all equal. Near and far gates share chunks."""
    low = -175.0 if abs(up) > 1e30 else -130.0
    g = np.linspace(low, -60.0, 1024).astype(np.float32)
    g[5::16] = 3.0
    h = S.to_bf16_bits(np.concatenate([g, np.full(1024, up, np.float32)])[None].repeat(2, 0))
    h[1, :1024] = S.to_bf16_bits(np.linspace(low, -87.5, 1024).astype(np.float32))      # far ones alone
    h[1, 1024:] = S.to_bf16_bits(np.full(1024, up, np.float32))
    h[0, 1024 + 5:2048:16] = S.to_bf16_bits(np.float32([1.0]))[0]
    act = O.silu_mul_f64(h)
    q, s = w4.w4_silu_mul_quant_block(bf16(h))
    torch.cuda.synchronize()
    blocks = act.reshape(2, 8, 128)
    rs = np.abs(blocks).max(axis=2) / 448
    assert rs.min() > 1e-36
    np.testing.assert_allclose(s.cpu().numpy(), rs, rtol=2.0 ** -19)
    ref = O.e4m3_encode((blocks / rs[:, :, None]).reshape(2, 1024)).astype(np.int64)
    got = codes(q).astype(np.int64)
    step = np.abs((ref & 0x7F) - (got & 0x7F))
    assert ((ref ^ got) & 0x80 == 0).all() and step.max() <= 1 and (step != 0).sum() <= 2


def test_silu_mul_quant_block_infinite_gate():
    """silu(inf) = inf: the block's scale is infinite, its finite products have code 0; other
    blocks are as without it."""
    h = S.activations_bf16(2, 512, seed=3)
    h[1] = h[0]
    h[1, 7], h[1, 256 + 7] = 0x7F80, 0x3F80
    q, s = w4.w4_silu_mul_quant_block(bf16(h))
    torch.cuda.synchronize()
    c, s = codes(q), s.cpu().numpy()
    assert np.isposinf(s[1, 0]) and c[1, 7] == 0x7F
    assert (np.delete(c[1, :128], 7) & 0x7F == 0).all()
    np.testing.assert_array_equal(c[1, 128:], c[0, 128:])
    assert s[1, 1] == s[0, 1]


def test_silu_mul_quant_block_products_below_any_scale():
    """A block whose largest product is not 0 but vanishes in fp32 when divided by 448 has
    scale 1 and codes 0, zeros among its products too; a product with it stays finite."""
    g = np.full((1, 256), -60.0, np.float32)
    u = np.full((1, 256), 1e-20, np.float32)          # 60 exp(-60) 1e-20 = 5e-45
    u[0, ::3] = 0.0
    u[0, 128:] = 1.0                                  # a second, ordinary block
    h = S.to_bf16_bits(np.concatenate([g, u], axis=1))
    assert 0 < np.abs(O.silu_mul_f64(h)[0, :128]).max() / 448 < 2.0 ** -150
    q, s = w4.w4_silu_mul_quant_block(bf16(h))
    qw, sw = weights(136, 256, seed=1)
    y = w4.w4_fp8_block_gemm(q, s, fp8(qw), to_dev(sw))
    torch.cuda.synchronize()
    assert s.cpu().numpy()[0, 0] == 1 and (codes(q)[0, :128] & 0x7F == 0).all()
    assert (codes(q)[0, 128:] & 0x7F == 0x7E).all()
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("R", [6, 40000])
def test_grouped_bf16in_of_no_tokens(R):
    """T = 0: every row id is outside [0, T), few rows and many alike, so all rows are zero
    and the status word says so. (The C entry point: an empty tensor has no address.)"""
    N, K, E = 136, 528, 2
    qw, sw = weights(N, K, seed=7, E=E)
    off, rt = to_dev(np.array([0, R // 3, R], np.int32)), torch.zeros(R, dtype=torch.int32, device="cuda")
    x, wd, sd = torch.empty((1, K), dtype=torch.bfloat16, device="cuda"), fp8(qw), to_dev(sw)
    y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    need = w4.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, R, N, K, E)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert w4.w4_device_status() == w4.W4_OK
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    st = w4.load().w4_fp8_block_moe_gemm_bf16in(p(x), 0, p(rt), p(off), E, p(wd), p(sd), p(y), R, N, K, p(ws), need,
                                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == w4.W4_OK
    assert w4.w4_device_status() == w4.W4_ERR_SHAPE
    assert not (bits(y) & 0x7FFF).any()


@pytest.mark.parametrize("f16", [False, True])
def test_quant_per_block_nan_and_infinity(f16):
    """NaN counts for nothing in the maximum and has a NaN code, a block of NaN a NaN scale;
    an infinity makes its block's scale infinite. Other blocks are as without them."""
    v = S.bf16_bits_to_f32(S.activations_bf16(2, 640, seed=4)).astype(np.float32)
    v[1] = v[0]
    v[1, 5], v[1, 128:256], v[1, 256 + 7], v[1, 384 + 9] = np.nan, np.nan, np.inf, -np.inf
    x = v.astype(np.float16) if f16 else S.to_bf16_bits(v)
    if not f16:
        x[1, 5], x[1, 128:256] = 0x7FC0, 0x7FC0
    q, s = w4.w4_quant_act_per_block(to_dev(x) if f16 else bf16(x))
    torch.cuda.synchronize()
    c, s = codes(q), s.cpu().numpy()
    v[0, 5] = 0                                           # the first block's maximum without the NaN
    assert s[1, 0] == np.float32(np.abs(v[0, :128]).max()) / np.float32(448)
    assert c[1, 5] & 0x7F == 0x7F and (np.delete(c[1, :128], 5) & 0x7F != 0x7F).all()
    assert np.isnan(s[1, 1]) and (c[1, 128:256] & 0x7F == 0x7F).all()
    for b, at in ((2, 7), (3, 9)):
        block = c[1, 128 * b:128 * b + 128] & 0x7F
        assert np.isposinf(s[1, b]) and block[at] == 0x7F and (np.delete(block, at) == 0).all()
    np.testing.assert_array_equal(c[1, 512:], c[0, 512:])
    assert s[1, 4] == s[0, 4]


@pytest.mark.parametrize("M", [1, 2, 3, 5, 7, 8, 9])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("N,K", [(2056, 1456), (200, 272), (40008, 272), (5128, 2064)])
def test_few_16_bit_rows(M, f16, N, K):
    """Rows that the product quantizes itself (up to eight) and the first count that it does
    not: K shared by a cluster and not, one item a CTA and several, ragged last blocks; equal
    to quantizer and product bit for bit, and to the oracle."""
    x = S.activations_bf16(M, K, seed=M + N, outlier_frac=0.01)
    x = S.bf16_bits_to_f32(x).astype(np.float16) if f16 else x
    t = to_dev(x) if f16 else bf16(x)
    qw, sw = weights(N, K, seed=M)
    b = S.bias_bf16(N)
    wd, sd, bd = fp8(qw), to_dev(sw), bf16(b)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4_fp8_block_gemm_bf16in(t, wd, sd, bias=bd, y=y)
    q, s = w4.w4_quant_act_per_block(t)
    two = w4.w4_fp8_block_gemm(q, s, wd, sd, bias=bd)
    torch.cuda.synchronize()
    assert w4.w4_device_status() == w4.W4_OK
    np.testing.assert_array_equal(bits(y), bits(two))
    rq, rs = O.quant_fp8_per_block(x)
    check_bf16_output(bits(y), O.fp8_block_linear(rq, rs, qw, sw, b), f"{M} rows")


@pytest.mark.parametrize("sweep", [False, True])
def test_silu_mul_quant_block_against_the_fp32_formula(sweep):
    """Codes and scales against fl(fl(g / fl(1 + fl(exp(-g)))) u), each step rounded once. A
    product is off by a few fp32 ulp at most (exponential and quotient one each, and the
    roundings), so by 2^-21; so is a scale. A quotient of the two crosses one of the code
    boundaries, which are 2^-4 apart at least, for a share of at most 2^-15 of the elements
    and by one step. Random gates, and every bf16 gate of magnitude up to 80."""
    if sweep:
        g = np.arange(1 << 16, dtype=np.uint16)
        g = g[np.abs(np.nan_to_num(S.bf16_bits_to_f32(g), nan=1e9)) <= 80]
        g = g[:g.size // 1024 * 1024].reshape(-1, 1024)
        R, I = g.shape
        h = np.concatenate([g, S.activations_bf16(R, I, seed=2, std=3.0)], axis=1)
    else:
        R, I = 512, 2048
        h = S.activations_bf16(R, 2 * I, seed=1, std=3.0, outlier_frac=0.01)
    q, s = w4.w4_silu_mul_quant_block(bf16(h))
    torch.cuda.synchronize()
    v = S.bf16_bits_to_f32(h)
    g, u = v[:, :I], v[:, I:]
    f32, f64 = np.float32, np.float64
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        d = (f32(1) + np.exp(-g.astype(f64)).astype(f32)).astype(f32)
        p = ((g / d).astype(f32) * u).astype(f32).reshape(R, I // 128, 128)
        rs = (np.abs(p).max(axis=2) / f32(448)).astype(f32)
        ordinary = rs > 1e-30
        quotient = (p / rs[:, :, None]).astype(f32)
    assert ordinary.mean() > 0.5
    np.testing.assert_allclose(s.cpu().numpy()[ordinary], rs[ordinary], rtol=2.0 ** -21)
    ref = O.e4m3_encode(np.nan_to_num(quotient[ordinary]).astype(f64)).astype(np.int64)
    got = codes(q).reshape(R, I // 128, 128)[ordinary].astype(np.int64)
    step = np.abs((ref & 0x7F) - (got & 0x7F))
    assert step.max() <= 1 and ((ref ^ got)[step == 0] == 0).all()
    assert (step != 0).sum() <= step.size * 2.0 ** -15 + 1, (step != 0).sum()
