"""Host-side checks of the 4-bit floating point layer and the few-token expert layer that
need no GPU: argument validation through the C ABI, workspace sizes, the compiled
binding's refusals, and pins of the oracle's formats."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
import oracle as O
from int4_weight_quantized_w4_gb300 import _build

FAKE = ctypes.c_void_p(1 << 20)    # 16-byte aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
MX, NV, INT4 = w4.W4_FMT_MXFP4, w4.W4_FMT_NVFP4, w4.W4_FMT_INT4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return w4.load()


def test_quantizer_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, dt=w4.W4_BF16, f=NV, g=None, M=4, K=64, q=FAKE, s=FAKE)
        a.update(kw)
        return lib.w4_quant_fp4(a["x"], a["dt"], a["f"], a["g"], a["M"], a["K"], a["q"], a["s"], None)
    assert call(dt=w4.W4_INT8) == w4.W4_ERR_DTYPE
    assert call(f=INT4) == w4.W4_ERR_DTYPE
    assert call(f=3) == w4.W4_ERR_DTYPE
    assert call(f=MX, g=FAKE) == w4.W4_ERR_UNSUPPORTED    # a power of two per block is all mxfp4 has
    assert call(g=ODD2) == w4.W4_ERR_ALIGN
    assert call(M=-1) == w4.W4_ERR_SHAPE
    assert call(K=0) == w4.W4_ERR_SHAPE
    assert call(K=36) == w4.W4_ERR_ALIGN
    assert call(K=48) == w4.W4_ERR_UNSUPPORTED
    assert call(M=1 << 40) == w4.W4_ERR_UNSUPPORTED
    assert call(K=1 << 32) == w4.W4_ERR_UNSUPPORTED
    assert call(q=None) == w4.W4_ERR_NULL
    assert call(x=ODD) == w4.W4_ERR_ALIGN
    assert call(q=ODD) == w4.W4_ERR_ALIGN
    assert call(M=0) == w4.W4_OK

    def silu(**kw):
        a = dict(h=FAKE, f=MX, g=None, R=4, I=64, q=FAKE, s=FAKE)
        a.update(kw)
        return lib.w4_silu_mul_quant_fp4(a["h"], a["f"], a["g"], a["R"], a["I"], a["q"], a["s"], None)
    assert silu(f=INT4) == w4.W4_ERR_DTYPE
    assert silu(g=FAKE) == w4.W4_ERR_UNSUPPORTED
    assert silu(R=-1) == w4.W4_ERR_SHAPE
    assert silu(I=8) == w4.W4_ERR_UNSUPPORTED
    assert silu(h=None) == w4.W4_ERR_NULL
    assert silu(h=ODD) == w4.W4_ERR_ALIGN
    assert silu(R=0, h=None, q=None, s=None) == w4.W4_OK

    def dequant(**kw):
        a = dict(q=FAKE, s=FAKE, f=MX, g=None, M=4, K=64, dt=w4.W4_BF16, o=FAKE)
        a.update(kw)
        return lib.w4_dequant_fp4(a["q"], a["s"], a["f"], a["g"], a["M"], a["K"], a["dt"], a["o"], None)
    assert dequant(dt=w4.W4_INT8) == w4.W4_ERR_DTYPE
    assert dequant(f=9) == w4.W4_ERR_DTYPE
    assert dequant(K=40) == w4.W4_ERR_UNSUPPORTED
    assert dequant(s=None) == w4.W4_ERR_NULL
    assert dequant(o=ODD) == w4.W4_ERR_ALIGN
    assert dequant(M=0) == w4.W4_OK


@pytest.mark.parametrize("fmt,unit", [(MX, 128), (NV, 64)])
def test_product_validation(lib, fmt, unit):
    def call(**kw):
        a = dict(x=FAKE, xs=FAKE, xg=None, w=FAKE, ws=FAKE, wg=None, f=fmt, b=None, y=FAKE, M=300, N=256, K=256)
        a.update(kw)
        return lib.w4_fp4_gemm(a["x"], a["xs"], a["xg"], a["w"], a["ws"], a["wg"], a["f"], a["b"], a["y"], a["M"], a["N"], a["K"], None)
    assert call(f=INT4) == w4.W4_ERR_DTYPE
    assert call(M=-1) == w4.W4_ERR_SHAPE
    assert call(N=0) == w4.W4_ERR_SHAPE
    assert call(N=12) == w4.W4_ERR_ALIGN
    assert call(K=12) == w4.W4_ERR_ALIGN
    assert call(K=unit + 32) == w4.W4_ERR_UNSUPPORTED     # rows of scales are whole words
    assert call(M=1 << 31) == w4.W4_ERR_UNSUPPORTED
    assert call(xs=None) == w4.W4_ERR_NULL
    assert call(ws=None) == w4.W4_ERR_NULL
    for name in ("x", "w", "y", "b"):
        assert call(**{name: ODD}) == w4.W4_ERR_ALIGN, name
    for name in ("xs", "ws"):
        assert call(**{name: ODD2}) == w4.W4_ERR_ALIGN, name
    if fmt == MX:
        assert call(wg=FAKE) == w4.W4_ERR_UNSUPPORTED
        assert call(xg=FAKE) == w4.W4_ERR_UNSUPPORTED
    else:
        assert call(wg=ODD2) == w4.W4_ERR_ALIGN
    assert call(M=0) == w4.W4_OK

    def act(**kw):
        a = dict(x=FAKE, dt=w4.W4_FP16, w=FAKE, ws=FAKE, b=None, y=FAKE, M=64, N=256, K=256, wk=None, wkb=0)
        a.update(kw)
        return lib.w4_fp4_gemm_bf16in(a["x"], a["dt"], None, a["w"], a["ws"], None, fmt, a["b"], a["y"], a["M"], a["N"],
                                      a["K"], a["wk"], a["wkb"], None)
    block = 16 if fmt == NV else 32
    assert act(dt=w4.W4_INT8) == w4.W4_ERR_DTYPE
    assert act(x=None) == w4.W4_ERR_NULL
    assert act(x=ODD) == w4.W4_ERR_ALIGN
    need = lib.w4_workspace_bytes(w4.W4_OP_FP4_IN, 64, 256, 256, block)
    assert need == 64 * 128 + 64 * 256 // block
    assert act() == w4.W4_ERR_WORKSPACE
    assert act(wk=FAKE, wkb=need - 1) == w4.W4_ERR_WORKSPACE
    assert act(wk=ODD, wkb=need) == w4.W4_ERR_WORKSPACE
    assert act(M=0) == w4.W4_OK
    assert lib.w4_workspace_bytes(w4.W4_OP_FP4_IN, 1, 256, 256, block) == 0      # the product quantizes
    assert lib.w4_workspace_bytes(w4.W4_OP_FP4_IN, 64, 256, 256, 64) == 0        # no format has such blocks


@pytest.mark.parametrize("fmt,block", [(MX, 32), (NV, 16)])
def test_experts_validation(lib, fmt, block):
    def call(**kw):
        a = dict(x=FAKE, xs=FAKE, off=FAKE, E=4, w=FAKE, ws=FAKE, y=FAKE, R=16, N=256, K=256)
        a.update(kw)
        return lib.w4_fp4_moe_grouped_gemm(a["x"], a["xs"], None, a["off"], a["E"], a["w"], a["ws"], None, fmt, a["y"], a["R"], a["N"], a["K"], None)
    assert call(E=0) == w4.W4_ERR_SHAPE
    assert call(E=1025) == w4.W4_ERR_UNSUPPORTED
    assert call(R=-1) == w4.W4_ERR_SHAPE
    assert call(off=None) == w4.W4_ERR_NULL
    assert call(off=ODD2) == w4.W4_ERR_ALIGN
    assert call(R=0) == w4.W4_OK

    def act(**kw):
        a = dict(x=FAKE, T=8, rt=FAKE, off=FAKE, E=4, w=FAKE, ws=FAKE, y=FAKE, R=16, N=256, K=256, wk=None, wkb=0)
        a.update(kw)
        return lib.w4_fp4_moe_gemm_bf16in(a["x"], a["T"], None, a["rt"], a["off"], a["E"], a["w"], a["ws"], None, fmt, a["y"],
                                          a["R"], a["N"], a["K"], a["wk"], a["wkb"], None)
    assert act(T=-1) == w4.W4_ERR_SHAPE
    assert act(rt=None) == w4.W4_ERR_SHAPE                # R != T without row ids
    assert act(off=None) == w4.W4_ERR_NULL
    assert act(rt=ODD2) == w4.W4_ERR_ALIGN
    assert act() == w4.W4_ERR_WORKSPACE
    assert act(R=0) == w4.W4_OK
    rows, tokens = 16 * 128 + 16 * 256 // block, 8 * 128 + 8 * 256 // block
    assert lib.w4_workspace_bytes(w4.W4_OP_FP4_MOE_IN, 16, 256, 256, block) == rows + tokens


def _decode(lib, **kw):
    a = dict(x=FAKE, lg=FAKE, f32=1, bias=None, T=4, E=64, k=8, g=1, tg=1, sc=w4.W4_SCORE_SOFTMAX, f=INT4, u=FAKE, us=FAKE, ug=None,
             gu=64, d=FAKE, ds=FAKE, dg=None, gd=64, y=FAKE, H=512, I=256, ws=None, wsb=0)
    a.update(kw)
    return lib.w4_moe_decode(a["x"], a["lg"], a["f32"], a["bias"], a["T"], a["E"], a["k"], a["g"], a["tg"], a["sc"], 1, 1.0, a["f"],
                             a["u"], a["us"], a["ug"], a["gu"], a["d"], a["ds"], a["dg"], a["gd"], a["y"], a["H"], a["I"], a["ws"],
                             a["wsb"], None)


def test_moe_decode_validation(lib):
    def call(**kw):
        return _decode(lib, **kw)
    assert call(T=-1) == w4.W4_ERR_SHAPE
    assert call(k=0) == w4.W4_ERR_SHAPE
    assert call(sc=2) == w4.W4_ERR_DTYPE
    assert call(g=7) == w4.W4_ERR_GROUP
    assert call(f=3) == w4.W4_ERR_DTYPE
    assert call(ug=FAKE) == w4.W4_ERR_UNSUPPORTED         # int4 has no scale per tensor
    assert call(f=MX, dg=FAKE) == w4.W4_ERR_UNSUPPORTED
    assert call(f=NV, dg=ODD2) == w4.W4_ERR_ALIGN
    assert call(H=0) == w4.W4_ERR_SHAPE
    assert call(H=12) == w4.W4_ERR_ALIGN
    assert call(H=96) == w4.W4_ERR_UNSUPPORTED
    assert call(I=32) == w4.W4_ERR_UNSUPPORTED
    assert call(T=17) == w4.W4_ERR_UNSUPPORTED
    assert call(E=257) == w4.W4_ERR_UNSUPPORTED
    assert call(k=33) == w4.W4_ERR_UNSUPPORTED
    assert call(gu=0) == w4.W4_ERR_GROUP
    assert call(gd=96) == w4.W4_ERR_GROUP                 # does not divide 256
    assert call(gd=16) == w4.W4_ERR_UNSUPPORTED
    assert call(x=None) == w4.W4_ERR_NULL
    assert call(ds=None) == w4.W4_ERR_NULL
    for name in ("x", "u", "us", "d", "ds", "y"):
        assert call(**{name: ODD}) == w4.W4_ERR_ALIGN, name
    assert call(lg=ODD2) == w4.W4_ERR_ALIGN
    assert call(bias=ODD2) == w4.W4_ERR_ALIGN
    need = lib.w4_workspace_bytes(w4.W4_OP_MOE_DECODE, 4, 8, 256, 0)
    assert need >= 32 * (2 * 256 + 256 // 8) and need % 16 == 0
    assert call() == w4.W4_ERR_WORKSPACE
    assert call(ws=FAKE, wsb=need - 1) == w4.W4_ERR_WORKSPACE
    assert call(ws=ODD, wsb=need) == w4.W4_ERR_WORKSPACE
    assert call(T=0) == w4.W4_OK
    for op in ((17, 8, 256), (4, 0, 256), (4, 33, 256), (4, 8, 0)):
        assert lib.w4_workspace_bytes(w4.W4_OP_MOE_DECODE, *op, 0) == 0


@pytest.mark.parametrize("fmt,group", [(INT4, 32), (INT4, 128), (INT4, -1), (MX, 32), (NV, 16)])
def test_moe_decode_sizes(lib, fmt, group):
    """What the header promises fits, and no size is left to the launch to refuse: index products of
    enormous ones stay out too."""
    def call(T, H, I):
        return _decode(lib, T=T, H=H, I=I, f=fmt, gu=group, gd=group)
    for I in (128, 1408, 7168):
        assert call(16, 2560, I) == w4.W4_ERR_WORKSPACE
        assert call(7, 4096, I) == w4.W4_ERR_WORKSPACE
    assert call(16, 1 << 15, 128) == w4.W4_ERR_UNSUPPORTED
    assert call(1, 128, 1 << 21) == w4.W4_ERR_UNSUPPORTED
    assert call(1, 1 << 28, 1 << 28) == w4.W4_ERR_UNSUPPORTED


def test_binding_refuses_tensors_that_are_not_on_a_gpu(lib):
    t = torch.zeros
    x, q = t((2, 128), dtype=torch.bfloat16), t((2, 64), dtype=torch.uint8)
    s = t((2, 4), dtype=torch.uint8)
    for call in (lambda: w4.w4_quant_fp4(x, "mxfp4"),
                 lambda: w4.w4_silu_mul_quant_fp4(x, "nvfp4"),
                 lambda: w4.w4_dequant_fp4(q, s, "mxfp4"),
                 lambda: w4.w4_fp4_gemm(q, s, q, s, "mxfp4"),
                 lambda: w4.w4_fp4_gemm_bf16in(x, q, s, "mxfp4"),
                 lambda: w4.w4_fp4_moe_grouped_gemm(q, s, None, q, s, "mxfp4"),
                 lambda: w4.w4_fp4_moe_gemm_bf16in(x, None, None, q, s, "mxfp4"),
                 lambda: w4.w4_moe_decode(x, x, q, s, q, s, 2, "mxfp4")):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="is required"):
        w4.w4_quant_fp4(None, "mxfp4")
    with pytest.raises(ValueError, match="format"):
        w4.w4_quant_fp4(x, "fp4")
    with pytest.raises(ValueError, match="format"):
        w4.w4_fp4_gemm(q, s, q, s, "int4")
    with pytest.raises(ValueError, match="format"):
        w4.w4_moe_decode(x, x, q, s, q, s, 2, "fp8")
    with pytest.raises(ValueError, match="scoring"):
        w4.w4_moe_decode(x, x, q, s, q, s, 2, "mxfp4", scoring="relu")
    with pytest.raises(ValueError, match="dtype"):
        w4.w4_dequant_fp4(q, s, "mxfp4", dtype=torch.float32)


@pytest.mark.parametrize("unit", ["fp4_gemm.cu", "fp4_quant.cu", "moe_decode.cu", "moe_decode_fp4.cu"])
def test_early_started_kernels_read_nothing_through_the_non_coherent_path(unit):
    """These kernels start while the kernels before them still write what they read."""
    with open(os.path.join(_build.CSRC, unit)) as f:
        text = f.read()
    assert re.search(r"griddepcontrol\.wait|grid_dependency_wait\(\)", text)
    assert not re.findall(r"ld_nc_\w+|ld_stream_\w+|__ldg\b|\.nc\b", text)
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__", text)


def test_oracle_codes():
    """e2m1 by hand: values, ties to the even code, the ends."""
    values = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    np.testing.assert_array_equal(O.e2m1_encode(values), range(8))
    np.testing.assert_array_equal(O.e2m1_encode([-v for v in values[1:]]), range(9, 16))
    np.testing.assert_array_equal(O.e2m1_encode([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), [0, 2, 2, 4, 4, 6, 6])
    np.testing.assert_array_equal(O.e2m1_encode([0.2501, 0.7499, 5.01, 100.0]), [1, 1, 7, 7])


def test_oracle_blocks():
    """One block of each format by hand."""
    x = np.zeros((1, 32), np.float16)
    x[0, :4] = 12.0, -6.0, 0.5, 2.9
    q, s = O.quant_fp4(x, "mxfp4")                        # 2^3 <= 12 < 2^4: scale 2^(3 - 2), codes of 6, -3, 0.25, 1.45
    assert s.tolist() == [[128]] and q[0, :2].tolist() == [7 | 13 << 4, 0 | 3 << 4]
    np.testing.assert_array_equal(O.dequant_fp4(q, s, "mxfp4")[0, :4], [12.0, -6.0, 0.0, 3.0])
    q, s = O.quant_fp4(x, "nvfp4")                        # scale 12 / 6 = 2 (e4m3 0x40), the same codes
    assert s.tolist() == [[0x40, 0x00]] and q[0, :2].tolist() == [7 | 13 << 4, 0 | 3 << 4]
    q, s = O.quant_fp4(x, "nvfp4", 0.5)                   # twice the scale in the block: 4 (0x48)
    assert s.tolist() == [[0x48, 0x00]]
    np.testing.assert_array_equal(O.dequant_fp4(q, s, "nvfp4", 0.5)[0, :4], [12.0, -6.0, 0.0, 3.0])
