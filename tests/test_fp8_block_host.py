"""Host-side checks of the fp8 block-scaled layer and the grouped router that need
no GPU: argument validation through the C ABI, workspace sizes, and the compiled
binding's refusals of tensors that are not on a GPU."""
import ctypes
import os
import re

import pytest
import torch

import int4_weight_quantized_w4_gb300 as w4
from int4_weight_quantized_w4_gb300 import _build

FAKE = ctypes.c_void_p(1 << 20)    # 16-byte aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
ODD2 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return w4.load()


def test_route_grouped_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, f32=1, bias=None, T=4, E=64, k=8, g=8, tg=4, sc=w4.W4_SCORE_SIGMOID, ids=FAKE, w=FAKE, off=FAKE,
                 rt=FAKE, ro=FAKE, ws=None, wsb=0)
        a.update(kw)
        return lib.w4_moe_route_grouped(a["x"], a["f32"], a["bias"], a["T"], a["E"], a["k"], a["g"], a["tg"], a["sc"], 1,
                                        1.0, a["ids"], a["w"], a["off"], a["rt"], a["ro"], a["ws"], a["wsb"], None)
    assert call(T=-1) == w4.W4_ERR_SHAPE
    assert call(E=0) == w4.W4_ERR_UNSUPPORTED
    assert call(E=1025) == w4.W4_ERR_UNSUPPORTED
    assert call(sc=2) == w4.W4_ERR_DTYPE
    assert call(g=0) == w4.W4_ERR_GROUP
    assert call(g=7) == w4.W4_ERR_GROUP                   # does not divide 64
    assert call(g=64, tg=8) == w4.W4_ERR_UNSUPPORTED      # more than 32 groups
    assert call(tg=0) == w4.W4_ERR_GROUP
    assert call(tg=9) == w4.W4_ERR_GROUP
    assert call(k=0) == w4.W4_ERR_SHAPE
    assert call(k=9, tg=1) == w4.W4_ERR_SHAPE             # one open group of eight experts
    assert b"of 8" in lib.w4_last_error()
    assert call(k=65, E=128) == w4.W4_ERR_SHAPE
    assert call(T=1 << 30) == w4.W4_ERR_UNSUPPORTED       # rows past int32
    assert call(x=None) == w4.W4_ERR_NULL
    assert call(ro=None) == w4.W4_ERR_NULL
    assert call(x=ODD2) == w4.W4_ERR_ALIGN
    assert call(bias=ODD2) == w4.W4_ERR_ALIGN
    assert call(T=1000) == w4.W4_ERR_WORKSPACE            # many tokens need a workspace
    assert call(T=1000, ws=FAKE, wsb=8) == w4.W4_ERR_WORKSPACE
    assert call(T=0) == w4.W4_OK
    assert lib.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE_GROUPED, 1, 64, 1, 0) == 0
    assert lib.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE_GROUPED, 1000, 64, 1, 0) % (64 * 4) == 0
    # the table of counts stays within one row per SM however many tokens
    assert lib.w4_workspace_bytes(w4.W4_OP_MOE_ROUTE_GROUPED, 1 << 24, 256, 1, 0) <= 152 * 256 * 4


def test_block_quant_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, dt=w4.W4_BF16, M=4, K=256, q=FAKE, s=FAKE)
        a.update(kw)
        return lib.w4_quant_act_per_block(a["x"], a["dt"], a["M"], a["K"], a["q"], a["s"], None)
    assert call(dt=w4.W4_INT8) == w4.W4_ERR_DTYPE
    assert call(M=-1) == w4.W4_ERR_SHAPE
    assert call(K=0) == w4.W4_ERR_SHAPE
    assert call(K=12) == w4.W4_ERR_ALIGN
    assert call(q=None) == w4.W4_ERR_NULL
    assert call(x=ODD) == w4.W4_ERR_ALIGN
    assert call(s=ODD2) == w4.W4_ERR_ALIGN
    assert call(M=0) == w4.W4_OK
    assert lib.w4_silu_mul_quant_block(FAKE, -1, 8, FAKE, FAKE, None) == w4.W4_ERR_SHAPE
    assert lib.w4_silu_mul_quant_block(FAKE, 1, 12, FAKE, FAKE, None) == w4.W4_ERR_ALIGN
    assert lib.w4_silu_mul_quant_block(None, 1, 8, FAKE, FAKE, None) == w4.W4_ERR_NULL
    assert lib.w4_silu_mul_quant_block(ODD, 1, 8, FAKE, FAKE, None) == w4.W4_ERR_ALIGN
    assert lib.w4_silu_mul_quant_block(None, 0, 8, None, None, None) == w4.W4_OK


def test_block_gemm_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, b=None, y=FAKE, M=300, N=256, K=256, wk=None, wkb=0)
        a.update(kw)
        return lib.w4_fp8_block_gemm(a["x"], a["xs"], a["w"], a["ws"], a["b"], a["y"], a["M"], a["N"], a["K"], a["wk"],
                                     a["wkb"], None)
    assert call(M=-1) == w4.W4_ERR_SHAPE
    assert call(N=0) == w4.W4_ERR_SHAPE
    assert call(N=12) == w4.W4_ERR_ALIGN
    assert call(K=12) == w4.W4_ERR_ALIGN
    assert call(K=264) == w4.W4_ERR_UNSUPPORTED           # K % 16
    assert call(x=None) == w4.W4_ERR_NULL
    assert call(ws=None) == w4.W4_ERR_NULL
    assert call(y=ODD) == w4.W4_ERR_ALIGN
    assert call(b=ODD) == w4.W4_ERR_ALIGN
    assert call(xs=ODD2) == w4.W4_ERR_ALIGN
    assert call(wk=ODD, wkb=64) == w4.W4_ERR_WORKSPACE
    assert call(M=1 << 31) == w4.W4_ERR_UNSUPPORTED
    assert call(M=0) == w4.W4_OK


def test_block_gemm_bf16in_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, dt=w4.W4_BF16, w=FAKE, ws=FAKE, b=None, y=FAKE, M=64, N=256, K=256, wk=None, wkb=0)
        a.update(kw)
        return lib.w4_fp8_block_gemm_bf16in(a["x"], a["dt"], a["w"], a["ws"], a["b"], a["y"], a["M"], a["N"], a["K"],
                                            a["wk"], a["wkb"], None)
    assert call(dt=w4.W4_INT8) == w4.W4_ERR_DTYPE
    assert call(x=None) == w4.W4_ERR_NULL
    assert call(x=ODD) == w4.W4_ERR_ALIGN
    need = lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, 64, 256, 256, 0)
    assert need == 64 * 256 + 64 * 2 * 4
    assert call() == w4.W4_ERR_WORKSPACE
    assert call(wk=FAKE, wkb=need - 1) == w4.W4_ERR_WORKSPACE
    assert call(wk=ODD, wkb=need) == w4.W4_ERR_WORKSPACE
    assert call(M=0, dt=w4.W4_FP16) == w4.W4_OK
    # few rows: the product quantizes, no workspace
    assert lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, 1, 256, 256, 0) == 0
    # a last wave cut along K: room for the part sums after the codes, in both entry points
    M, N, K = 300, 4096, 4096
    parts = lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK, M, N, K, 0)
    assert parts > 0 and parts % (128 * 256 * 4) == 0
    assert lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, M, N, K, 0) == M * K + M * 32 * 4 + parts


def test_block_experts_validation(lib):
    def call(**kw):
        a = dict(x=FAKE, xs=FAKE, off=FAKE, E=4, w=FAKE, ws=FAKE, y=FAKE, R=16, N=256, K=256)
        a.update(kw)
        return lib.w4_fp8_block_moe_grouped_gemm(a["x"], a["xs"], a["off"], a["E"], a["w"], a["ws"], a["y"], a["R"],
                                                 a["N"], a["K"], None)
    assert call(E=0) == w4.W4_ERR_SHAPE
    assert call(E=1025) == w4.W4_ERR_UNSUPPORTED
    assert call(K=264) == w4.W4_ERR_UNSUPPORTED
    assert call(off=None) == w4.W4_ERR_NULL
    assert call(off=ODD2) == w4.W4_ERR_ALIGN
    assert call(R=0) == w4.W4_OK

    def act(**kw):
        a = dict(x=FAKE, T=8, rt=FAKE, off=FAKE, E=4, w=FAKE, ws=FAKE, y=FAKE, R=16, N=256, K=256, wk=None, wkb=0)
        a.update(kw)
        return lib.w4_fp8_block_moe_gemm_bf16in(a["x"], a["T"], a["rt"], a["off"], a["E"], a["w"], a["ws"], a["y"], a["R"],
                                                a["N"], a["K"], a["wk"], a["wkb"], None)
    assert act(T=-1) == w4.W4_ERR_SHAPE
    assert act(rt=None) == w4.W4_ERR_SHAPE                # R != T without row ids
    assert act(off=None) == w4.W4_ERR_NULL
    assert act() == w4.W4_ERR_WORKSPACE
    assert act(R=0) == w4.W4_OK
    rows, tokens = 16 * 256 + 16 * 2 * 4, 8 * 256 + 8 * 2 * 4
    assert lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK_IN, 16, 256, 256, 4) == rows + tokens


def test_binding_refuses_tensors_that_are_not_on_a_gpu(lib):
    t = torch.zeros
    x, q, s = t((2, 128), dtype=torch.bfloat16), t((2, 128), dtype=torch.float8_e4m3fn), t((2, 1))
    for call in (lambda: w4.w4_moe_route_grouped(t((2, 8)), 2),
                 lambda: w4.w4_quant_act_per_block(x),
                 lambda: w4.w4_silu_mul_quant_block(x),
                 lambda: w4.w4_fp8_block_gemm(q, s, q, s),
                 lambda: w4.w4_fp8_block_gemm_bf16in(x, q, s),
                 lambda: w4.w4_fp8_block_moe_grouped_gemm(q, s, None, q, s),
                 lambda: w4.w4_fp8_block_moe_gemm_bf16in(x, None, None, q, s)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="is required"):
        w4.w4_quant_act_per_block(None)
    with pytest.raises(ValueError, match="scoring"):
        w4.w4_moe_route_grouped(t((2, 8)), 2, scoring="relu")


def test_every_part_of_a_split_tile_has_a_block(lib):
    """A tile is cut along K into at most as many parts as K has blocks of 128, over
    every K up to 4096 and every count of tiles in the last wave."""
    tile = 128 * 256 * 4
    split = 0
    for K in range(16, 4097, 16):
        blocks = -(-K // 128)
        for pairs in range(1, 77):
            need = lib.w4_workspace_bytes(w4.W4_OP_FP8_BLOCK, 256, 256 * pairs, K, 0)
            if need == 0:
                continue
            tiles = 2 * pairs % 152
            parts, rest = divmod(need, tiles * tile)
            assert rest == 0 and 2 <= parts <= min(16, blocks), (K, pairs, parts)
            split += 1
    assert split > 1000


@pytest.mark.parametrize("unit", ["fp8_block.cu", "fp8_quant.cu", "moe_route.cu"])
def test_early_started_kernels_read_nothing_through_the_non_coherent_path(unit):
    """These kernels start while the kernels before them still write what they read, so
    none of their loads may be one that takes its data as constant for the whole kernel:
    not spelled out, and not by a const __restrict__ pointer."""
    with open(os.path.join(_build.CSRC, unit)) as f:
        text = f.read()
    assert "griddepcontrol.wait" in text
    assert not re.findall(r"ld_nc_\w+|ld_stream_\w+|__ldg\b|\.nc\b", text)
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__", text)


def test_block_quant_of_too_many_rows_is_unsupported(lib):
    """Rows times blocks past what one grid numbers: refused as such, not by the launch."""
    for M, K in ((1 << 31, 8), (1 << 31, 512), (1 << 30, 1032), (1 << 40, 128)):
        assert lib.w4_quant_act_per_block(FAKE, w4.W4_BF16, M, K, FAKE, FAKE, None) == w4.W4_ERR_UNSUPPORTED
        assert lib.w4_silu_mul_quant_block(FAKE, M, K, FAKE, FAKE, None) == w4.W4_ERR_UNSUPPORTED


def test_expert_offsets_are_read_from_l2():
    """The expert products may read the offsets before they have waited for the kernels
    before them (the quantizer starts them only when the routing is done), so that an L1 line
    of an earlier routing must not answer."""
    with open(os.path.join(_build.CSRC, "fp8_block.cu")) as f:
        text = f.read()
    assert "__ldcg(p.offsets" in text
    assert not re.findall(r"p\.offsets\s*\[|\*\s*p\.offsets", text)
