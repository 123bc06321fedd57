"""Sizes of the few-token expert layer that the library takes, asked of the C ABI without a GPU (a
call that is taken gets as far as its workspace), and the sources of its kernels."""
import os
import re

import pytest

import int4_weight_quantized_w4_gb300 as w4
from int4_weight_quantized_w4_gb300 import _build
from test_fp4_host import _decode, lib  # noqa: F401

FORMATS = {"int4": (w4.W4_FMT_INT4, 64), "mxfp4": (w4.W4_FMT_MXFP4, 32), "nvfp4": (w4.W4_FMT_NVFP4, 16)}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I", [(16, 2048, 1408), (14, 4096, 14336), (14, 4096, 1536), (8, 4864, 2048), (8, 7168, 2048),
                                   (16, 2816, 2048), (1, 16384, 53248)])
def test_sizes_that_are_taken(lib, fmt, T, H, I):  # noqa: F811
    f, group = FORMATS[fmt]
    assert _decode(lib, T=T, H=H, I=I, f=f, gu=group, gd=group) == w4.W4_ERR_WORKSPACE


@pytest.mark.parametrize("T,H", [(8, 5632), (16, 3584)])
def test_sizes_that_mxfp4_takes(lib, T, H):  # noqa: F811
    assert _decode(lib, T=T, H=H, I=2048, f=w4.W4_FMT_MXFP4) == w4.W4_ERR_WORKSPACE


def test_early_started_kernels_read_nothing_through_the_non_coherent_path():
    for unit in ("moe_decode.cuh", "moe_chosen.cuh", "route.cuh"):
        with open(os.path.join(_build.CSRC, unit)) as f:
            text = f.read()
        assert not re.findall(r"ld_nc_\w+|ld_stream_\w+|__ldg\b|\.nc\b", text)
        assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__", text)
