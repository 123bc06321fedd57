"""Oracle of the microscaled 4-bit floating point layer: float64 numpy, from the
definitions alone (no code shared with the CUDA path).

Codes are e2m1, two in a byte, the lower column in the low half. ``mxfp4`` has a
power of two (byte - 127) per 32 columns, ``nvfp4`` an e4m3 scale per 16 columns and a
float32 scale per tensor.
"""
from __future__ import annotations

import numpy as np

from .fp8_block_oracle import silu_mul_f64
from .w4_oracle import _activations_f32, e4m3_decode, e4m3_encode

FP4_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e2m1_encode(v):
    """Codes of the nearest e2m1 values, ties to the even code, held to +-6."""
    v = np.asarray(v, np.float64)
    m = np.abs(v)
    code = np.zeros(v.shape, np.uint8)
    for i in range(7):
        border = (FP4_VALUES[i] + FP4_VALUES[i + 1]) / 2
        code += (m >= border) if i % 2 else (m > border)
    return code | (np.signbit(v).astype(np.uint8) << 3)


def fp4_pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def fp4_unpack(q):
    return np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], -1)


def fp4_decode(q):
    """Packed codes [..., K/2] as values [..., K]."""
    c = fp4_unpack(np.asarray(q))
    return np.where(c > 7, -1.0, 1.0) * FP4_VALUES[c & 7]


def fp4_scale_decode(s, fmt):
    """Scale bytes as values."""
    s = np.asarray(s).view(np.uint8)
    if fmt == "nvfp4":
        return e4m3_decode(s)
    return np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))


def _quant_rows(x, fmt, g):
    M, K = x.shape
    p = x.reshape(M, -1, FP4_BLOCK[fmt])
    amax = np.abs(p).max(axis=2)
    odd = ~np.isfinite(amax)
    p, amax = np.where(odd[:, :, None], 0, p), np.where(odd, 0, amax)
    if fmt == "mxfp4":
        e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127, 127)
        code = e2m1_encode(p.astype(np.float64) * np.exp2(-e.astype(np.float64))[:, :, None])
        s = np.where(odd, 255, e + 127).astype(np.uint8)
    else:
        g = np.float32(1.0 if g is None else g)
        with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
            v = ((amax.astype(np.float32) / np.float32(6)).astype(np.float32) / g).astype(np.float32)
            s = e4m3_encode(np.minimum(v, np.float32(448)))
            d = (e4m3_decode(s).astype(np.float32) * g).astype(np.float32)[:, :, None]
            code = e2m1_encode(np.where(d > 0, (p.astype(np.float32) / d).astype(np.float32), np.float32(0)))
        s = np.where(odd, 0x7F, s).astype(np.uint8)
    code = np.where(odd[:, :, None], 0, code).astype(np.uint8)
    return fp4_pack(code.reshape(M, K)), s


def quant_fp4(x_bits, fmt, g=None):
    """Packed codes and scale bytes of bf16 bit patterns or a float16 array ``[M, K]``."""
    return _quant_rows(_activations_f32(x_bits), fmt, g)


def silu_mul_quant_fp4(h_bits, fmt, g=None):
    """The same of silu(gate) * up, rounded from float64 to float32 in between."""
    return _quant_rows(silu_mul_f64(h_bits).astype(np.float32), fmt, g)


def dequant_fp4(q, s, fmt, g=None):
    """float64 values of packed codes."""
    d = fp4_scale_decode(s, fmt)
    if fmt == "nvfp4" and g is not None:
        d = (d.astype(np.float32) * np.float32(g)).astype(np.float64)
    v = fp4_decode(q)
    return (v.reshape(*d.shape, -1) * d[..., None]).reshape(v.shape)


def fp4_linear(qx, x_scale, qweight, w_scale, fmt, x_global=None, w_global=None, bias_bits=None):
    """``y = x_global w_global (qx x_scale) (qweight w_scale)^T + bias`` in float64."""
    from .w4_oracle import bf16_to_f64
    y = dequant_fp4(qx, x_scale, fmt) @ dequant_fp4(qweight, w_scale, fmt).T
    for v in (x_global, w_global):
        y = y * (1.0 if v is None else np.float64(np.float32(v)))
    return y if bias_bits is None else y + bf16_to_f64(bias_bits)


def fp4_grouped_linear(qx, x_scale, offsets, qweight, w_scale, fmt, x_global=None, w_global=None):
    """Rows [offsets[e], offsets[e+1]) times expert e; rows of no expert are NaN."""
    y = np.full((qx.shape[0], qweight.shape[1]), np.nan)
    for e in range(qweight.shape[0]):
        r = slice(max(0, int(offsets[e])), int(offsets[e + 1]))
        if r.stop > r.start:
            y[r] = fp4_linear(qx[r], x_scale[r], qweight[e], w_scale[e], fmt, x_global,
                              None if w_global is None else w_global[e])
    return y


def moe_decode(x_bits, logits, gate_up, down, top_k, **route):
    """A whole routed layer in float64. gate_up(e) [2I, H] and down(e) [H, I] give an expert's
    weights as values. Returns ``(y [T, H], size [T, H])``: size is the sum of the
    magnitudes that make up y, weight by weight and activation by activation."""
    from .fp8_block_oracle import moe_route_grouped
    from .w4_oracle import bf16_to_f64
    x = bf16_to_f64(x_bits)
    ids, wts, _ = moe_route_grouped(logits, top_k, **route)
    y, size = np.zeros(x.shape), np.zeros(x.shape)
    for e in sorted(set(ids.ravel().tolist())):
        gu, d = gate_up(e), down(e)
        for t, j in zip(*np.nonzero(ids == e)):
            h = gu @ x[t]
            I = h.size // 2
            with np.errstate(over="ignore"):
                a = h[:I] / (1.0 + np.exp(-h[:I])) * h[I:]
            y[t] += wts[t, j] * (d @ a)
            size[t] += wts[t, j] * (np.abs(d) @ np.abs(a))
    return y, size
