"""Oracle of the fp8 block-scaled layer and the grouped router: float64 numpy,
from the definitions alone (no code shared with the CUDA path).

A block is 128 consecutive columns (and, for weights, 128 rows); the last one
of a row may be shorter.
"""
from __future__ import annotations

import numpy as np

from .w4_oracle import _activations_f32, bf16_to_f64, e4m3_decode, e4m3_encode

BLOCK = 128


def _quant_rows_f32(x: np.ndarray):
    M, K = x.shape
    nb = -(-K // BLOCK)
    q = np.zeros((M, K), np.uint8)
    s = np.ones((M, nb), np.float32)
    for b in range(nb):
        c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        amax = np.max(np.abs(x[:, c]), axis=1)
        sb = (amax / np.float32(448.0)).astype(np.float32)
        s[:, b] = np.where(amax == 0, np.float32(1.0), sb)
        with np.errstate(divide="ignore", invalid="ignore"):
            v = (x[:, c] / s[:, b:b + 1]).astype(np.float32)
        # a quotient that is 0 / 0 or beyond fp32 comes from a block whose scale underflowed
        q[:, c] = e4m3_encode(np.nan_to_num(v, nan=0.0, posinf=448.0, neginf=-448.0))
    return q, s


def quant_fp8_per_block(x_bits):
    """Per row and block: ``s = fp32(amax / 448)`` (1 if amax is 0), ``q =
    e4m3(fp32(x / s))``. ``x_bits``: bf16 bit patterns, or a float16 array.
    Returns ``(q uint8 [M, K], s float32 [M, ceil(K/128)])``."""
    return _quant_rows_f32(_activations_f32(x_bits))


def silu_mul_f64(h_bits):
    """silu(gate) * up of bf16 ``h [R, 2I]`` in float64."""
    h = bf16_to_f64(h_bits)
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def fp8_block_linear(qx, x_scale, qweight, w_scale, bias_bits=None):
    """``y[m, n] = sum_b sx[m, b] sw[n // 128, b] sum_{k in b} x[m, k] w[n, k] +
    bias[n]`` in float64, returned as float32 ``[M, N]``. qx, qweight: codes."""
    x, w = e4m3_decode(qx), e4m3_decode(qweight)
    M, K = x.shape
    N = w.shape[0]
    y = np.zeros((M, N))
    for b in range(-(-K // BLOCK)):
        c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        sw = np.repeat(np.asarray(w_scale, np.float64)[:, b], BLOCK)[:N]
        y += np.asarray(x_scale, np.float64)[:, b:b + 1] * (x[:, c] @ w[:, c].T) * sw
    if bias_bits is not None:
        y += bf16_to_f64(bias_bits)
    return y.astype(np.float32)


def fp8_block_grouped_linear(qx, x_scale, offsets, qweight, w_scale):
    """``fp8_block_linear`` of rows ``offsets[e] .. offsets[e+1]`` with expert e."""
    y = np.zeros((qx.shape[0], qweight.shape[1]), np.float32)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            y[a:b] = fp8_block_linear(qx[a:b], x_scale[a:b], qweight[e], w_scale[e])
    return y


def row_order(ids, E):
    """Offsets, row_token and row_of of chosen experts ``ids [T, k]``: the pairs
    (token, choice) listed by expert, then token."""
    T, k = ids.shape
    pairs = sorted((int(ids[t, j]), t, j) for t in range(T) for j in range(k))
    offsets = np.zeros(E + 1, np.int32)
    row_token, row_of = np.zeros(T * k, np.int32), np.zeros((T, k), np.int32)
    for r, (e, t, j) in enumerate(pairs):
        offsets[e + 1:] += 1
        row_token[r] = t
        row_of[t, j] = r
    return offsets, row_token, row_of


def moe_route_grouped(logits, top_k, bias=None, n_group=1, topk_group=1, scoring="sigmoid", renormalize=True,
                      scale=1.0):
    """Choice and weights in float64, with the score rounded to fp32 before the
    bias is added in fp32. Returns ``(ids, weights, gap)``: ``gap[t]`` is the
    smallest nonzero difference between two values that the choice of token t
    compared (an fp32 evaluation of scores may order closer ones the other way)."""
    lg = np.asarray(logits, np.float32).astype(np.float64)
    lg = np.where(np.isnan(lg), -np.inf, np.minimum(lg, float(np.finfo(np.float32).max)))
    T, E = lg.shape
    gs = E // n_group
    ids, wts, gap = np.zeros((T, top_k), np.int32), np.zeros((T, top_k)), np.full(T, np.inf)
    for t in range(T):
        with np.errstate(over="ignore", invalid="ignore"):
            if scoring == "sigmoid":
                score = 1.0 / (1.0 + np.exp(-lg[t]))
            elif np.all(np.isneginf(lg[t])):
                score = np.zeros(E)
            else:
                ex = np.exp(lg[t] - lg[t].max())
                score = ex / ex.sum()
        if bias is None:
            key = lg[t]
        else:
            key = (score.astype(np.float32) + np.asarray(bias, np.float32)).astype(np.float64)
        value = []
        for g in range(n_group):
            best = sorted(key[g * gs:(g + 1) * gs], reverse=True)
            value.append(best[0] if bias is None or gs == 1 else float(np.float32(best[0] + best[1])))
        order = sorted(range(n_group), key=lambda g: (-value[g], g))
        open_e = [e for g in order[:topk_group] for e in range(g * gs, (g + 1) * gs)]
        ranked = sorted(open_e, key=lambda e: (-key[e], e))
        ids[t] = ranked[:top_k]
        near = [key[e] for e in ranked[:top_k + 1]]
        pairs = list(zip(near, near[1:]))
        if topk_group < n_group:
            pairs.append((value[order[topk_group - 1]], value[order[topk_group]]))
        diffs = [a - b for a, b in pairs if np.isfinite(a) and np.isfinite(b) and a > b]
        gap[t] = min(diffs) if diffs else np.inf
        w = score[ids[t]]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        wts[t] = w * scale
    return ids, wts, gap
