"""Cases for measuring the 4-bit floating point layer and the few-token expert layer.

Four operators, each in its plain form (elementary torch operations in 32
bits) and as the library's calls; ``own`` says which one ``run`` makes:

* ``quant``: microscaled 4-bit codes of a weight, of activations or of
  silu(gate) * up, and the values that the codes stand for
  (``w4_quant_fp4`` or ``w4_silu_mul_quant_fp4``, then ``w4_dequant_fp4``);
* ``linear``: y = x W^T with 4-bit floating point weights, of 16-bit
  activations that are quantized alike (``w4_fp4_gemm_bf16in``);
* ``experts``: the same product over the routed rows of a set of experts
  (``w4_fp4_moe_gemm_bf16in``);
* ``layer``: a whole mixture-of-experts layer for a few tokens, from router
  logits to the weighted sum, with 4-bit weights and 16-bit activations
  (``w4_moe_decode``).

Two formats of microscaled 4-bit floats, both e2m1 codes: ``mxfp4`` has a power of
two per 32 columns, ``nvfp4`` an e4m3 scale per 16 columns and one fp32 scale per
tensor (per expert, for weights of experts). ``int4`` is the library's integer
format, q - 8 times an fp16 scale per group.
"""
import torch

own = False

MAX = 6.0                                   # largest e2m1 magnitude
BLOCK = {"mxfp4": 32, "nvfp4": 16}          # columns of one scale
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a large projection's weight, quantized when a checkpoint is converted
        {"name": "quant 14336x4096 nvfp4", "op": "quant", "M": 14336, "K": 4096, "format": "nvfp4", "silu": False,
         "dtype": "bf16"},
        # between the two expert projections of a prefill chunk: an odd number of rows
        {"name": "quant silu 4097x1408 mxfp4", "op": "quant", "M": 4097, "K": 1408, "format": "mxfp4", "silu": True,
         "dtype": "bf16"},
        # a few tokens through a small projection: the smallest call, launch latency counts
        {"name": "linear 5x2048x1408 mxfp4", "op": "linear", "M": 5, "N": 2048, "K": 1408, "format": "mxfp4",
         "bias": False, "dtype": "bf16"},
        # one decoded token through a large projection: the weights are read once
        {"name": "linear 1x14336x4096 nvfp4", "op": "linear", "M": 1, "N": 14336, "K": 4096, "format": "nvfp4",
         "bias": False, "dtype": "bf16"},
        # a decode batch
        {"name": "linear 64x4096x4096 mxfp4", "op": "linear", "M": 64, "N": 4096, "K": 4096, "format": "mxfp4",
         "bias": False, "dtype": "bf16"},
        # a ragged mixed batch of decode and prefill tokens, with bias, fp16 activations
        {"name": "linear 517x11008x4096 nvfp4", "op": "linear", "M": 517, "N": 11008, "K": 4096, "format": "nvfp4",
         "bias": True, "dtype": "fp16"},
        # a prefill chunk: the largest product
        {"name": "linear 4096x11008x4096 nvfp4", "op": "linear", "M": 4096, "N": 11008, "K": 4096, "format": "nvfp4",
         "bias": False, "dtype": "bf16"},
        # a decode batch through the gate_up projection of 64 experts: a few rows an expert
        {"name": "experts 24 tokens nvfp4", "op": "experts", "T": 24, "E": 64, "k": 8, "N": 2816, "K": 2048,
         "format": "nvfp4"},
        # the same projection for a prefill chunk: about 512 rows an expert
        {"name": "experts 4096 tokens mxfp4", "op": "experts", "T": 4096, "E": 64, "k": 8, "N": 2816, "K": 2048,
         "format": "mxfp4"},
        # one decoded token through a whole expert layer of int4 weights
        {"name": "layer 1 token int4", "op": "layer", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1408, "format": "int4",
         "group": 128, "groups": 1, "keep": 1, "scoring": "softmax", "bias": False, "renorm": True},
        # a few sequences through smaller experts, sigmoid scores with a balance bias, the best 3 of 8 expert groups
        {"name": "layer 5 tokens mxfp4", "op": "layer", "T": 5, "E": 96, "k": 6, "H": 1024, "I": 704,
         "format": "mxfp4", "group": 32, "groups": 8, "keep": 3, "scoring": "sigmoid", "bias": True, "renorm": True},
        # the largest batch of the call: most experts are read, some by several tokens
        {"name": "layer 16 tokens nvfp4", "op": "layer", "T": 16, "E": 64, "k": 8, "H": 2048, "I": 1408,
         "format": "nvfp4", "group": 16, "groups": 1, "keep": 1, "scoring": "sigmoid", "bias": False, "renorm": True},
    ]


def _log(rng, lo, hi, step=1):
    """An integer of [lo, hi], spread over its logarithm, a multiple of ``step``."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "experts", "layer", "layer"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    step = 128 if fmt == "mxfp4" else 64     # columns that the products take
    if op == "quant":
        K = _log(rng, 64, 8192, 32)
        silu = rng.random() < 0.4
        return {"op": op, "M": _log(rng, 1, max(16, 14336 * 4096 // (K * (2 if silu else 1)))), "K": K, "format": fmt,
                "silu": silu, "dtype": "bf16" if silu else rng.choice(["bf16", "fp16"])}
    if op == "linear":
        K, N = _log(rng, 256, 8192, step), _log(rng, 256, 14336, 8)
        return {"op": op, "M": min(_log(rng, 1, 4096), 4096 * 11008 * 4096 // (N * K)), "N": N, "K": K, "format": fmt,
                "bias": rng.random() < 0.3, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "experts":
        E, K, N = _log(rng, 4, 64), _log(rng, 256, 2048, step), _log(rng, 256, 2816, 8)
        return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)), "N": N, "K": K,
                "format": fmt}
    fmt = rng.choice(["int4", "int4", "mxfp4", "nvfp4"])
    groups = rng.choice([1, 1, 2, 4])
    E = groups * _log(rng, 4, 64 // groups)
    keep = rng.randint(max(1, groups // 2), groups)
    H, I = _log(rng, 256, 2048, 64), _log(rng, 128, 1408, 64)
    group = {"int4": rng.choice([32, 64, 128]), "mxfp4": 32, "nvfp4": 16}[fmt]
    if fmt == "int4" and (H % group or I % group):
        group = 64
    return {"op": op, "T": rng.randint(1, 16), "E": E, "k": rng.randint(1, min(8, keep * (E // groups))), "H": H,
            "I": I, "format": fmt, "group": group, "groups": groups, "keep": keep,
            "scoring": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.4, "renorm": rng.random() < 0.7}


def _weight_bytes(N, K, fmt, group=None):
    """Codes and scales of N x K weights."""
    return N * K // 2 + (2 * N * (K // group) if fmt == "int4" else N * (K // BLOCK[fmt]))


def work(case):
    c = case
    fmt = c["format"]
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        return {"bytes": M * K * (6 if c["silu"] else 4), "flops": M * K * (8 if c["silu"] else 4)}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _weight_bytes(N, K, fmt) + 2 * M * (K + N) + 2 * N * c["bias"], "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    active = E * (1 - (1 - k / E) ** T)       # experts that get a row, on average
    if c["op"] == "experts":
        N, K = c["N"], c["K"]
        return {"bytes": active * _weight_bytes(N, K, fmt) + 2 * T * K + 2 * T * k * N + 4 * T * k + 4 * (E + 1),
                "flops": 2 * T * k * N * K}
    H, I, g = c["H"], c["I"], c["group"]
    return {"bytes": active * (_weight_bytes(2 * I, H, fmt, g) + _weight_bytes(H, I, fmt, g)) + 4 * T * H + 4 * T * E,
            "flops": 6 * T * k * H * I}


# ---- inputs ----------------------------------------------------------------


def _activations(g, M, K, dtype):
    """N(0, 1) with one column in a hundred 20 times larger, as activations have."""
    x = torch.randn((M, K), generator=g, device="cuda")
    big = torch.rand((K,), generator=g, device="cuda") < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _weights(g, N, K, fmt, group=None):
    """N(0, 0.02^2) weights with a spread of row norms in a 4-bit format: codes, scales, tensor scale (or None)."""
    w = torch.randn((N, K), generator=g, device="cuda") * (0.02 * torch.rand((N, 1), generator=g, device="cuda") + 0.01)
    if fmt == "int4":
        p = w.view(N, K // group, group)
        s = (p.abs().amax(dim=2) / 7.5).half()
        q = (torch.round(p / s.float()[:, :, None]) + 8).clamp(0, 15).to(torch.int64).view(N, K // 8, 8)
        q = (q << (4 * torch.arange(8, device="cuda"))).sum(dim=2)
        return torch.where(q >= 1 << 31, q - (1 << 32), q).to(torch.int32), s, None
    t = (w.abs().amax() / (448.0 * MAX)).reshape(1) if fmt == "nvfp4" else None
    q, s = _quant(w, fmt, t)
    return _pack(q), s, t


def _stack(parts):
    q, s, t = zip(*parts)
    scales = torch.stack([x.view(torch.uint8) if x.dtype != torch.float16 else x for x in s])
    return (torch.stack(q), scales if s[0].dtype == torch.float16 else scales.view(s[0].dtype),
            None if t[0] is None else torch.cat(t))


def _act_scale(x, fmt):
    """A calibrated tensor scale of activations, for nvfp4."""
    return (x.float().abs().amax() / (448.0 * MAX)).reshape(1) if fmt == "nvfp4" else None


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    fmt = c["format"]
    if c["op"] == "quant":
        c["x"] = _activations(g, c["M"], c["K"] * (2 if c["silu"] else 1), _DTYPES[c["dtype"]])
        c["xt"] = _act_scale(c["x"], fmt)
    elif c["op"] == "linear":
        c["x"] = _activations(g, c["M"], c["K"], _DTYPES[c["dtype"]])
        c["xt"] = _act_scale(c["x"], fmt)
        c["w"], c["ws"], c["wt"] = _weights(g, c["N"], c["K"], fmt)
        c["b"] = (0.1 * torch.randn((c["N"],), generator=g, device="cuda")).to(torch.bfloat16) if c["bias"] else None
    elif c["op"] == "experts":
        T, E, k = c["T"], c["E"], c["k"]
        c["x"] = _activations(g, T, c["K"], torch.bfloat16)
        c["xt"] = _act_scale(c["x"], fmt)
        c["w"], c["ws"], c["wt"] = _stack([_weights(g, c["N"], c["K"], fmt) for _ in range(E)])
        ids = torch.randn((T, E), generator=g, device="cuda").topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        c["row_expert"] = ids[order]
        c["row_token"] = (order // k).to(torch.int32)
        c["offsets"] = torch.searchsorted(c["row_expert"], torch.arange(E + 1, device="cuda")).to(torch.int32)
        c["most"] = int((c["offsets"][1:] - c["offsets"][:-1]).max())     # rows of the fullest expert
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        c["x"] = _activations(g, T, H, torch.bfloat16)
        c["logits"] = torch.randn((T, E), generator=g, device="cuda")
        c["balance"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if c["bias"] else None
        c["up"], c["ups"], c["upt"] = _stack([_weights(g, 2 * I, H, fmt, c["group"]) for _ in range(E)])
        c["down"], c["downs"], c["downt"] = _stack([_weights(g, H, I, fmt, c["group"]) for _ in range(E)])
    return c


# ---- the plain forms -------------------------------------------------------


def _power(e):
    """2^e in 32 bits for whole numbers e of [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e2m1(v):
    """v rounded to the nearest e2m1 value, ties to the even code, held to +-6."""
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp(max=MAX), v)


def _quant(x, fmt, t):
    """e2m1 values and scales (e8m0 or e4m3) of x [M, K] in 32 bits, per row and block of columns."""
    M, K = x.shape
    p = x.view(M, -1, BLOCK[fmt])
    amax = p.abs().amax(dim=2)
    if fmt == "mxfp4":
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
        q = _e2m1(p * _power(-e)[:, :, None])
        return q.view(M, K), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    s = (amax / torch.full_like(amax, MAX) / t).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s.float() * t)[:, :, None]
    return torch.where(d > 0, _e2m1(p / d), 0.0).view(M, K), s


def _pack(v):
    """e2m1 values [M, K] as codes, two in a byte, the lower column in the low half."""
    m = v.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _values(q):
    """The e2m1 values of packed codes [..., K/2], as [..., K] in 32 bits."""
    both = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)
    m = (both & 7).float()
    m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(both > 7, -m, m)


def _scales(s, t):
    """Scales in 32 bits; t: the tensor's scale, or one per expert."""
    if s.dtype == torch.float8_e8m0fnu:
        return _power(s.view(torch.uint8).int() - 127)
    return s.float() * (t.view(-1, 1, 1) if s.dim() == 3 else t)


def _dequant(q, s, t, fmt):
    """Weights [..., N, K] as the values their codes stand for."""
    if fmt == "int4":
        q = (q[..., None] >> (4 * torch.arange(8, device=q.device))) & 15
        q = q.flatten(-2).float() - 8.0
        s = s.float()
    else:
        q, s = _values(q), _scales(s, t)
    return (q.view(*s.shape, -1) * s[..., None]).flatten(-2)


def _dequant_rows(x, fmt, t):
    """x after its quantization, as the values the codes stand for."""
    q, s = _quant(x, fmt, t)
    return (q.view(*s.shape, -1) * _scales(s, t)[..., None]).flatten(-2)


def _silu_mul(h):
    gate, up = h[..., :h.shape[-1] // 2], h[..., h.shape[-1] // 2:]
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_route(c):
    """Chosen experts and their weights, [T, k]."""
    x = c["logits"]
    T, E = x.shape
    G = c["groups"]
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        score = e / e.double().sum(dim=1, keepdim=True).float()
    key = x if c["balance"] is None else score + c["balance"]      # what the choice goes by
    if c["keep"] < G:
        by = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        group = by[:, :, 0] if c["balance"] is None or E == G else by[:, :, 0] + by[:, :, 1]
        best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones((T, G), dtype=torch.bool, device=x.device).scatter_(1, best, False)
        key = key.masked_fill(out.repeat_interleave(E // G, dim=1), -torch.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    return ids, w / w.sum(dim=1, keepdim=True) if c["renorm"] else w


def _plain(c):
    fmt, x = c["format"], c["x"].float()
    if c["op"] == "quant":
        return _dequant_rows(_silu_mul(x) if c["silu"] else x, fmt, c["xt"]).to(torch.bfloat16)
    if c["op"] == "linear":
        y = _dequant_rows(x, fmt, c["xt"]) @ _dequant(c["w"], c["ws"], c["wt"], fmt).T
        return (y if c["b"] is None else y + c["b"].float()).to(torch.bfloat16)
    if c["op"] == "experts":
        # every expert's rows in a block of their own, as many rows as the fullest has
        E, K = c["E"], c["K"]
        x = _dequant_rows(x, fmt, c["xt"])
        e = c["row_expert"]
        at = e * c["most"] + torch.arange(e.numel(), device=e.device) - c["offsets"].long()[e]
        p = torch.zeros((E * c["most"], K), device=x.device)
        p[at] = x[c["row_token"].long()]
        y = torch.bmm(p.view(E, c["most"], K), _dequant(c["w"], c["ws"], c["wt"], fmt).transpose(1, 2))
        return y.view(E * c["most"], -1)[at].to(torch.bfloat16)
    # layer: every expert on every token, of which the chosen ones count
    ids, w = _plain_route(c)
    a = _silu_mul(x @ _dequant(c["up"], c["ups"], c["upt"], fmt).transpose(1, 2))
    y = torch.bmm(a, _dequant(c["down"], c["downs"], c["downt"], fmt).transpose(1, 2))
    chosen = y[ids, torch.arange(c["T"], device=x.device)[:, None]]
    return (w[:, :, None] * chosen).sum(dim=1).to(torch.bfloat16)


def _library(c):
    import int4_weight_quantized_w4_gb300 as w4
    fmt = c["format"]
    if c["op"] == "quant":
        call = w4.w4_silu_mul_quant_fp4 if c["silu"] else w4.w4_quant_fp4
        q, s = call(c["x"], fmt, c["xt"])
        return w4.w4_dequant_fp4(q, s, fmt, c["xt"])
    if c["op"] == "linear":
        return w4.w4_fp4_gemm_bf16in(c["x"], c["w"], c["ws"], fmt, c["xt"], c["wt"], bias=c["b"])
    if c["op"] == "experts":
        return w4.w4_fp4_moe_gemm_bf16in(c["x"], c["row_token"], c["offsets"], c["w"], c["ws"], fmt, c["xt"], c["wt"])
    return w4.w4_moe_decode(c["x"], c["logits"], c["up"], c["ups"], c["down"], c["downs"], c["k"], fmt,
                            gate_up_global=c["upt"], down_global=c["downt"], bias=c["balance"], n_group=c["groups"],
                            topk_group=c["keep"], scoring=c["scoring"], renormalize=c["renorm"])


def run(state):
    return _library(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest_64(v):
    """v as the nearest e2m1 value, the one with the even code where two are as near: by the borders between them."""
    m, at = v.abs(), torch.zeros(v.shape, dtype=torch.int64, device=v.device)
    for i in range(7):
        border = (_GRID[i] + _GRID[i + 1]) / 2
        at += (m >= border) if i % 2 else (m > border)
    return torch.tensor(_GRID, dtype=torch.float64, device=v.device)[at] * torch.sign(v)


def _quant_64(x, fmt, t):
    """The values of x after its quantization; nvfp4's scales and quotients are 32-bit numbers by definition."""
    out, b = torch.zeros_like(x), BLOCK[fmt]
    for k in range(0, x.shape[1], b):
        p = x[:, k:k + b]
        a = p.abs().amax(dim=1, keepdim=True)
        if fmt == "mxfp4":
            d = torch.where(a > 0, torch.exp2((torch.frexp(a).exponent - 3).clamp(-127, 127).double()), 1.0)
            v = p / d
        else:
            g = t.double()
            s = ((a / 6.0).float().double() / g).float().double()
            e = (torch.frexp(s).exponent - 1).clamp(min=-6)
            unit = torch.ldexp(torch.ones_like(s), e - 3)
            s = (torch.round(s / unit) * unit).clamp(max=448.0)
            d = (s * g).float().double()
            v = torch.where(d > 0, p / torch.where(d > 0, d, 1.0), 0.0).float().double()
            d = s * g
        out[:, k:k + b] = _nearest_64(v) * d
    return out


def _weights_64(q, s, t, fmt):
    """One weight [N, K] as the values its codes stand for."""
    if fmt == "int4":
        v = torch.stack([(q >> (4 * j)) & 15 for j in range(8)], dim=2).flatten(1).double() - 8
        return v * s.double().repeat_interleave(v.shape[1] // s.shape[1], dim=1)
    code = torch.stack((q & 15, q >> 4), dim=2).flatten(1).long()
    v = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device=q.device)[code]
    s = torch.exp2(s.view(torch.uint8).double() - 127) if fmt == "mxfp4" else s.double() * t.double()
    return v * s.repeat_interleave(BLOCK[fmt], dim=1)


def exact(case, seed):
    c = prepare(case, seed)
    fmt, x = c["format"], c["x"].double()
    if c["op"] == "quant":
        if c["silu"]:
            x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
        return _quant_64(x, fmt, c["xt"])
    if c["op"] == "linear":
        y = _quant_64(x, fmt, c["xt"]) @ _weights_64(c["w"], c["ws"], c["wt"], fmt).T
        return y if c["b"] is None else y + c["b"].double()
    if c["op"] == "experts":
        off, rows = c["offsets"].tolist(), c["row_token"].long()
        x = _quant_64(x, fmt, c["xt"])
        t = c["wt"] if c["wt"] is not None else [None] * c["E"]
        return torch.cat([x[rows[a:b]] @ _weights_64(c["w"][e], c["ws"][e], t[e], fmt).T
                          for e, (a, b) in enumerate(zip(off, off[1:])) if b > a])
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.sigmoid(c["logits"].double()) if c["scoring"] == "sigmoid" else torch.softmax(c["logits"].double(), dim=1)
    key = c["logits"].double() if c["balance"] is None else score + c["balance"].double()
    y, size, top = torch.zeros_like(x), E // c["groups"], 1 if c["balance"] is None else 2
    pairs = {}
    for t in range(T):
        row = key[t].tolist()
        members = [range(i * size, (i + 1) * size) for i in range(c["groups"])]
        value = [sum(sorted((row[e] for e in m), reverse=True)[:top]) for m in members]
        kept = sorted(range(c["groups"]), key=lambda i: (-value[i], i))[:c["keep"]]
        allowed = [e for i in kept for e in members[i]]
        ids = sorted(allowed, key=lambda e: (-row[e], e))[:k]
        w = score[t, ids]
        w = w / w.sum() if c["renorm"] else w
        for e, v in zip(ids, w.tolist()):
            pairs.setdefault(e, []).append((t, v))
    for e, chosen in pairs.items():
        up = _weights_64(c["up"][e], c["ups"][e], None if c["upt"] is None else c["upt"][e], fmt)
        down = _weights_64(c["down"][e], c["downs"][e], None if c["downt"] is None else c["downt"][e], fmt)
        for t, v in chosen:
            h = up @ x[t]
            a = h[:c["I"]] * torch.sigmoid(h[:c["I"]]) * h[c["I"]:]
            y[t] += v * (down @ a)
    return y
