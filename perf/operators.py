"""Cases for measuring the fp8 block-scaled layer and its router.

Four operators, each in its plain form (elementary torch operations in 32
bits) and as the library's call; ``own`` says which one ``run`` makes:

* ``route``: grouped top-k routing of router logits, with the expert-sorted
  row order that the expert products read (``w4_moe_route_grouped``);
* ``quant``: e4m3 codes with one scale per token and 128 columns, of
  activations (``w4_quant_act_per_block``) or of silu(gate) * up
  (``w4_silu_mul_quant_block``);
* ``linear``: y = x W^T with e4m3 weights and one scale per 128 x 128 block,
  from 16-bit activations (``w4_fp8_block_gemm_bf16in``);
* ``experts``: the same product over the routed rows of a set of experts
  (``w4_fp8_block_moe_gemm_bf16in``).
"""
import torch

own = False

B = 128           # columns of one scale (and rows, for weights)
Q = 448.0         # largest e4m3 magnitude


def listed():
    return [
        # one decoded token through the router: latency only
        {"name": "route 1 token", "op": "route", "T": 1, "E": 64, "k": 8, "groups": 1, "keep": 1,
         "scoring": "sigmoid", "bias": True, "renorm": True, "dtype": "f32"},
        # a serving batch of odd size, softmax scores, the best 3 of 8 expert groups, bf16 logits (many ties)
        {"name": "route 333 softmax", "op": "route", "T": 333, "E": 96, "k": 6, "groups": 8, "keep": 3,
         "scoring": "softmax", "bias": False, "renorm": False, "dtype": "bf16"},
        # a long prefill over many experts, sigmoid scores with a balance bias, 4 of 8 groups
        {"name": "route 16384 sigmoid", "op": "route", "T": 16384, "E": 256, "k": 8, "groups": 8, "keep": 4,
         "scoring": "sigmoid", "bias": True, "renorm": True, "dtype": "f32"},
        # the input of a prefill projection, one token over a power of two
        {"name": "quant 4097x4096", "op": "quant", "M": 4097, "K": 4096, "silu": False, "dtype": "bf16"},
        # between the two expert projections of the 4096-token, top-8 layer
        {"name": "quant silu 32768x1408", "op": "quant", "M": 32768, "K": 1408, "silu": True, "dtype": "bf16"},
        # a few tokens through a small projection: the smallest call, launch latency counts
        {"name": "linear 5x2048x1408", "op": "linear", "M": 5, "N": 2048, "K": 1408, "bias": False, "dtype": "bf16"},
        # one decoded token through a large projection: the weights are read once
        {"name": "linear 1x14336x4096", "op": "linear", "M": 1, "N": 14336, "K": 4096, "bias": False,
         "dtype": "bf16"},
        # a decode batch
        {"name": "linear 64x4096x4096", "op": "linear", "M": 64, "N": 4096, "K": 4096, "bias": False,
         "dtype": "bf16"},
        # a ragged mixed batch of decode and prefill tokens, with bias, fp16 activations
        {"name": "linear 517x11008x4096", "op": "linear", "M": 517, "N": 11008, "K": 4096, "bias": True,
         "dtype": "fp16"},
        # a prefill chunk: compute bound
        {"name": "linear 4096x11008x4096", "op": "linear", "M": 4096, "N": 11008, "K": 4096, "bias": False,
         "dtype": "bf16"},
        # a decode batch through the gate_up projection of 64 experts: a few rows an expert
        {"name": "experts 24 tokens", "op": "experts", "T": 24, "E": 64, "k": 8, "N": 2816, "K": 2048},
        # the same projection for a prefill chunk: about 512 rows an expert
        {"name": "experts 4096 tokens", "op": "experts", "T": 4096, "E": 64, "k": 8, "N": 2816, "K": 2048},
    ]


def _log(rng, lo, hi, step=1):
    """An integer of [lo, hi], spread over its logarithm, a multiple of ``step``."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "quant", "linear", "linear", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 256 // groups)
        keep = rng.randint(max(1, groups // 4), groups)
        scoring = rng.choice(["sigmoid", "softmax"])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, keep * (E // groups))),
                "groups": groups, "keep": keep, "scoring": scoring, "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "dtype": rng.choice(["f32", "bf16"])}
    if op == "quant":
        K = _log(rng, 128, 8192, 16)
        silu = rng.random() < 0.5
        return {"op": op, "M": _log(rng, 1, max(16, 32768 * 1408 // K)), "K": K, "silu": silu,
                "dtype": "bf16" if silu else rng.choice(["bf16", "fp16"])}
    if op == "linear":
        K, N = _log(rng, 256, 8192, 16), _log(rng, 256, 14336, 8)
        return {"op": op, "M": min(_log(rng, 1, 4096), 4096 * 11008 * 4096 // (N * K)), "N": N, "K": K,
                "bias": rng.random() < 0.3, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    E, K, N = _log(rng, 4, 64), _log(rng, 256, 2048, 16), _log(rng, 256, 2816, 8)
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)), "N": N, "K": K}


def _blocks(n):
    return (n + B - 1) // B


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (4 if c["dtype"] == "f32" else 2) + 16 * T * k + 4 * (E + 1), "flops": 8 * T * E}
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        return {"bytes": M * K * (5 if c["silu"] else 3) + 4 * M * _blocks(K), "flops": M * K * (8 if c["silu"] else 3)}
    N, K = c["N"], c["K"]
    w = N * K + 4 * _blocks(N) * _blocks(K)
    if c["op"] == "linear":
        M = c["M"]
        return {"bytes": w + 2 * M * (K + N) + 2 * N * c["bias"], "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    active = E * (1 - (1 - k / E) ** T)       # experts that get a row, on average
    return {"bytes": active * w + 2 * T * K + 2 * T * k * N + 4 * T * k + 4 * (E + 1), "flops": 2 * T * k * N * K}


_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _activations(g, M, K, dtype):
    """N(0, 1) with one column in a hundred 20 times larger, as activations have."""
    x = torch.randn((M, K), generator=g, device="cuda")
    big = torch.rand((K,), generator=g, device="cuda") < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _weights(g, N, K):
    """N(0, 0.02^2) weights with a spread of row norms, quantized per 128 x 128 block."""
    w = torch.randn((N, K), generator=g, device="cuda") * (0.02 * torch.rand((N, 1), generator=g, device="cuda") + 0.01)
    nb, kb = _blocks(N), _blocks(K)
    p = torch.zeros((nb * B, kb * B), device="cuda")
    p[:N, :K] = w
    p = p.view(nb, B, kb, B)
    s = p.abs().amax(dim=(1, 3)) / Q
    q = (p / s[:, None, :, None]).clamp(-Q, Q).to(torch.float8_e4m3fn).view(nb * B, kb * B)
    return q.view(torch.uint8)[:N, :K].contiguous().view(torch.float8_e4m3fn), s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "route":
        c["logits"] = torch.randn((c["T"], c["E"]), generator=g, device="cuda").to(_DTYPES[c["dtype"]])
        c["balance"] = 0.1 * torch.randn((c["E"],), generator=g, device="cuda") if c["bias"] else None
    elif c["op"] == "quant":
        c["x"] = _activations(g, c["M"], c["K"] * (2 if c["silu"] else 1), _DTYPES[c["dtype"]])
    elif c["op"] == "linear":
        c["x"] = _activations(g, c["M"], c["K"], _DTYPES[c["dtype"]])
        c["w"], c["ws"] = _weights(g, c["N"], c["K"])
        c["b"] = (0.1 * torch.randn((c["N"],), generator=g, device="cuda")).to(torch.bfloat16) if c["bias"] else None
    else:
        T, E, k = c["T"], c["E"], c["k"]
        c["x"] = _activations(g, T, c["K"], torch.bfloat16)
        w = [_weights(g, c["N"], c["K"]) for _ in range(E)]
        c["w"] = torch.stack([q.view(torch.uint8) for q, _ in w]).view(torch.float8_e4m3fn)
        c["ws"] = torch.stack([s for _, s in w])
        ids = torch.randn((T, E), generator=g, device="cuda").topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        c["row_expert"] = ids[order]
        c["row_token"] = (order // k).to(torch.int32)
        c["offsets"] = torch.searchsorted(c["row_expert"], torch.arange(E + 1, device="cuda")).to(torch.int32)
        c["most"] = int((c["offsets"][1:] - c["offsets"][:-1]).max())     # rows of the fullest expert
    return c


# ---- the plain forms -------------------------------------------------------


def _split(x):
    """[M, K] in 32 bits as [M, blocks, 128], zeros past K."""
    M, K = x.shape
    p = torch.zeros((M, _blocks(K) * B), device=x.device)
    p[:, :K] = x
    return p.view(M, -1, B)


def _quant(x):
    """e4m3 codes and scales of x [M, K], per row and 128 columns."""
    M, K = x.shape
    p = _split(x)
    amax = p.abs().amax(dim=2)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, Q))
    q = (p / s[:, :, None]).clamp(-Q, Q).to(torch.float8_e4m3fn)
    return q.view(M, -1)[:, :K], s


def _dequant_rows(x):
    """x after its quantization, as the values the codes stand for."""
    q, s = _quant(x)
    return q.float() * s.repeat_interleave(B, dim=1)[:, :x.shape[1]]


def _dequant_weights(w, s):
    """Weights [..., N, K] as the values their codes stand for."""
    full = s.repeat_interleave(B, dim=-1).repeat_interleave(B, dim=-2)
    return w.float() * full[..., :w.shape[-2], :w.shape[-1]]


def _plain_route(c):
    x = c["logits"].float()
    T, E = x.shape
    k, G = c["k"], c["groups"]
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
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * 2.5
    flat = ids.reshape(-1)
    in_order, order = torch.sort(flat, stable=True)                 # rows by expert, then token
    row_of = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=x.device))
    offsets = torch.searchsorted(in_order, torch.arange(E + 1, device=x.device))
    i32 = torch.int32
    return ids.to(i32), w, offsets.to(i32), (order // k).to(i32), row_of.view(T, k).to(i32)


def _plain(c):
    if c["op"] == "route":
        return _plain_route(c)
    if c["op"] == "quant":
        x = c["x"].float()
        if c["silu"]:
            gate, up = x[:, :c["K"]], x[:, c["K"]:]
            x = gate / (1.0 + torch.exp(-gate)) * up
        return _quant(x)
    if c["op"] == "linear":
        y = _dequant_rows(c["x"].float()) @ _dequant_weights(c["w"], c["ws"]).T
        return (y if c["b"] is None else y + c["b"].float()).to(torch.bfloat16)
    # experts: every expert's rows in a block of their own, as many rows as the fullest has
    E, K = c["E"], c["K"]
    x = _dequant_rows(c["x"].float())
    e = c["row_expert"]
    at = e * c["most"] + torch.arange(e.numel(), device=e.device) - c["offsets"].long()[e]
    p = torch.zeros((E * c["most"], K), device=x.device)
    p[at] = x[c["row_token"].long()]
    y = torch.bmm(p.view(E, c["most"], K), _dequant_weights(c["w"], c["ws"]).transpose(1, 2))
    return y.view(E * c["most"], -1)[at].to(torch.bfloat16)


def _library(c):
    import int4_weight_quantized_w4_gb300 as w4
    if c["op"] == "route":
        return w4.w4_moe_route_grouped(c["logits"], c["k"], bias=c["balance"], n_group=c["groups"],
                                       topk_group=c["keep"], scoring=c["scoring"], renormalize=c["renorm"], scale=2.5)
    if c["op"] == "quant":
        return w4.w4_silu_mul_quant_block(c["x"]) if c["silu"] else w4.w4_quant_act_per_block(c["x"])
    if c["op"] == "linear":
        return w4.w4_fp8_block_gemm_bf16in(c["x"], c["w"], c["ws"], bias=c["b"])
    return w4.w4_fp8_block_moe_gemm_bf16in(c["x"], c["row_token"], c["offsets"], c["w"], c["ws"])


def run(state):
    return _library(state) if own else _plain(state)


# ---- the definition in 64 bits ---------------------------------------------


def _e4m3_64(v):
    """v rounded to the nearest e4m3 value, ties to even, held to +-448."""
    e = (torch.frexp(v).exponent - 1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / step) * step).clamp(-Q, Q)


def _quant_64(x):
    """Codes (as values) and scales of x in 64 bits; the scale and each quotient are 32-bit numbers by definition."""
    q, s = torch.zeros_like(x), []
    for k in range(0, x.shape[1], B):
        a = x[:, k:k + B].abs().amax(dim=1, keepdim=True)
        sk = torch.where(a > 0, a / Q, torch.ones_like(a)).float().double()
        q[:, k:k + B] = _e4m3_64((x[:, k:k + B] / sk).float().double())
        s.append(sk)
    return q, torch.cat(s, dim=1)


def _product_64(x, w, ws):
    """Quantized rows x [M, K] times W [N, K], one pair of blocks at a time."""
    q, s = _quant_64(x)
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    for i, k in enumerate(range(0, x.shape[1], B)):
        part = q[:, k:k + B] @ w[:, k:k + B].double().T
        y += s[:, i:i + 1] * part * ws[:, i].double().repeat_interleave(B)[:w.shape[0]]
    return y


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "route":
        x = c["logits"].double()
        score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, dim=1)
        key = (x if c["balance"] is None else score + c["balance"].double()).cpu()
        score, size, chosen = score.cpu(), c["E"] // c["groups"], []
        for t in range(min(c["T"], 16384)):
            row = key[t].tolist()
            members = [range(i * size, (i + 1) * size) for i in range(c["groups"])]
            top = 1 if c["balance"] is None else 2
            value = [sum(sorted((row[e] for e in m), reverse=True)[:top]) for m in members]
            kept = sorted(range(c["groups"]), key=lambda i: (-value[i], i))[:c["keep"]]
            allowed = [e for i in kept for e in members[i]]
            chosen.append(sorted(allowed, key=lambda e: (-row[e], e))[:c["k"]])
        w = score.gather(1, torch.tensor(chosen))
        w = w / w.sum(dim=1, keepdim=True) if c["renorm"] else w
        return None, 2.5 * w, None, None, None
    x = c["x"].double()
    if c["op"] == "quant":
        if c["silu"]:
            x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
        return _quant_64(x)
    if c["op"] == "linear":
        y = _product_64(x, c["w"], c["ws"])
        return y if c["b"] is None else y + c["b"].double()
    off = c["offsets"].tolist()
    rows = c["row_token"].long()
    return torch.cat([_product_64(x[rows[a:b]], c["w"][e], c["ws"][e]) for e, (a, b) in
                      enumerate(zip(off, off[1:])) if b > a])
