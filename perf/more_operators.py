"""Workloads of a feed-forward layer's training step: the gated feed-forward block on
FP8 operands and its backward pass, the FP8 quantiser that makes their operands, and the
Newton-Schulz orthogonalisation of the weight gradient.

Each case names one operator and its sizes.  ``run`` computes it either in plain
torch operations in 32 bits (``own`` false) or through the library (``own``
true); ``exact`` gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
COEF = (3.4445, -4.7750, 2.0315)    # a, b, c of X <- a X + (b A + c A A) X, A = X X^T
EPS = 1e-7

# Largest amount of work drawn for each operator (that of its largest listed case).
FFN_MAX = 8192 * 2048 * 7168
FFN_MAX_WEIGHTS = 8 * 2048 * 7168
QUANT_MAX = 8 * 4096 * 7168
NS_MAX = 4 * 2048 * 2048 * (2 * 7168 + 2048)


def listed():
    return [
        # a few rows through a small model's block: latency counts
        {"name": "ffn 7x1408x2048", "op": "ffn", "e": 1, "m": 7, "i": 1408, "k": 2048, "save": False},
        # a training batch of a shared expert; gate and up are kept for the backward pass
        {"name": "ffn 4096x2048x7168 saved", "op": "ffn", "e": 1, "m": 4096, "i": 2048, "k": 7168, "save": True},
        # a prefill chunk's experts, rows sorted by expert, ragged counts padded to whole blocks
        {"name": "ffn e8 8192x2048x7168", "op": "ffn", "e": 8, "m": 8192, "i": 2048, "k": 7168, "save": False},
        # backward: a ragged batch of a small model, a width that is no multiple of 128
        {"name": "ffn_bwd 515x1360x2048", "op": "ffn_bwd", "e": 1, "m": 515, "i": 1360, "k": 2048},
        # backward of the shared expert's training batch
        {"name": "ffn_bwd 4096x2048x7168", "op": "ffn_bwd", "e": 1, "m": 4096, "i": 2048, "k": 7168},
        # backward of routed experts
        {"name": "ffn_bwd e8 8192x2048x7168", "op": "ffn_bwd", "e": 8, "m": 8192, "i": 2048, "k": 7168},
        # activations of a small batch before a product: nothing but latency
        {"name": "quant rows 96x7168 bf16", "op": "quant", "form": "rows", "b": 1, "r": 96, "c": 7168, "dtype": "bf16"},
        # activations or gradients of a training batch, for the products along both of their axes
        {"name": "quant both 8192x7168 bf16", "op": "quant", "form": "both", "b": 1, "r": 8192, "c": 7168,
         "dtype": "bf16"},
        # FP32 master weights of eight experts after an update
        {"name": "quant blocks 8x4096x7168 f32", "op": "quant", "form": "blocks", "b": 8, "r": 4096, "c": 7168,
         "dtype": "f32"},
        # the update of a small projection, an odd size; launches and latency count
        {"name": "ns 1x250x1000 f32", "op": "ns", "b": 1, "r": 250, "c": 1000, "dtype": "f32", "steps": 5},
        # a tall 16-bit gradient: the short side is the columns
        {"name": "ns 2x2112x1536 bf16", "op": "ns", "b": 2, "r": 2112, "c": 1536, "dtype": "bf16", "steps": 5},
        # the weight gradients of four experts
        {"name": "ns 4x2048x7168 f32", "op": "ns", "b": 4, "r": 2048, "c": 7168, "dtype": "f32", "steps": 5},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("ffn", "ffn_bwd", "quant", "ns"))
    while True:
        if op in ("ffn", "ffn_bwd"):
            e = rng.choice((1, 1, rng.randint(2, 16)))
            c = {"op": op, "e": e, "m": _log_int(rng, 1, 8192), "i": 16 * _log_int(rng, 16, 448),
                 "k": 16 * _log_int(rng, 16, 448)}
            if e > 1:
                c["m"] = 128 * max(1, c["m"] // 128)
                c["k"] = 128 * max(1, c["k"] // 128)
            if op == "ffn":
                c["save"] = rng.random() < 0.5
            if c["m"] * c["i"] * c["k"] <= FFN_MAX and c["e"] * c["i"] * c["k"] <= FFN_MAX_WEIGHTS:
                return c
        elif op == "quant":
            form = rng.choice(("rows", "both", "blocks"))
            c = {"op": op, "form": form, "b": rng.randint(1, 8) if form == "blocks" else 1,
                 "r": _log_int(rng, 1, 16384), "c": 16 * _log_int(rng, 4, 1024), "dtype": rng.choice(("bf16", "f32"))}
            if c["b"] * c["r"] * c["c"] <= QUANT_MAX:
                return c
        else:
            c = {"op": op, "b": rng.randint(1, 4), "r": _log_int(rng, 24, 7168), "c": _log_int(rng, 24, 7168),
                 "dtype": rng.choice(("bf16", "f32")), "steps": 5}
            lo, hi = sorted((c["r"], c["c"]))
            if c["b"] * lo * lo * (2 * hi + lo) <= NS_MAX:
                return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _exps(amax):
    """Biased exponent of the smallest power of two s with amax / s <= 448 (1 for 0)."""
    mant, e = torch.frexp(amax.to(torch.float32))               # amax = mant 2^e, 448 = 0.875 2^9
    p = e - 9 + (mant > 0.875).to(torch.int32)
    return torch.where(amax == 0, torch.full_like(p, 127), (p + 127).clamp(1, 254)).to(torch.int32)


def _pad(n, to):
    return (n + to - 1) // to * to


def _pack(exps, mn):
    """[groups, mn] biased exponents (any leading dimensions) -> int32 words [ceil(groups/4), align4(mn)]."""
    gk = exps.shape[-2]
    w = torch.zeros(*exps.shape[:-2], _pad(gk, 4), _pad(mn, 4), dtype=torch.int32, device=exps.device)
    w[..., :gk, :mn] = exps
    w = w.unflatten(-2, (-1, 4))
    return (w[..., 0, :] | (w[..., 1, :] << 8) | (w[..., 2, :] << 16) | (w[..., 3, :] << 24)).contiguous()


def _pow2(exps):
    """2^(exps - 127) in FP32, exactly (made from its bits)."""
    return (exps.to(torch.int32) << 23).view(torch.float32)


def _codes(x, exps):
    """E4M3 codes of x (FP32) over its scales (both of one shape, or broadcast)."""
    return (x * _pow2(254 - exps)).to(torch.float8_e4m3fn)


def _quant_rows(x):
    """x [R, C] -> codes and exponents [ceil(C/128), R], a scale for each 1 x 128."""
    r, c = x.shape
    v = torch.nn.functional.pad(x, (0, _pad(c, 128) - c)).view(r, -1, 128)
    e = _exps(v.abs().amax(-1))
    return _codes(v, e[..., None]).view(r, -1)[:, :c].contiguous(), e.t()


def _quant_cols(x):
    """x [R, C] -> codes and exponents [ceil(R/128), C], a scale for each 128 x 1."""
    r, c = x.shape
    v = torch.nn.functional.pad(x, (0, 0, 0, _pad(r, 128) - r)).view(-1, 128, c)
    e = _exps(v.abs().amax(1))
    return _codes(v, e[:, None, :]).view(-1, c)[:r].contiguous(), e


def _quant_blocks(w):
    """w [B, R, C] -> codes and exponents [B, ceil(R/128), ceil(C/128)], a scale for each 128 x 128."""
    b, r, c = w.shape
    v = torch.nn.functional.pad(w, (0, _pad(c, 128) - c, 0, _pad(r, 128) - r)).view(b, _pad(r, 128) // 128, 128, -1, 128)
    e = _exps(v.abs().amax(dim=(2, 4)))
    return _codes(v, e[:, :, None, :, None]).view(b, _pad(r, 128), -1)[:, :r, :c].contiguous(), e


def _weights(g, e, n, k, std):
    """Gaussian weights [e, n, k]: codes and block exponents [e, ceil(n/128), ceil(k/128)]."""
    made = [_quant_blocks(std * torch.randn(1, n, k, generator=g, device=DEV)) for _ in range(e)]
    return torch.cat([q for q, _ in made]), torch.cat([x for _, x in made])


def _words_nt(exps, n):
    """Block exponents [e, n blocks, k blocks] -> packed words of an [n][k] operand used along k."""
    return _pack(exps.repeat_interleave(128, 1)[:, :n].transpose(1, 2), n)


def _layout(g, m, e):
    """Expert of each row: ragged counts of at least one expert, each padded to whole blocks of 128."""
    blocks = m // 128
    cut = torch.sort(torch.randint(0, blocks + 1, (e - 1,), generator=g, device=DEV))[0]
    which = (torch.arange(blocks, device=DEV)[:, None] >= cut[None, :]).sum(1)
    return which.repeat_interleave(128).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("ffn", "ffn_bwd"):
        e, m, i, k = case["e"], case["m"], case["i"], case["k"]
        bf16 = dict(dtype=torch.bfloat16, device=DEV)
        s["layout"] = _layout(g, m, e) if e > 1 else None
        s["w2"], s["e2"] = _weights(g, e, k, i, i ** -0.5)
        # activations as a norm leaves them, a few channels larger than the rest; gradients are small
        x = torch.randn(m, k, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))
        if case["op"] == "ffn":
            s["w1"], s["e1"] = _weights(g, e, 2 * i, k, k ** -0.5)
            s["sf1"], s["sf2"] = _words_nt(s["e1"], 2 * i), _words_nt(s["e2"], k)
            s["x"], s["ex"] = _quant_rows(x)
            s["gu"] = torch.empty(m, 2 * i, **bf16) if case["save"] else None
            s["y"] = torch.empty(m, k, **bf16)
            s["hq"] = torch.empty(m, i, dtype=torch.float8_e4m3fn, device=DEV)
            s["sfh"] = torch.empty((i + 511) // 512, _pad(m, 4), dtype=torch.int32, device=DEV)
        else:
            s["sf2"] = _pack(s["e2"].repeat_interleave(128, 2)[..., :i], i)
            s["x"], s["ex"] = _quant_rows(1e-3 * x)
            s["gu"] = torch.randn(m, 2 * i, generator=g, device=DEV).to(torch.bfloat16)
            s["dgu"] = torch.empty(m, 2 * i, **bf16)
            s["h"] = torch.empty(m, i, **bf16)
        s["sfx"] = _pack(s["ex"], m)
        return s
    b, r, c = case["b"], case["r"], case["c"]
    if case["op"] == "quant":
        x = torch.randn(b, r, c, generator=g, device=DEV) * torch.exp(0.7 * torch.randn(c, generator=g, device=DEV))
        if case["form"] == "blocks":
            x *= c ** -0.5
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        u8 = dict(dtype=torch.float8_e4m3fn, device=DEV)
        i32 = dict(dtype=torch.int32, device=DEV)
        if case["form"] == "blocks":
            s["q"] = torch.empty(b, r, c, **u8)
            s["sf"] = torch.empty(b, (c + 511) // 512, _pad(r, 4), **i32)
            s["sft"] = torch.empty(b, (r + 511) // 512, _pad(c, 4), **i32)
        else:
            s["x"] = s["x"][0]
            s["q"], s["sf"] = torch.empty(r, c, **u8), torch.empty((c + 511) // 512, _pad(r, 4), **i32)
            if case["form"] == "both":
                s["qk"], s["sfk"] = torch.empty(r, c, **u8), torch.empty((r + 511) // 512, _pad(c, 4), **i32)
        return s
    # a gradient: a few strong directions over noise, of small magnitude
    low = torch.randn(b, r, 8, generator=g, device=DEV) @ torch.randn(b, 8, c, generator=g, device=DEV)
    grad = 1e-3 * (torch.randn(b, r, c, generator=g, device=DEV) + 0.3 * low)
    s["g"] = grad.to(torch.bfloat16) if case["dtype"] == "bf16" else grad
    s["out"] = torch.empty(b, r, c, dtype=torch.bfloat16, device=DEV)
    if own:
        from block_scaled_fp8_gb300 import binding as dg
        s["ws"] = torch.empty(dg.newton_schulz_workspace_bytes(b, r, c), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _values(q, exps_rows):
    """Codes [R, C] and exponents [groups, R], a scale for each 1 x 128 -> FP32."""
    r, c = q.shape
    s = _pow2(exps_rows.t())
    return q.to(torch.float32) * s.repeat_interleave(128, 1)[:, :c]


def _block_values(q, exps):
    """Codes [n, k] and block exponents -> FP32."""
    n, k = q.shape
    s = _pow2(exps)
    return q.to(torch.float32) * s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def _ffn_plain(s):
    x = _values(s["x"], s["ex"])
    m, i = s["m"], s["i"]
    gu = x.new_empty(m, 2 * i)
    y = x.new_empty(m, s["k"])
    for j in range(s["e"]):
        rows = (s["layout"] == j).nonzero().flatten() if s["e"] > 1 else slice(None)
        gu[rows] = x[rows] @ _block_values(s["w1"][j], s["e1"][j]).t()
    g, u = gu[:, :i], gu[:, i:]
    h = _values(*_quant_rows(g / (1.0 + torch.exp(-g)) * u))
    for j in range(s["e"]):
        rows = (s["layout"] == j).nonzero().flatten() if s["e"] > 1 else slice(None)
        y[rows] = h[rows] @ _block_values(s["w2"][j], s["e2"][j]).t()
    y = y.to(torch.bfloat16)
    return {"y": y, "gu": gu.to(torch.bfloat16)} if s["save"] else {"y": y}


def _ffn_bwd_plain(s):
    dy = _values(s["x"], s["ex"])
    m, i = s["m"], s["i"]
    dh = dy.new_empty(m, i)
    for j in range(s["e"]):
        rows = (s["layout"] == j).nonzero().flatten() if s["e"] > 1 else slice(None)
        dh[rows] = dy[rows] @ _block_values(s["w2"][j], s["e2"][j])
    g, u = s["gu"][:, :i].to(torch.float32), s["gu"][:, i:].to(torch.float32)
    sig = 1.0 / (1.0 + torch.exp(-g))
    dgu = torch.cat((dh * u * (sig * (1.0 + g * (1.0 - sig))), dh * (g * sig)), 1)
    return {"dgu": dgu.to(torch.bfloat16), "h": (g * sig * u).to(torch.bfloat16)}


def _quant_plain(s):
    x = s["x"].to(torch.float32)
    r, c = s["r"], s["c"]
    if s["form"] == "blocks":
        q, e = _quant_blocks(x)
        return {"q": q, "sf": _words_nt(e, r), "sft": _pack(e.repeat_interleave(128, 2)[..., :c], c)}
    q, e = _quant_rows(x)
    out = {"q": q, "sf": _pack(e, r)}
    if s["form"] == "both":
        q, e = _quant_cols(x)
        out.update(qk=q, sfk=_pack(e, c))
    return out


def _ns_plain(s):
    x = s["g"].to(torch.float32)
    tall = s["r"] > s["c"]
    if tall:
        x = x.transpose(1, 2)
    # the sum of squares of a large matrix in 64 bits
    x = x / (x.double().square().sum(dim=(1, 2), keepdim=True).sqrt().to(torch.float32) + EPS)
    a, b, c = COEF
    for _ in range(s["steps"]):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        return {"ffn": _ffn_plain, "ffn_bwd": _ffn_bwd_plain, "quant": _quant_plain, "ns": _ns_plain}[s["op"]](s)
    from block_scaled_fp8_gb300 import binding as dg
    if s["op"] == "ffn":
        if s["e"] > 1:
            dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(s["x"], s["sfx"], s["w1"], s["sf1"], s["layout"], hq=s["hq"],
                                                         sfh=s["sfh"], gu=s["gu"])
            dg.dg_m_grouped_fp8_gemm_nt_contiguous(s["hq"], s["sfh"], s["w2"], s["sf2"], s["y"], s["layout"])
        else:
            dg.dg_fp8_gated_gemm_nt(s["x"], s["sfx"], s["w1"][0], s["sf1"][0], hq=s["hq"], sfh=s["sfh"], gu=s["gu"])
            dg.dg_fp8_gemm_nt(s["hq"], s["sfh"], s["w2"][0], s["sf2"][0], s["y"])
        return {"y": s["y"], "gu": s["gu"]} if s["save"] else {"y": s["y"]}
    if s["op"] == "ffn_bwd":
        if s["e"] > 1:
            dg.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(s["x"], s["sfx"], s["w2"], s["sf2"], s["layout"],
                                                                  s["gu"], s["dgu"], h=s["h"])
        else:
            dg.dg_fp8_gated_gemm_nn_backward(s["x"], s["sfx"], s["w2"][0], s["sf2"][0], s["gu"], s["dgu"], h=s["h"])
        return {"dgu": s["dgu"], "h": s["h"]}
    if s["op"] == "quant":
        if s["form"] == "blocks":
            dg.dg_quantize_fp8_blocks(s["x"], s["q"], sf=s["sf"], sft=s["sft"])
            return {"q": s["q"], "sf": s["sf"], "sft": s["sft"]}
        if s["form"] == "both":
            dg.dg_quantize_fp8(s["x"], q=s["q"], sf=s["sf"], qk=s["qk"], sfk=s["sfk"])
            return {"q": s["q"], "sf": s["sf"], "qk": s["qk"], "sfk": s["sfk"]}
        dg.dg_quantize_fp8(s["x"], q=s["q"], sf=s["sf"])
        return {"q": s["q"], "sf": s["sf"]}
    return dg.dg_newton_schulz(s["g"], s["out"], steps=s["steps"], coef=COEF, eps=EPS, workspace=s["ws"])


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] in ("ffn", "ffn_bwd"):
        m, i, k = case["m"], case["i"], case["k"]
        e = min(case["e"], (m + 127) // 128)
        per = 1 + 1 / 128
        if case["op"] == "ffn":
            return {"bytes": e * 3 * i * k * per + m * k * (per + 2) + (4 * m * i if case["save"] else 0),
                    "flops": 6 * m * i * k}
        return {"bytes": e * i * k * per + m * k * per + m * i * (4 + 4 + 2), "flops": 2 * m * i * k}
    n = case["b"] * case["r"] * case["c"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quant":
        if case["form"] == "blocks":
            return {"bytes": n * (size + 1 + 2 / 128), "flops": 3 * n}
        two = 2 if case["form"] == "both" else 1
        return {"bytes": n * (size + two * (1 + 1 / 128)), "flops": 3 * two * n}
    lo, hi = sorted((case["r"], case["c"]))
    # both symmetric products need half of their results
    return {"bytes": n * (size + 2), "flops": case["b"] * case["steps"] * lo * lo * (3 * hi + lo)}


# ------------------------------------------------------------------ the definition in 64 bits

def _two64(p):
    """2^p in 64 bits, exactly."""
    return ((p.to(torch.int64) + 1023) << 52).view(torch.float64)


def _scale64(amax):
    """2^ceil(log2(amax / 448)) in 64 bits by comparison, 1 for 0; and the same for what is below the smallest scale."""
    p = torch.floor(torch.log2(amax.clamp_min(1e-290) / 448.0)) - 1
    for _ in range(3):
        p = torch.where(448.0 * _two64(p) < amax, p + 1, p)
    return torch.where(amax == 0, torch.ones_like(p), _two64(p.clamp(-126, 127)))


def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) in 64 bits; |v| <= 448."""
    exp = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    exp = torch.where(_two64(exp) > v.abs().clamp_min(2.0 ** -6), exp - 1, exp)
    exp = torch.where(_two64(exp + 1) <= v.abs(), exp + 1, exp)
    step = _two64(exp - 3)
    return torch.round(v / step) * step


def _words64(scale, mn):
    """Scales [..., groups, mn] -> packed words."""
    return _pack((torch.log2(scale).round() + 127).to(torch.int32), mn)


def _group64(x, dim, size=128):
    """Largest magnitude of each run of `size` along `dim`, spread back over the run, and by run."""
    runs = [t.abs().amax(dim) for t in x.split(size, dim)]
    by_run = torch.stack(runs, dim)
    return by_run, by_run.repeat_interleave(size, dim).narrow(dim, 0, x.shape[dim])


def _deq64(q, exps, n_first):
    """Codes [n, k], exponents of 1 x 128 (n_first: [groups, n]) or of 128 x 128 blocks -> 64 bits."""
    n, k = q.shape
    row = torch.arange(n, device=q.device)[:, None]
    col = torch.arange(k, device=q.device)[None, :] // 128
    e = exps[col, row] if n_first else exps[row // 128, col]
    return q.double() * _two64(e - 127)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ffn", "ffn_bwd"):
        if case["m"] * case["i"] * case["k"] > 1.3 * FFN_MAX:
            return None
        m, i, k = case["m"], case["i"], case["k"]
        x = _deq64(s["x"], s["ex"], True)
        owner = s["layout"] if s["e"] > 1 else torch.zeros(m, dtype=torch.int32, device=DEV)
        first = torch.zeros(m, 2 * i if case["op"] == "ffn" else i, dtype=torch.float64, device=DEV)
        for j in range(case["e"]):
            who = (owner == j).nonzero().flatten()
            if case["op"] == "ffn":
                first[who] = x[who] @ _deq64(s["w1"][j], s["e1"][j], False).t()
            else:
                first[who] = x[who] @ _deq64(s["w2"][j], s["e2"][j], False)
        if case["op"] == "ffn_bwd":
            g, u = s["gu"].double().split(i, 1)
            sg = torch.sigmoid(g)
            dsilu = sg + g * sg * (1 - sg)
            return {"dgu": torch.cat((first * u * dsilu, first * g * sg), 1), "h": g * sg * u}
        g, u = first.split(i, 1)
        h = torch.nn.functional.silu(g) * u
        scale = _scale64(_group64(h, 1)[1])
        h = _e4m3_64(h / scale) * scale
        y = torch.zeros(m, k, dtype=torch.float64, device=DEV)
        for j in range(case["e"]):
            who = (owner == j).nonzero().flatten()
            y[who] = h[who] @ _deq64(s["w2"][j], s["e2"][j], False).t()
        return {"y": y, "gu": first} if case["save"] else {"y": y}
    if case["op"] == "quant":
        x, r, c = s["x"].double(), case["r"], case["c"]
        if case["form"] == "blocks":
            b, nr = case["b"], (r + 127) // 128
            amax = _group64(_group64(x, 1)[0], 2)[0]
            scale = _scale64(amax)
            q = torch.empty_like(x)
            for j in range(b):
                full = scale[j].repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :c]
                q[j] = _e4m3_64(x[j] / full)
            return {"q": q, "sf": _words64(scale.transpose(1, 2).repeat_interleave(128, 2)[..., :r], r),
                    "sft": _words64(scale.repeat_interleave(128, 2)[..., :c], c)} if nr else None
        out = {}
        for dim, q, sf in ((1, "q", "sf"), (0, "qk", "sfk"))[:2 if case["form"] == "both" else 1]:
            by_run, full = _group64(x, dim)
            out[q] = _e4m3_64(x / _scale64(full))
            out[sf] = _words64(_scale64(by_run.t() if dim == 1 else by_run), r if dim == 1 else c)
        return out
    lo, hi = sorted((case["r"], case["c"]))
    if case["b"] * case["steps"] * lo * lo * (4 * hi + 2 * lo) > 1.5e13:
        return None
    out = torch.empty(case["b"], case["r"], case["c"], dtype=torch.float64, device=DEV)
    for j in range(case["b"]):
        x = s["g"][j].double()
        x = x / (torch.linalg.matrix_norm(x) + EPS)
        for _ in range(case["steps"]):
            if case["r"] <= case["c"]:
                p = x @ x.t()
                x = COEF[0] * x + COEF[1] * (p @ x) + COEF[2] * (p @ (p @ x))
            else:
                p = x.t() @ x
                x = COEF[0] * x + COEF[1] * (x @ p) + COEF[2] * ((x @ p) @ p)
        out[j] = x
    return out
