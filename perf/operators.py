"""Workloads of the decode-side operators: few-row products with 4- and 8-bit
weights, top-k routing, and the mixture-of-experts layer for few tokens.

Each case names one operator and its sizes.  ``run`` computes it either in plain
torch operations in 32 bits (``own`` false) or through the library (``own``
true); ``exact`` gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# Largest amount of work drawn for each operator (that of its largest listed case).
GEMV_MAX_NK = 131064 * 7168
MOE_MAX_EHI = 64 * 7168 * 2048
ROUTE_MAX_TE = 32768 * 256


def listed():
    return [
        # one token through the latent down-projection of a decode step: 8 MB of codes, latency counts
        {"name": "gemv fp4 1x2112x7168", "op": "gemv", "fmt": "fp4", "m": 1, "n": 2112, "k": 7168, "out": "bf16",
         "c": False},
        # one token through a wide up-projection with a short K
        {"name": "gemv fp4 1x24576x1536", "op": "gemv", "fmt": "fp4", "m": 1, "n": 24576, "k": 1536, "out": "bf16",
         "c": False},
        # a few tokens (speculative decoding) through an output projection, added to the residual stream
        {"name": "gemv fp4 5x7168x16384 c", "op": "gemv", "fmt": "fp4", "m": 5, "n": 7168, "k": 16384, "out": "bf16",
         "c": True},
        # a small batch through a projection with 8-bit weights
        {"name": "gemv fp8 17x4096x7168", "op": "gemv", "fmt": "fp8", "m": 17, "n": 4096, "k": 7168, "out": "bf16",
         "c": False},
        # a full decode batch through a vocabulary projection, FP32 logits; the largest product
        {"name": "gemv fp4 64x131064x7168 f32", "op": "gemv", "fmt": "fp4", "m": 64, "n": 131064, "k": 7168,
         "out": "f32", "c": False},
        # routing of a single token: one launch, nothing but latency
        {"name": "route 1x256 top8 sigmoid", "op": "route", "t": 1, "e": 256, "topk": 8, "scoring": "sigmoid",
         "bias": True, "dtype": "f32"},
        # routing of a chunk of a prompt, an odd number of tokens, 16-bit logits (many ties)
        {"name": "route 4099x128 top6 softmax", "op": "route", "t": 4099, "e": 128, "topk": 6, "scoring": "softmax",
         "bias": False, "dtype": "bf16"},
        # routing of a large prefill batch
        {"name": "route 32768x256 top8 sigmoid", "op": "route", "t": 32768, "e": 256, "topk": 8,
         "scoring": "sigmoid", "bias": True, "dtype": "f32"},
        # the MoE layer for a single token
        {"name": "moe fp4 t1 e64 7168x2048", "op": "moe", "fmt": "fp4", "t": 1, "e": 64, "topk": 8, "h": 7168,
         "i": 2048, "c": False, "masked": 0.0},
        # a small model's layer with an odd number of tokens and of 128-wide blocks; latency counts
        {"name": "moe fp4 t7 e64 2048x1408", "op": "moe", "fmt": "fp4", "t": 7, "e": 64, "topk": 6, "h": 2048,
         "i": 1408, "c": False, "masked": 0.0},
        # 8-bit experts of which some live on another device (their slots are -1), added to the residual stream
        {"name": "moe fp8 t16 e32 7168x2048 c", "op": "moe", "fmt": "fp8", "t": 16, "e": 32, "topk": 8, "h": 7168,
         "i": 2048, "c": True, "masked": 0.25},
        # a full decode batch: every expert is read
        {"name": "moe fp4 t64 e64 7168x2048", "op": "moe", "fmt": "fp4", "t": 64, "e": 64, "topk": 8, "h": 7168,
         "i": 2048, "c": False, "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("gemv", "gemv", "route", "moe", "moe"))
    while True:
        if op == "gemv":
            c = {"op": op, "fmt": rng.choice(("fp4", "fp8")), "m": _log_int(rng, 1, 64),
                 "n": 8 * _log_int(rng, 32, 16383), "k": 128 * _log_int(rng, 2, 128),
                 "out": rng.choice(("bf16", "f32")), "c": rng.random() < 0.3}
            bits = 1 if c["fmt"] == "fp4" else 2
            if c["n"] * c["k"] * bits <= GEMV_MAX_NK and 3072 not in (c["n"], c["k"]):
                return c
        elif op == "route":
            e = _log_int(rng, 4, 512)
            c = {"op": op, "t": _log_int(rng, 1, 32768), "e": e, "topk": rng.randint(1, min(10, e)),
                 "scoring": rng.choice(("softmax", "sigmoid")), "dtype": rng.choice(("f32", "bf16"))}
            # a selection bias goes with sigmoid scores
            c["bias"] = c["scoring"] == "sigmoid" and rng.random() < 0.7
            if c["t"] * e <= ROUTE_MAX_TE and c["t"] != 3072:
                return c
        else:
            e = _log_int(rng, 4, 64)
            c = {"op": op, "fmt": rng.choice(("fp4", "fp8")), "t": _log_int(rng, 1, 64), "e": e,
                 "topk": rng.randint(1, min(8, e)), "h": 128 * _log_int(rng, 4, 56), "i": 128 * _log_int(rng, 2, 16),
                 "c": rng.random() < 0.3, "masked": rng.choice((0.0, 0.0, 0.25))}
            bits = 1 if c["fmt"] == "fp4" else 2
            if c["e"] * c["h"] * c["i"] * bits <= MOE_MAX_EHI and 3072 not in (c["h"], c["i"], 2 * c["i"]):
                return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _exponent(amax, limit):
    """Biased exponent of the smallest power of two s with amax / s <= limit."""
    e = torch.ceil(torch.log2(amax.clamp_min(1e-20) / limit)).to(torch.int32)
    return (e + 127).clamp(1, 254)


def _pack(exps, mn):
    """[groups_k, mn] biased exponents -> packed words int32 [ceil(groups_k/4), align4(mn)]."""
    gk = exps.shape[0]
    w = torch.zeros((gk + 3) // 4 * 4, (mn + 3) // 4 * 4, dtype=torch.int32, device=DEV)
    w[:gk, :mn] = exps
    w = w.view(-1, 4, w.shape[1])
    return (w[:, 0] | (w[:, 1] << 8) | (w[:, 2] << 16) | (w[:, 3] << 24)).contiguous()


def _weights(g, n, k, fmt):
    """Gaussian weights of standard deviation 1/sqrt(k), quantised: (codes, packed scales)."""
    w = torch.randn(n, k, generator=g, device=DEV) * (k ** -0.5)
    if fmt == "fp4":
        v = w.view(n, k // 32, 32)
        e = _exponent(v.abs().amax(-1), 6.0)
        v = v * torch.exp2(127.0 - e)[..., None]
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        code = torch.bucketize(v.abs(), mids, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        code = code.view(n, k // 2, 2)
        return code[..., 0] | (code[..., 1] << 4), _pack(e.t(), n)
    nb = (n + 127) // 128
    v = torch.nn.functional.pad(w, (0, 0, 0, nb * 128 - n)).view(nb, 128, k // 128, 128)
    e = _exponent(v.abs().amax(dim=(1, 3)), 448.0)
    code = (v * torch.exp2(127.0 - e)[:, None, :, None]).view(nb * 128, k)[:n].to(torch.float8_e4m3fn)
    return code.contiguous(), _pack(e.t().repeat_interleave(128, 1)[:, :n], n)


def _experts(g, e, n, k, fmt):
    codes = torch.empty(e, n, k // 2 if fmt == "fp4" else k, device=DEV,
                        dtype=torch.uint8 if fmt == "fp4" else torch.float8_e4m3fn)
    groups = k // 32 if fmt == "fp4" else k // 128
    sf = torch.empty(e, (groups + 3) // 4, n, dtype=torch.int32, device=DEV)
    for j in range(e):
        codes[j], sf[j] = _weights(g, n, k, fmt)
    return codes, sf


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        s["b"], s["sfb"] = _weights(g, n, k, case["fmt"])
        # activations as a norm leaves them, a few channels much larger than the rest
        gain = torch.exp(0.7 * torch.randn(k, generator=g, device=DEV))
        s["a"] = (torch.randn(m, k, generator=g, device=DEV) * gain).to(torch.bfloat16)
        dt = torch.float32 if case["out"] == "f32" else torch.bfloat16
        s["cin"] = torch.randn(m, n, generator=g, device=DEV).to(dt) if case["c"] else None
        s["d"] = torch.empty(m, n, dtype=dt, device=DEV)
    elif case["op"] == "route":
        t, e = case["t"], case["e"]
        logits = torch.randn(t, e, generator=g, device=DEV) * 1.5
        s["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        s["b"] = torch.randn(e, generator=g, device=DEV) * 0.1 if case["bias"] else None
        s["ids"] = torch.empty(t, case["topk"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(t, case["topk"], dtype=torch.float32, device=DEV)
    else:
        t, e, h, i = case["t"], case["e"], case["h"], case["i"]
        s["w1"], s["sf1"] = _experts(g, e, 2 * i, h, case["fmt"])
        s["w2"], s["sf2"] = _experts(g, e, h, i, case["fmt"])
        s["x"] = torch.randn(t, h, generator=g, device=DEV).to(torch.bfloat16)
        score, ids = torch.softmax(torch.randn(t, e, generator=g, device=DEV), -1).topk(case["topk"], -1)
        gone = torch.rand(t, case["topk"], generator=g, device=DEV) < case["masked"]
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).to(torch.int32)
        s["weights"] = score / score.sum(-1, keepdim=True)
        s["cin"] = torch.randn(t, h, generator=g, device=DEV).to(torch.bfloat16) if case["c"] else None
        s["y"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _decode(codes, sf, n, k):
    """Codes [..., n, k or k/2] and packed scales [..., slices, align4(n)] -> FP32 weights [..., n, k]."""
    if codes.dtype == torch.uint8:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        pairs = torch.stack((table.repeat(16), table.repeat_interleave(16)), -1)        # by byte: (low, high) nibble
        w = pairs[codes.reshape(-1).to(torch.int32)].view(*codes.shape[:-1], k)
        gran = 32
    else:
        w = codes.to(torch.float32)
        gran = 128
    shifts = torch.tensor([0, 8, 16, 24], device=sf.device, dtype=torch.int32)
    e = (sf.unsqueeze(-2) >> shifts[:, None]) & 255                                      # [..., slices, 4, align4(n)]
    e = e.flatten(-3, -2)[..., :k // gran, :n].transpose(-1, -2)                         # [..., n, k/gran]
    return (w.unflatten(-1, (k // gran, gran)) * torch.exp2(e.to(torch.float32) - 127.0).unsqueeze(-1)).flatten(-2)


def _gemv_plain(s):
    d = s["a"].to(torch.float32) @ _decode(s["b"], s["sfb"], s["n"], s["k"]).t()
    if s["cin"] is not None:
        d = d + s["cin"].to(torch.float32)
    return d.to(s["d"].dtype)


def _route_plain(s):
    x = s["logits"].to(torch.float32)
    if s["scoring"] == "softmax":
        score = torch.exp(x - x.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
        key = x                                     # the scores' order
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
        key = score if s["b"] is None else score + s["b"]
    ids = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :s["topk"]]
    w = score.gather(-1, ids)
    return {"ids": ids.to(torch.int32), "weights": w / w.sum(-1, keepdim=True)}


def _moe_plain(s):
    t, h, i = s["t"], s["h"], s["i"]
    used = torch.unique(s["ids"])
    used = used[used >= 0].long()
    share = ((s["ids"].long()[:, :, None] == used) * s["weights"][:, :, None]).sum(1)     # [t, used]
    x = s["x"].to(torch.float32)
    gate_up = x @ _decode(s["w1"][used], s["sf1"][used], 2 * i, h).transpose(1, 2)        # [used, t, 2i]
    gate, up = gate_up[..., :i], gate_up[..., i:]
    act = gate / (1.0 + torch.exp(-gate)) * up * share.t()[..., None]
    y = (act @ _decode(s["w2"][used], s["sf2"][used], h, i).transpose(1, 2)).sum(0)
    if s["cin"] is not None:
        y = y + s["cin"].to(torch.float32)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        return {"gemv": _gemv_plain, "route": _route_plain, "moe": _moe_plain}[s["op"]](s)
    from block_scaled_fp8_gb300 import binding as dg
    if s["op"] == "gemv":
        if s["out"] == "f32":
            fn = dg.dg_bf16_fp4_gemv_nt_f32 if s["fmt"] == "fp4" else dg.dg_bf16_fp8_gemv_nt_f32
        else:
            fn = dg.dg_bf16_fp4_gemv_nt if s["fmt"] == "fp4" else dg.dg_bf16_fp8_gemv_nt
        return fn(s["a"], s["b"], s["sfb"], s["d"], c=s["cin"])
    if s["op"] == "route":
        dg.dg_moe_route(s["logits"], s["ids"], s["weights"], bias=s["b"], scoring=s["scoring"], renormalize=True)
        return {"ids": s["ids"], "weights": s["weights"]}
    fn = dg.dg_moe_fp4_layer if s["fmt"] == "fp4" else dg.dg_moe_fp8_layer
    return fn(s["x"], s["ids"], s["weights"], s["w1"], s["sf1"], s["w2"], s["sf2"], s["y"], c=s["cin"])


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["out"] == "f32" else 2
        per = 0.5 + 1 / 32 if case["fmt"] == "fp4" else 1 + 1 / 128
        return {"bytes": n * k * per + 2 * m * k + m * n * out * (2 if case["c"] else 1), "flops": 2 * m * n * k}
    if case["op"] == "route":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["t"] * (case["e"] * size + case["topk"] * 8) + 4 * case["e"] * case["bias"],
                "flops": 5 * case["t"] * case["e"]}
    t, e, h, i = case["t"], case["e"], case["h"], case["i"]
    used = e * (1 - (1 - case["topk"] * (1 - case["masked"]) / e) ** t)                    # expected distinct experts
    per = 0.5 + 1 / 32 if case["fmt"] == "fp4" else 1 + 1 / 128
    return {"bytes": used * 3 * h * i * per + t * (case["topk"] * 8 + h * (6 if case["c"] else 4)),
            "flops": 6 * t * case["topk"] * (1 - case["masked"]) * h * i}


# ------------------------------------------------------------------ the definition in 64 bits

def _w64(codes, sf, rows, k):
    """One weight matrix in 64 bits, element by element of its definition."""
    if codes.dtype == torch.uint8:
        c = torch.empty(rows, k, dtype=torch.int32, device=codes.device)
        c[:, 0::2] = codes & 15
        c[:, 1::2] = codes >> 4
        exp, man = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(exp == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, exp - 1))
        val, gran = torch.where(c >= 8, -mag, mag), 32
    else:
        val, gran = codes.double(), 128
    j = torch.arange(k, device=codes.device) // gran
    words = sf[j // 4][:, :rows].t()
    exps = (words >> (8 * (j % 4)).to(torch.int32)) & 255
    return torch.ldexp(val, exps - 127)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemv":
        n, k = case["n"], case["k"]
        a, out = s["a"].double(), []
        for r in range(0, n, 16384):
            q = min(n, r + 16384)
            out.append(a @ _w64(s["b"][r:q], s["sfb"][:, r:q], q - r, k).t())
        d = torch.cat(out, 1)
        return d if s["cin"] is None else d + s["cin"].double()
    if case["op"] == "route":
        x = s["logits"].double()
        score = torch.softmax(x, -1) if case["scoring"] == "softmax" else torch.sigmoid(x)
        key = score if s["b"] is None else score + s["b"].double()
        order = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :case["topk"]]
        w = torch.gather(score, 1, order)
        return {"ids": None, "weights": w / w.sum(1, keepdim=True)}
    h, i = case["h"], case["i"]
    y = torch.zeros(case["t"], h, dtype=torch.float64, device=DEV)
    if s["cin"] is not None:
        y += s["cin"].double()
    for e in range(case["e"]):
        who, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if who.numel():
            gu = s["x"][who].double() @ _w64(s["w1"][e], s["sf1"][e], 2 * i, h).t()
            act = torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]
            y.index_add_(0, who, (act @ _w64(s["w2"][e], s["sf2"][e], h, i).t()) * s["weights"][who, slot, None].double())
    return y
