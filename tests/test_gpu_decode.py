"""The decode-side operators against plain 64-bit forms: few-row products with FP4 and
FP8 weights, top-k routing, the MoE layer for few tokens."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding
from tests import _decode as D

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

GEMV = {("fp4", False): binding.dg_bf16_fp4_gemv_nt, ("fp4", True): binding.dg_bf16_fp4_gemv_nt_f32,
        ("fp8", False): binding.dg_bf16_fp8_gemv_nt, ("fp8", True): binding.dg_bf16_fp8_gemv_nt_f32}


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _check(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: off by {float((got - ref).abs().max())}, {int((over > 0).sum())} over the bound"


def _gemv(fmt, a, codes, sf, f32=False, c=None, d=None, pad=0, **kw):
    m, n = a.shape[0], codes.shape[0]
    if d is None:
        d = D.padded(torch.full((m, n), 7.0, dtype=torch.float32 if f32 else torch.bfloat16), pad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    GEMV[fmt, f32](a, codes, sf, d, c=c, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return d


SHAPES = [(1, 8, 128), (1, 24, 384), (2, 128, 256), (3, 264, 896), (7, 136, 128), (8, 512, 1024), (9, 120, 640),
          (16, 1000, 512), (17, 2112, 1408), (31, 248, 384), (33, 256, 2048), (64, 776, 1152), (64, 128, 7168),
          (1, 7168, 2048), (5, 2112, 7168), (1, 40000, 128), (12, 33000, 256)]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemv_matches_the_64_bit_product(fmt, m, n, k):
    g = _gen(m * 131 + n + k)
    pad = 32 if (m + n // 8) % 2 else 0
    with_c = (n // 8) % 3 == 0
    a = (torch.randn(m, k, generator=g) * torch.exp(torch.randn(k, generator=g))).bfloat16()
    codes, s, gran = D.quantize(torch.randn(n, k, generator=g), fmt)
    w = D.dequantize(codes, s, gran)
    sf = D.pack_scales(s)
    ref, tol = a.double() @ w.t(), D.product_bound(a.double(), w)
    ad, bd = D.padded(a, pad), D.padded(codes.view(torch.uint8), pad).view(codes.dtype)
    for f32 in (False, True):
        dt = torch.float32 if f32 else torch.bfloat16
        c = torch.randn(m, n, generator=g).to(dt) if with_c else None
        full = ref if c is None else ref + c.double()
        d = _gemv(fmt, ad, bd, sf, f32, None if c is None else D.padded(c, pad), pad=pad)
        # one rounding of the sum to bf16 (or of the FP32 sum with C)
        _check(d, full, tol + full.abs() * (2.0 ** -22 if f32 else 2.0 ** -8), f"{fmt} {m}x{n}x{k} f32={f32}")


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_gemv_small_integers_are_exact(fmt):
    """Integers whose every partial sum fits 23 bits: the FP32 result is the integer."""
    m, n, k = 6, 392, 1024
    g = _gen(5)
    a = torch.randint(-255, 256, (m, k), generator=g).bfloat16()
    w = torch.tensor([0.0, 1.0, 2.0, 3.0, -1.0, -2.0, -3.0, 4.0])[torch.randint(0, 8, (n, k), generator=g)]
    if fmt == "fp4":
        mags = D.MAGS.float()
        code = (w.abs()[..., None] == mags).float().argmax(-1).to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)
        codes, groups = code[:, 0::2] | (code[:, 1::2] << 4), k // 32
    else:
        codes, groups = w.to(torch.float8_e4m3fn), k // 128
    sf = D.pack_scales(torch.ones(n, groups))
    d = _gemv(fmt, a.cuda(), codes.cuda(), sf, True)
    assert torch.equal(d.cpu().double(), a.double() @ w.double().t())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_gemv_rows_do_not_depend_on_the_batch(fmt):
    n, k = 1032, 1664
    g = _gen(9)
    a = torch.randn(64, k, generator=g).bfloat16().cuda()
    codes, s, _ = D.quantize(torch.randn(n, k, generator=g), fmt)
    codes, sf = codes.cuda(), D.pack_scales(s)
    full = _gemv(fmt, a, codes, sf, True)
    few = full
    if fmt == "fp4":                                # up to 8 rows: other pieces
        few = torch.cat([_gemv(fmt, a[i:i + 8], codes, sf, True) for i in range(0, 64, 8)])
    for m in (1, 2, 3, 7, 8, 9, 16, 17, 32, 33, 63):
        want = few if m <= 8 else full
        assert torch.equal(_gemv(fmt, a[:m], codes, sf, True), want[:m]), m
        assert torch.equal(_gemv(fmt, a[64 - m:], codes, sf, True), want[64 - m:]), m


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("few", [False, True])
def test_gemv_extreme_values(fmt, few):
    """Zero rows, groups of very different magnitude, the ends of the scale range, and
    non-finite rows, which stay alone."""
    m, n, k = 10, 256, 512
    g = _gen(11)
    a = torch.randn(m, k, generator=g)
    a[1] = 0.0
    a[2] *= 1e30
    a[3] *= 1e-30
    a[4, 32:] *= 1e-4
    a[5, ::2] = 0.0
    a[6, 7] = 3e4          # one large channel in its group
    a[7] = 2.0 ** -133       # the smallest bf16
    a = a.bfloat16()
    run = (lambda x: torch.cat([_gemv(fmt, x[:5].cuda(), codes.cuda(), sf, True),      # 5 rows at a time
                                _gemv(fmt, x[5:].cuda(), codes.cuda(), sf, True)]).cpu().double()) if few else \
        (lambda x: _gemv(fmt, x.cuda(), codes.cuda(), sf, True).cpu().double())
    codes, s, gran = D.quantize(torch.randn(n, k, generator=g), fmt)
    s[::4] *= 2.0 ** -100
    s[1::4] *= 2.0 ** 90
    w = D.dequantize(codes, s, gran)
    # rows whose results leave the FP32 range are kept out of the comparison
    ref, tol = a.double() @ w.t(), D.product_bound(a.double(), w)
    sane = (ref.abs() < 1e37) & (a.double().abs() @ w.abs().t() < 1e38)
    if few and fmt == "fp4":
        tol = tol + 2.0 ** -128 * w.abs().sum(1)      # the digits' absolute bound, an element
    sf = D.pack_scales(s)
    d = run(a)
    # sums below the normal range may lose their last bits
    over = (d - ref).abs() - tol - 2.0 ** -22 * ref.abs() - 2.0 ** -126
    assert (over[sane] <= 0).all()
    assert (d[1] == 0).all()
    bad = a.clone()
    bad[0, 3] = float("nan")
    bad[8, 100] = float("inf")
    bad[9, 511] = float("-inf")
    e = run(bad)
    assert torch.isnan(e[[0, 8, 9]]).all()
    assert torch.allclose(e[1:8], d[1:8], rtol=0.0, atol=0.0, equal_nan=True)   # row 2 overflows in places


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_gemv_in_place_stream_and_graph(fmt):
    m, n, k = 4, 520, 768
    g = _gen(13)
    a = torch.randn(m, k, generator=g).bfloat16().cuda()
    codes, s, _ = D.quantize(torch.randn(n, k, generator=g), fmt)
    codes, sf = codes.cuda(), D.pack_scales(s)
    c = torch.randn(m, n, generator=g).bfloat16().cuda()
    want = _gemv(fmt, a, codes, sf, c=c)
    d = c.clone()
    _gemv(fmt, a, codes, sf, c=d, d=d)              # accumulated in place
    assert torch.equal(d, want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    e = torch.zeros_like(c)
    GEMV[fmt, False](a, codes, sf, e, c=c, stream=other)
    other.synchronize()
    assert torch.equal(e, want)
    graph = torch.cuda.CUDAGraph()
    f = torch.zeros_like(c)
    with torch.cuda.graph(graph):
        GEMV[fmt, False](a, codes, sf, f, c=c)
        GEMV[fmt, False](a, codes, sf, f, c=f)      # reads what the first wrote
    graph.replay()
    torch.cuda.synchronize()
    twice = _gemv(fmt, a, codes, sf, c=want)
    assert torch.equal(f, twice)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_gemv_empty(fmt):
    codes = torch.zeros(64, 64 if fmt == "fp4" else 128, dtype=torch.uint8, device="cuda")
    codes = codes if fmt == "fp4" else codes.view(torch.float8_e4m3fn)
    sf = torch.zeros(1, 64, dtype=torch.int32, device="cuda")
    d = torch.full((0, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    GEMV[fmt, False](torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"), codes, sf, d)
    for f32, dt in ((False, torch.bfloat16), (True, torch.float32)):
        d = torch.full((3, 64), 7.0, dtype=dt, device="cuda")
        a = torch.zeros(3, 0, dtype=torch.bfloat16, device="cuda")
        GEMV[fmt, f32](a, codes[:, :0], sf, d)
        assert (d == 0).all()
        c = torch.full((3, 64), 2.0, dtype=dt, device="cuda")
        GEMV[fmt, f32](a, codes[:, :0], sf, d, c=c)
        assert torch.equal(d, c)


# ------------------------------------------------------------------ routing

def _route(logits, topk, **kw):
    t = logits.shape[0]
    ids = torch.full((t, topk), 99, dtype=torch.int32, device="cuda")
    w = torch.full((t, topk), 99.0, device="cuda")
    binding.dg_moe_route(logits, ids, w, **kw)
    torch.cuda.synchronize()
    return ids.cpu(), w.cpu()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,topk,dtype,bias,renorm,scale", [
    (1, 1, 1, torch.float32, False, True, 1.0), (3, 5, 5, torch.float32, True, False, 2.5),
    (1, 256, 8, torch.float32, True, True, 2.5), (257, 33, 4, torch.bfloat16, False, True, 1.0),
    (100, 64, 6, torch.bfloat16, True, False, 1.0), (65, 160, 7, torch.float32, False, False, 1.0),
    (31, 512, 10, torch.float32, True, True, 1.0), (9, 1000, 32, torch.bfloat16, True, True, 0.5),
    (2000, 128, 6, torch.float32, False, True, 1.0), (8, 384, 1, torch.float32, True, True, 1.0)])
def test_route_matches_the_64_bit_choice(scoring, t, e, topk, dtype, bias, renorm, scale):
    g = _gen(t + e * 7 + topk)
    logits = (torch.randn(t, e, generator=g) * 2).to(dtype)
    b = torch.randn(e, generator=g) * 0.2 if bias else None
    wide = D.padded(logits, 3)
    ids, w = _route(wide, topk, bias=None if b is None else b.cuda(), scoring=scoring, renormalize=renorm, scale=scale)
    want, weights, clear = D.route_plain(logits, b, topk, scoring, renorm, scale)
    assert clear.float().mean() > 0.98 - 2 / t
    assert torch.equal(ids[clear], want[clear])
    # exp, a sum of up to 1000 positive terms (32 at a time) and two divisions, 2^-24 each
    assert ((w.double() - weights)[clear].abs() <= weights[clear].abs() * 2.0 ** -18 + 1e-37).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_masks_ties_and_special_values(scoring):
    inf, low = float("inf"), torch.finfo(torch.float32).min
    logits = torch.zeros(8, 40)
    logits[1] = -inf                                     # nothing left
    logits[2] = -inf
    logits[2, 30] = 1.0                                  # fewer experts than slots
    logits[2, 7] = 2.0
    logits[3] = low                                      # masked with the lowest value
    logits[3, 39] = 0.0
    logits[4, ::2] = float("nan")
    logits[5, 3:9] = 5.0                                 # a tie across the last slot
    logits[6] = torch.tensor([-0.0, 0.0] * 20)            # one key
    logits[7] = low                                      # the lowest value everywhere
    ids, w = _route(logits.cuda(), 4, scoring=scoring)
    assert ids[0].tolist() == [0, 1, 2, 3]
    assert ids[1].tolist() == [-1] * 4 and (w[1] == 0).all()
    assert ids[2].tolist() == [7, 30, -1, -1] and (w[2, 2:] == 0).all()
    assert abs(float(w[2].sum()) - 1) < 1e-6
    assert ids[3].tolist() == [39, 0, 1, 2] and w[3].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert ids[4].tolist() == [1, 3, 5, 7] and abs(float(w[4, 0]) - 0.25) < 1e-6
    assert ids[5].tolist() == [3, 4, 5, 6]
    assert ids[6].tolist() == [0, 1, 2, 3]
    assert ids[7].tolist() == [0, 1, 2, 3] and torch.isfinite(w[7]).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [40, 64, 127, 256, 500])
def test_route_many_candidates(scoring, dtype, e):
    """Logits of a few values only: far more ties than lanes, on either side of the last slot;
    saturated scores; biases of +-infinity and NaN; unaligned rows."""
    topk = min(e, 9)
    logits = torch.randint(-2, 3, (50, e), generator=_gen(e)).to(dtype)
    logits[1] = 100.0                          # every sigmoid 1
    logits[2] = -200.0                         # every sigmoid 0
    logits[3, :5] = float("nan")
    bias = torch.zeros(e)
    bias[7], bias[8], bias[9] = float("inf"), float("-inf"), float("nan")
    for b in (None, bias):
        for shift in (0, 1):
            wide = torch.zeros(50, e + 8, dtype=dtype, device="cuda")
            wide[:, shift:shift + e] = logits.cuda()
            ids, w = _route(wide[:, shift:shift + e], topk, bias=None if b is None else b.cuda(), scoring=scoring)
            # 64-bit keys are as distinct as 32-bit ones here: the logits are small integers
            x = torch.where(torch.isnan(logits.double()), float("-inf"), logits.double())
            s = torch.softmax(x, -1) if scoring == "softmax" else torch.sigmoid(logits.float()).double()
            key = s if b is None else s + torch.nan_to_num(b.double(), nan=float("-inf"), posinf=float("inf"),
                                                           neginf=float("-inf"))
            key = torch.where(x > float("-inf"), key, float("-inf"))
            want = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :topk].int()
            assert torch.equal(ids, want)
            picked = s.gather(1, want.long())
            picked = picked / picked.sum(1, keepdim=True).clamp_min(2.0 ** -126)
            assert ((w.double() - picked).abs() <= 1e-6).all()


# ------------------------------------------------------------------ the MoE layer

LAYER = {"fp4": binding.dg_moe_fp4_layer, "fp8": binding.dg_moe_fp8_layer}


def _experts(g, e, n, k, fmt):
    q = [D.quantize(torch.randn(n, k, generator=g) * k ** -0.5, fmt) for _ in range(e)]
    codes = torch.stack([c.view(torch.uint8) for c, _, _ in q]).view(q[0][0].dtype)
    sf = D.pack_scales(torch.stack([s for _, s, _ in q]))
    w = torch.stack([D.dequantize(c, s, gran) for c, s, gran in q])
    return codes.cuda(), sf, w


def _layer_case(fmt, t, e, topk, h, i, seed=0):
    g = _gen(seed + t + e * 10 + h + i)
    w1, sf1, d1 = _experts(g, e, 2 * i, h, fmt)
    w2, sf2, d2 = _experts(g, e, h, i, fmt)
    x = torch.randn(t, h, generator=g).bfloat16()
    ids = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(t)]).int()
    weights = torch.rand(t, topk, generator=g) + 0.1
    return dict(x=x, ids=ids, weights=weights, w1=w1, sf1=sf1, w2=w2, sf2=sf2, d1=d1, d2=d2, fmt=fmt)


def _layer(s, status_is=0, y=None, **kw):
    t, h = s["x"].shape
    y = torch.full((t, h), 7.0, dtype=torch.bfloat16, device="cuda") if y is None else y
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    LAYER[s["fmt"]](kw.pop("x", s["x"].cuda()), s["ids"].cuda(), s["weights"].cuda(), s["w1"], s["sf1"], s["w2"],
                    s["sf2"], y, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == status_is
    return y


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("t,e,topk,h,i", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (2, 4, 4, 640, 128), (3, 16, 6, 384, 256), (7, 5, 3, 896, 640),
    (8, 32, 8, 512, 256), (9, 3, 2, 256, 512), (16, 64, 4, 256, 128), (17, 6, 6, 384, 384), (32, 4, 1, 512, 128),
    (33, 12, 5, 256, 256), (64, 8, 2, 640, 384), (64, 4, 4, 256, 1408), (1, 8, 8, 7168, 128), (4, 3, 2, 128, 2048)])
def test_layer_matches_the_64_bit_form(fmt, t, e, topk, h, i):
    s = _layer_case(fmt, t, e, topk, h, i)
    if t % 3 == 0:
        s["ids"][0] = -1                      # a token with no expert
        s["ids"][t // 2, 0] = -7
        s["weights"][s["ids"] < 0] = float("nan")
    with_c = t % 2 == 0
    c = torch.randn(t, h, generator=_gen(1)).bfloat16() if with_c else None
    y = _layer(s, c=None if c is None else D.padded(c, 8), x=D.padded(s["x"], 16))
    ref, tol = D.layer_plain(s["x"], s["ids"], s["weights"], s["d1"], s["d2"], c)
    _check(y, ref, tol, f"{fmt} t{t} e{e} k{topk} {h}x{i}")
    again = _layer(s, c=None if c is None else c.cuda())
    assert torch.equal(y, again)              # nothing depends on the order of events
    if t % 3 == 0:
        assert torch.equal(y[0].cpu(), torch.zeros(h).bfloat16() if c is None else c[0])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_layer_slots(fmt):
    """An expert named twice, ids out of range, all slots empty, C in place, a larger workspace."""
    s = _layer_case(fmt, 5, 6, 3, 256, 256)
    s["ids"][0] = torch.tensor([2, 2, 4])
    s["ids"][1] = torch.tensor([5, 6, 1000])
    s["ids"][2] = -1
    s["ids"][4] = torch.tensor([3, 3, 3])
    c = torch.randn(5, 256, generator=_gen(2)).bfloat16()
    ref, tol = D.layer_plain(s["x"], s["ids"], s["weights"], s["d1"], s["d2"], c)
    y = c.cuda()
    ws = torch.full((binding.moe_layer_workspace_bytes(5, 3, 256, 256, 6) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    _layer(s, status_is=binding.DG_DEV_BAD_GROUP, y=y, c=y, workspace=ws)
    _check(y, ref, tol, fmt)
    s["ids"][:] = -1
    assert torch.equal(_layer(s, c=c.cuda()).cpu(), c)
    assert (_layer(s) == 0).all()


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_layer_non_finite_token_stays_alone(fmt):
    s = _layer_case(fmt, 12, 4, 2, 384, 256)
    clean = _layer(s)
    s["x"][3, 5] = float("inf")
    s["x"][10, 383] = float("nan")
    y = _layer(s)
    rest = [r for r in range(12) if r not in (3, 10)]
    assert torch.isnan(y[[3, 10]].float()).all()
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_layer_other_stream_graph_and_chain(fmt):
    """On a stream of its own, in a graph, and as route -> layer -> product without a
    synchronisation between them."""
    s = _layer_case(fmt, 6, 16, 4, 512, 256)
    want = _layer(s)
    x, ids, wt = s["x"].cuda(), s["ids"].cuda(), s["weights"].cuda()
    args = (s["w1"], s["sf1"], s["w2"], s["sf2"])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    LAYER[fmt](x, ids, wt, *args, y, stream=other)
    other.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(binding.moe_layer_workspace_bytes(6, 4, 512, 256, 16), dtype=torch.uint8, device="cuda")
    g1, g2 = torch.zeros_like(want), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        LAYER[fmt](x, ids, wt, *args, g1, workspace=ws)
        LAYER[fmt](x, ids, wt, *args, g2, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g1, want) and torch.equal(g2, want)
    logits = torch.randn(6, 16, generator=_gen(3)).cuda()
    codes, sc, _ = D.quantize(torch.randn(264, 512, generator=_gen(4)), fmt)
    codes, sf = codes.cuda(), D.pack_scales(sc)

    def step(sync):
        i2 = torch.empty(6, 4, dtype=torch.int32, device="cuda")
        w2 = torch.empty(6, 4, device="cuda")
        y2 = torch.empty_like(want)
        d2 = torch.empty(6, 264, device="cuda")
        binding.dg_moe_route(logits, i2, w2, scoring="sigmoid")
        if sync:
            torch.cuda.synchronize()
        LAYER[fmt](x, i2, w2, *args, y2, c=x)
        if sync:
            torch.cuda.synchronize()
        GEMV[fmt, True](y2, codes, sf, d2)
        torch.cuda.synchronize()
        return i2, w2, y2, d2
    slow = step(True)
    for _ in range(20):
        for p, q in zip(step(False), slow):
            assert torch.equal(p, q)


def test_layer_empty():
    s = _layer_case("fp4", 2, 2, 1, 128, 128)
    y = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    binding.dg_moe_fp4_layer(s["x"][:0].cuda(), s["ids"][:0].cuda(), s["weights"][:0].cuda(), s["w1"], s["sf1"],
                             s["w2"], s["sf2"], y)
