"""The decode-side operators where the launch rules change form: rounds of persistent CTAs,
uneven routing in short segments, the largest tables, results beside and in the ring."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding
from tests import _decode as D
from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("m,n,k", [
    (4, 40000, 256), (12, 40000, 384), (40, 40000, 256),   # 313 tiles: 9 after whole rounds of two CTAs on each SM
    (4, 65536, 128), (20, 65536, 128), (64, 65536, 128),   # 512 tiles
    (3, 3584, 2560), (8, 3584, 2560), (24, 3584, 2560), (40, 3584, 2560),   # split: results beside, in the ring
    (6, 9216, 1152),                                       # clusters that fill the GPU
])
def test_gemv_forms(fmt, m, n, k):
    g = T._gen(m + n + k)
    a = torch.randn(m, k, generator=g).bfloat16()
    codes, s, gran = D.quantize(torch.randn(n, k, generator=g), fmt)
    w = D.dequantize(codes, s, gran)
    sf = D.pack_scales(s)
    ref, tol = a.double() @ w.t(), D.product_bound(a.double(), w)
    T._check(T._gemv(fmt, a.cuda(), codes.cuda(), sf, True), ref, tol + ref.abs() * 2.0 ** -23, f"{fmt} {m}x{n}x{k} f32")
    c = torch.randn(m, n, generator=g).bfloat16()
    d = T._gemv(fmt, a.cuda(), codes.cuda(), sf, c=c.cuda())
    full = ref + c.double()
    T._check(d, full, tol + full.abs() * 2.0 ** -8, f"{fmt} {m}x{n}x{k} bf16 + c")


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("t,e,topk", [(64, 64, 2), (40, 32, 8), (8, 16, 2), (5, 64, 6)])
def test_layer_uneven_routing(fmt, t, e, topk):
    """All tokens name the same experts, more of them than a segment has room for; one expert
    has a single token."""
    s = T._layer_case(fmt, t, e, topk, 256, 128, seed=7)
    s["ids"][:] = torch.arange(topk).int() * (e // topk)
    s["ids"][t // 3, 0] = e - 1
    y = T._layer(s)
    ref, tol = D.layer_plain(s["x"], s["ids"], s["weights"], s["d1"], s["d2"], None)
    T._check(y, ref, tol, f"{fmt} t{t} e{e} k{topk}")
    assert torch.equal(y, T._layer(s))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("t,topk", [(64, 16), (8, 16), (1, 1)])
def test_layer_most_experts(fmt, t, topk):
    """1024 experts: the largest tables.  The experts' weights are copies of a few."""
    few, e, h, i = 5, 1024, 128, 128
    s = T._layer_case(fmt, t, few, 1, h, i, seed=3)
    pick = torch.arange(e) % few
    for name in ("w1", "w2"):
        w = s[name].view(torch.uint8)
        s[name] = w[pick.cuda()].contiguous().view(s[name].dtype)
    for name in ("sf1", "sf2"):
        s[name] = s[name][pick.cuda()].contiguous()
    g = T._gen(t)
    s["ids"] = torch.stack([torch.randperm(e, generator=g)[:topk] for _ in range(t)]).int()
    s["ids"][0, 0] = e - 1
    s["weights"] = torch.rand(t, topk, generator=g) + 0.1
    y = T._layer(s)
    ref, tol = D.layer_plain(s["x"], s["ids"], s["weights"], s["d1"][pick], s["d2"][pick], None)
    T._check(y, ref, tol, f"{fmt} t{t} k{topk}")


@pytest.mark.parametrize("spread", [0.0, 1.5, 12.0])
@pytest.mark.parametrize("topk", [1, 8, 20, 32])
@pytest.mark.parametrize("bias", [0.0, 0.1, 1000.0])
def test_route_sigmoid_near_one(spread, topk, bias):
    """Sigmoid scores that crowd near 1, equal ones among them, with small and large biases:
    the keys are recomputed in FP32 as the contract states them, the order is theirs."""
    t, e = 37, 256
    g = T._gen(topk)
    logits = torch.randn(t, e, generator=g) * spread + 9.0
    b = torch.randn(e, generator=g) * bias if bias else None
    ids = torch.empty(t, topk, dtype=torch.int32, device="cuda")
    w = torch.empty(t, topk, device="cuda")
    binding.dg_moe_route(logits.cuda(), ids, w, bias=None if b is None else b.cuda(), scoring="sigmoid",
                         renormalize=False)
    torch.cuda.synchronize()
    got = ids.cpu().long()
    score = torch.sigmoid(logits.double())
    key = score if b is None else score + b.double()
    # an FP32 score is within 4 units of 2^-24 below 1, a key within one more rounding of its size
    slack = 2.0 ** -21 + key.abs().amax(-1, keepdim=True) * 2.0 ** -23
    assert all(len(set(r.tolist())) == topk for r in got)
    chosen = key.gather(1, got)
    best = key.topk(topk, -1)[0]
    assert ((chosen - best).abs() <= slack).all()
    assert ((w.cpu().double() - score.gather(1, got)).abs() <= 2.0 ** -21).all()
