"""The FP8 quantiser against its definition: codes and scale words have to be equal bit for bit.

Every step of the definition is exact but the one rounding to E4M3 (the scale is a power of two),
so nothing here has a tolerance.  The comparison's own rounding is torch's CPU cast."""
import pytest
import torch

from tests._ffn import cdiv, pack, scale64
from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
E4M3 = torch.float8_e4m3fn


def finite_amax(x, dim):
    x = x.double().abs()
    return torch.where(torch.isfinite(x), x, torch.zeros_like(x)).amax(dim)


def codes(x, s):
    """x / s to E4M3 (both FP64; the quotient is exact in FP32); infinities are NaN."""
    v = torch.where(torch.isinf(x), torch.full_like(x, float("nan")), x) / s
    q = v.float().to(E4M3).view(torch.uint8)
    return torch.where(v.isnan(), torch.full_like(q, 0x7F), q)   # (one NaN code, whatever the sign)


def exps(s):
    return (torch.frexp(s)[1] - 1 + 127).int()


def rows_form(x):
    r, c = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -c % 128)).view(r, -1, 128)
    s = scale64(finite_amax(v, -1))
    return codes(v, s[..., None]).reshape(r, -1)[:, :c], pack(exps(s).t(), r)


def cols_form(x, ks=None):
    r, c = x.shape
    q, words = torch.empty(r, c, dtype=torch.uint8), []
    first = 0
    for k in ([r] if ks is None else ks):
        v = torch.nn.functional.pad(x[first:first + k].double(), (0, 0, 0, -k % 128)).view(-1, 128, c)
        s = scale64(finite_amax(v, 1))
        q[first:first + k] = codes(v, s[:, None]).reshape(-1, c)[:k]
        words.append(pack(exps(s), c))
        first += k
    return q, torch.cat(words)


def blocks_form(x):
    r, c = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -c % 128, 0, -r % 128)).view(cdiv(r, 128), 128, -1, 128)
    s = scale64(finite_amax(finite_amax(v, 3), 1))
    q = codes(v, s[:, None, :, None]).reshape(cdiv(r, 128) * 128, -1)[:r, :c]
    e = exps(s)
    return q, pack(e.repeat_interleave(128, 0)[:r].t(), r), pack(e.repeat_interleave(128, 1)[:, :c], c)


def same(q, want):
    q = q.cpu().view(torch.uint8)
    q = torch.where(q == 0xFF, torch.full_like(q, 0x7F), q)
    return torch.equal(q, want)


def values(r, c, dtype, seed):
    """Values over many binades, with zeros, ties, whole groups of zeros, the largest and smallest
    FP32 and bf16 magnitudes, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, c, generator=g) * torch.exp2(torch.randint(-12, 12, (r, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-6, 6, (1, c), generator=g).float())
    x[torch.rand(r, c, generator=g) < 0.1] = 0
    x[torch.rand(r, c, generator=g) < 0.02] = 448.0
    flat = x.view(-1)
    n = flat.numel()
    if n > 600:
        at = torch.randperm(n, generator=g)[:8]
        flat[at] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0e38, -3.0e38, 1e-45, 2.0 ** -126, 1.75])
    x[r // 2] = 0
    x[:, c // 3] = 0
    return x.to(dtype)


SIZES = [(1, 16), (3, 8), (96, 7168), (129, 144), (128, 128), (1000, 1037), (513, 520), (4097, 272), (5, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r,c", SIZES)
def test_rows_and_columns(r, c, dtype):
    step = 8 if dtype == torch.bfloat16 else 4
    buf = torch.zeros(r, cdiv(c, step) * step, dtype=dtype)   # rows start on 16 bytes
    x = buf[:, :c]
    x.copy_(values(r, c, dtype, r + c))
    dev = buf.cuda()[:, :c]
    ld = cdiv(c, 16) * 16

    def out():
        return torch.full((r, ld), 0x55, dtype=torch.uint8, device="cuda").view(E4M3)

    def words(a, b):
        return torch.full((cdiv(a, 512), cdiv(b, 4) * 4), -1, dtype=torch.int32, device="cuda")
    wq, wsf = rows_form(x)
    wqk, wsfk = cols_form(x)
    q, sf, qk, sfk = out(), words(c, r), out(), words(r, c)
    dg.dg_quantize_fp8(dev, q=q[:, :c], sf=sf)
    dg.dg_quantize_fp8(dev, qk=qk[:, :c], sfk=sfk)
    assert same(q[:, :c], wq) and torch.equal(sf.cpu(), wsf)
    assert same(qk[:, :c], wqk) and torch.equal(sfk.cpu(), wsfk)
    b, sb, bk, sbk = out(), words(c, r), out(), words(r, c)
    dg.dg_quantize_fp8(dev, q=b[:, :c], sf=sb, qk=bk[:, :c], sfk=sbk)
    for s, t in ((q, b), (sf, sb), (qk, bk), (sfk, sbk)):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    for t in (q, qk):
        assert bool((t.view(torch.uint8)[:, c:] == 0x55).all()), "nothing beside the rows"


@pytest.mark.parametrize("ks", [[128], [256, 640, 0, 128], [0, 0, 512], [128, 0, 1152]])
def test_k_grouped(ks):
    r, c = sum(ks), 204
    x = values(r, c, torch.bfloat16, r)
    ld = 208
    buf = torch.zeros(r, ld, dtype=torch.bfloat16)
    buf[:, :c] = x
    dev = buf.cuda()[:, :c]
    q = torch.empty(r, ld, dtype=E4M3, device="cuda")[:, :c]
    words = torch.full((dg.k_grouped_packed_sf_rows(ks), c), -1, dtype=torch.int32, device="cuda")
    dg.dg_quantize_fp8(dev, qk=q, sfk=words, ks=ks)
    wq, wsf = cols_form(x, ks)
    assert same(q, wq) and torch.equal(words.cpu(), wsf[:words.shape[0]])
    assert words.shape[0] == wsf.shape[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,r,c", [(1, 128, 128), (3, 200, 144), (2, 512, 1040), (1, 1, 8), (2, 1027, 24)])
def test_blocks(b, r, c, dtype):
    x = torch.stack([values(r, c, dtype, b + r + c + j) for j in range(b)])
    dev = x.cuda()
    ld = cdiv(c, 16) * 16
    q = torch.empty(b, r, ld, dtype=E4M3, device="cuda")[:, :, :c]
    sf = torch.full((b, cdiv(c, 512), cdiv(r, 4) * 4), -1, dtype=torch.int32, device="cuda")
    sft = torch.full((b, cdiv(r, 512), cdiv(c, 4) * 4), -1, dtype=torch.int32, device="cuda")
    dg.dg_quantize_fp8_blocks(dev, q, sf=sf, sft=sft)
    for j in range(b):
        wq, wsf, wsft = blocks_form(x[j])
        assert same(q[j], wq) and torch.equal(sf[j].cpu(), wsf) and torch.equal(sft[j].cpu(), wsft)
    q2 = torch.empty(b, r, ld, dtype=E4M3, device="cuda")[:, :, :c]
    one = torch.full_like(sft, -1)
    dg.dg_quantize_fp8_blocks(dev, q2, sft=one)
    assert torch.equal(one, sft) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


def test_many_rows():
    """More row tiles than a grid's second dimension holds (65535), and rows past 2^31 bytes in."""
    r, c = 65535 * 16 + 40, 1040
    x = torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 15, 16, 65535 * 16 - 1, 65535 * 16, r - 1], device="cuda")
    pick = torch.randn(len(rows), c, device="cuda").bfloat16()
    x[rows] = pick
    q = torch.empty(r, c, dtype=E4M3, device="cuda")
    sf = torch.empty(cdiv(c, 512), r, dtype=torch.int32, device="cuda")
    dg.dg_quantize_fp8(x, q=q, sf=sf)
    wq, wsf = rows_form(pick.cpu())
    assert same(q[rows], wq) and torch.equal(sf[:, rows].cpu(), wsf[:, :len(rows)])
    assert int((q.view(torch.uint8).view(torch.int64).view(r, -1) != 0).any(1).sum()) == len(rows)


def test_captured_and_on_another_stream():
    x = values(300, 640, torch.float32, 3).cuda()
    q, qk = torch.empty(300, 640, dtype=E4M3, device="cuda"), torch.empty(300, 640, dtype=E4M3, device="cuda")
    sf = torch.empty(2, 300, dtype=torch.int32, device="cuda")
    sfk = torch.empty(1, 640, dtype=torch.int32, device="cuda")
    wq, wsf = rows_form(x.cpu())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dg.dg_quantize_fp8(x, q=q, sf=sf, qk=qk, sfk=sfk, stream=side)
    side.synchronize()
    assert same(q, wq) and torch.equal(sf.cpu(), wsf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_quantize_fp8(x, q=q, sf=sf, qk=qk, sfk=sfk)
    x.copy_(values(300, 640, torch.float32, 4))
    graph.replay()
    wq, wsf = rows_form(x.cpu())
    wqk, wsfk = cols_form(x.cpu())
    assert same(q, wq) and torch.equal(sf.cpu(), wsf) and same(qk, wqk) and torch.equal(sfk.cpu(), wsfk)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nothing_finite(dtype):
    """Groups without a finite value, and NaN in all values of one place beside an infinity in another."""
    nan, inf = float("nan"), float("inf")
    x = torch.randn(256, 512, generator=torch.Generator().manual_seed(5))
    x[:128, :128] = nan
    x[3, 128:256] = inf
    x[:128, 130] = -inf
    x[128:, 0:512:2] = nan
    x[200, 1] = inf
    x = x.to(dtype)
    q, qk = (torch.empty(256, 512, dtype=E4M3, device="cuda") for _ in range(2))
    sf, sfk = torch.empty(1, 256, dtype=torch.int32, device="cuda"), torch.empty(1, 512, dtype=torch.int32, device="cuda")
    dg.dg_quantize_fp8(x.cuda(), q=q, sf=sf, qk=qk, sfk=sfk)
    (wq, wsf), (wqk, wsfk) = rows_form(x), cols_form(x)
    assert same(q, wq) and torch.equal(sf.cpu(), wsf) and same(qk, wqk) and torch.equal(sfk.cpu(), wsfk)
    sft = torch.empty_like(sfk)
    dg.dg_quantize_fp8_blocks(x.cuda(), q, sf=sf, sft=sft)
    wq, wsf, wsft = blocks_form(x)
    assert same(q, wq) and torch.equal(sf.cpu(), wsf) and torch.equal(sft.cpu(), wsft)
