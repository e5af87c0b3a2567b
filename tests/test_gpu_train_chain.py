"""One training step of a layer's experts, every operator in its place: values quantised, the gated
block and the down product, the backward pass, input and weight gradients, the orthogonalised
update, and the new weights quantised.

The gradients are compared with autograd's of the same step in 64 bits without quantisation.  Every
operand in 8 bits carries a relative error of at most 2^-4, 2^-4 / sqrt(3) in the mean square if
it is evenly spread; the gradient of W1 passes six of them (x forward and as an operand, W1,
W2, dy, dgu), whose errors are independent: sqrt(6) 2^-4 / sqrt(3) = 0.089 of its norm."""
import pytest
import torch

from tests._ffn import cdiv
from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
E, I, K = 4, 272, 384
COUNTS = [130, 0, 256, 77]                       # rows of each expert, padded with zeros to whole blocks
KS = [cdiv(c, 128) * 128 for c in COUNTS]
M = sum(KS)
LR = 0.02


def words(*s):
    return torch.empty(*s, dtype=torch.int32, device="cuda")


def codes(*s):
    return torch.empty(*s, dtype=E4M3, device="cuda")


class Step:
    """The buffers of a step and the step itself."""

    def __init__(self):
        g = torch.Generator().manual_seed(3)
        live = torch.cat([torch.arange(k) < c for c, k in zip(COUNTS, KS)])[:, None]
        self.x = (torch.randn(M, K, generator=g) * live).cuda()
        self.dy = (1e-3 * torch.randn(M, K, generator=g) * live).to(BF16).cuda()
        self.w1 = (torch.randn(E, 2 * I, K, generator=g) * K ** -0.5).cuda()
        self.w2 = (torch.randn(E, K, I, generator=g) * I ** -0.5).cuda()
        self.layout = torch.repeat_interleave(torch.arange(E), torch.tensor(KS)).to(torch.int32).cuda()
        self.ks_dev = torch.tensor(KS, dtype=torch.int32, device="cuda")
        rows = dg.k_grouped_packed_sf_rows(KS)
        self.xq, self.sfx, self.xk, self.sfxk = codes(M, K), words(cdiv(K, 512), M), codes(M, K), words(rows, K)
        self.yq, self.sfy, self.yk, self.sfyk = codes(M, K), words(cdiv(K, 512), M), codes(M, K), words(rows, K)
        self.gq, self.sfg, self.gk, self.sfgk = codes(M, 2 * I), words(cdiv(2 * I, 512), M), codes(M, 2 * I), words(rows, 2 * I)
        self.hk, self.sfhk = codes(M, I), words(rows, I)
        self.hq, self.sfh = codes(M, I), words(cdiv(I, 512), M)
        self.w1q, self.sf1, self.sf1t = codes(E, 2 * I, K), words(E, cdiv(K, 512), 2 * I), words(E, cdiv(2 * I, 512), K)
        self.w2q, self.sf2, self.sf2t = codes(E, K, I), words(E, cdiv(I, 512), K), words(E, cdiv(K, 512), I)
        bf = dict(dtype=BF16, device="cuda")
        self.gu, self.dgu, self.h = torch.empty(M, 2 * I, **bf), torch.empty(M, 2 * I, **bf), torch.empty(M, I, **bf)
        self.y, self.dx = torch.empty(M, K, **bf), torch.empty(M, K, **bf)
        self.dw1, self.dw2 = torch.empty(E, 2 * I, K, device="cuda"), torch.empty(E, K, I, device="cuda")
        self.up1, self.up2 = torch.empty(E * 2, I, K, **bf), torch.empty(E, K, I, **bf)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def __call__(self):
        s, st = self, dict(status=self.status)
        dg.dg_quantize_fp8_blocks(s.w1, s.w1q, sf=s.sf1, sft=s.sf1t)
        dg.dg_quantize_fp8_blocks(s.w2, s.w2q, sf=s.sf2, sft=s.sf2t)
        dg.dg_quantize_fp8(s.x, q=s.xq, sf=s.sfx, qk=s.xk, sfk=s.sfxk, ks=KS)
        dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(s.xq, s.sfx, s.w1q, s.sf1, s.layout, hq=s.hq, sfh=s.sfh, gu=s.gu, **st)
        dg.dg_m_grouped_fp8_gemm_nt_contiguous(s.hq, s.sfh, s.w2q, s.sf2, s.y, s.layout, **st)
        dg.dg_quantize_fp8(s.dy, q=s.yq, sf=s.sfy, qk=s.yk, sfk=s.sfyk, ks=KS)
        dg.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(s.yq, s.sfy, s.w2q, s.sf2t, s.layout, s.gu, s.dgu, h=s.h, **st)
        dg.dg_quantize_fp8(s.dgu, q=s.gq, sf=s.sfg, qk=s.gk, sfk=s.sfgk, ks=KS)
        dg.dg_quantize_fp8(s.h, qk=s.hk, sfk=s.sfhk, ks=KS)
        first = 0
        for e, k in enumerate(KS):               # (the input gradient has no grouped form: expert by expert)
            if k:
                rows = slice(first, first + k)
                dg.dg_fp8_gemm_nn(s.gq[rows], s.sfg[:, rows].contiguous(), s.w1q[e], s.sf1t[e], s.dx[rows], **st)
            first += k
        s.dw1.zero_()
        s.dw2.zero_()
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(s.gk, s.sfgk, s.xk, s.sfxk, s.dw1, KS, ks_dev=s.ks_dev, c=s.dw1, **st)
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(s.yk, s.sfyk, s.hk, s.sfhk, s.dw2, KS, ks_dev=s.ks_dev, c=s.dw2, **st)
        dg.dg_newton_schulz(s.dw1.view(E * 2, I, K), s.up1, **st)
        dg.dg_newton_schulz(s.dw2, s.up2, **st)
        s.w1.sub_(s.up1.view(E, 2 * I, K).float(), alpha=LR)
        s.w2.sub_(s.up2.float(), alpha=LR)


def share(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_step():
    s = Step()
    x, dy = s.x.double().requires_grad_(), s.dy.double()
    w1, w2 = s.w1.double().requires_grad_(), s.w2.double().requires_grad_()
    old1, old2 = s.w1.clone(), s.w2.clone()
    ys, first = [], 0
    for e, k in enumerate(KS):
        g, u = (x[first:first + k] @ w1[e].t()).split(I, 1)
        ys.append((torch.nn.functional.silu(g) * u) @ w2[e].t())
        first += k
    y = torch.cat(ys)
    y.backward(dy)
    s()
    torch.cuda.synchronize()
    assert int(s.status) == 0
    # forward: x, W1, h, W2 in 8 bits: sqrt(4) 2^-4 / sqrt(3)
    assert share(s.y, y.detach()) < 0.073
    for got, want in ((s.dx, x.grad), (s.dw1, w1.grad), (s.dw2, w2.grad)):
        assert share(got, want) < 0.089
    # padded rows stay zero, and an expert without rows has no gradient and no update
    pad = torch.cat([torch.arange(k) >= c for c, k in zip(COUNTS, KS)]).cuda()
    assert not bool(s.y[pad].any()) and not bool(s.dx[pad].any())
    assert not bool(s.dw1[1].any()) and torch.equal(s.w1[1], old1[1]) and torch.equal(s.w2[1], old2[1])
    # the update is the polynomial of the gradient that the step made (tolerance as the operator's own)
    for grad, up in ((s.dw1.view(E * 2, I, K), s.up1), (s.dw2, s.up2)):
        for j in range(grad.shape[0]):
            v = grad[j].double()
            tall = v.shape[0] > v.shape[1]
            v = v.t() if tall else v
            v = v / (v.norm() + 1e-7)
            for _ in range(5):
                p = v @ v.t()
                v = 3.4445 * v + (-4.7750 * p + 2.0315 * (p @ p)) @ v
            v = v.t() if tall else v
            assert float((up[j].double() - v).norm()) <= 5e-3 * float(v.norm())


def test_captured():
    """The step in a graph, replayed twice, gives what two steps give."""
    a, b = Step(), Step()
    for _ in range(3):
        a()
    b()                                           # (what is built once is there before the capture)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for n in ("y", "dx", "dw1", "dw2", "up1", "up2", "w1", "w2"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    assert int(a.status) == 0 and int(b.status) == 0


def test_nothing_to_do():
    """Tensors of no rows, columns or matrices: no error, and nothing is written."""
    def e4m3(*s):
        return torch.empty(*s, dtype=torch.float8_e4m3fn, device="cuda")

    def words(*s):
        return torch.empty(*s, dtype=torch.int32, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 256, **bf16)
    dg.dg_quantize_fp8(x, q=e4m3(0, 256), sf=words(1, 0))
    dg.dg_quantize_fp8(x, qk=e4m3(0, 256), sfk=words(0, 256))
    dg.dg_quantize_fp8(x, qk=e4m3(0, 256), sfk=words(0, 256), ks=[0, 0])
    dg.dg_quantize_fp8(torch.empty(4, 0, **bf16), q=e4m3(4, 0), sf=words(0, 4))
    dg.dg_quantize_fp8_blocks(torch.empty(0, 8, 16, **bf16), e4m3(0, 8, 16), sf=words(0, 1, 8))
    dg.dg_newton_schulz(torch.empty(0, 8, 16, **bf16), torch.empty(0, 8, 16, **bf16))
    dg.dg_newton_schulz(torch.empty(8, 0, **bf16), torch.empty(8, 0, **bf16))
    dg.dg_fp8_gated_gemm_nt(e4m3(0, 128), words(1, 0), e4m3(64, 128), words(1, 64), h=torch.empty(0, 32, **bf16))
    dg.dg_fp8_gated_gemm_nt(e4m3(0, 128), words(1, 0), e4m3(64, 128), words(1, 64), hq=e4m3(0, 32), sfh=words(1, 0))
    dg.dg_fp8_gated_gemm_nn_backward(e4m3(0, 128), words(1, 0), e4m3(128, 32), words(1, 32), torch.empty(0, 64, **bf16),
                                     torch.empty(0, 64, **bf16), h=torch.empty(0, 32, **bf16))
    dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(e4m3(0, 128), words(1, 0), e4m3(2, 64, 128), words(2, 1, 64), words(0),
                                                 h=torch.empty(0, 32, **bf16))
    torch.cuda.synchronize()
