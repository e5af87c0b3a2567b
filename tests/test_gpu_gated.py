"""The gated feed-forward block and its backward pass against the definition in 64 bits.

Tolerances: the tensor cores' sums are within (k/32 + 16) 2^-23 of the sum of the products'
magnitudes (32 products a step, each step truncated); what is stored in bf16 adds 2^-8 of its
value, E4M3 2^-4 of it or 2^-10 of its scale (subnormal codes); the sigmoid is within 2^-19 for
the |g| < 32 of these inputs (2^-21 + 2^-23 |g|, and three more FP32 roundings)."""
import pytest
import torch

from tests._ffn import block_operand, cdiv, gated64, gated_backward64, pack, rows_operand, scale64
from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def sum_error(a, b, k):
    return (cdiv(k, 32) + 16) * 2.0 ** -23 * (a.abs() @ b.abs())


def within(got, ref, tol, what):
    bad = ((got.cpu().double() - ref).abs() > tol) | got.cpu().double().isnan()
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def forward_bounds(x, w1, k):
    gu, h = gated64(x, w1)
    i = w1.shape[0] // 2
    e = sum_error(x, w1.t(), k)
    g, u = gu.split(i, 1)
    tol_h = 1.1 * e[:, :i] * (u.abs() + e[:, i:]) + torch.nn.functional.silu(g).abs() * e[:, i:] + 2.0 ** -18 * h.abs()
    return gu, h, e, tol_h


def check_quantised(hq, sfh, h, tol, what):
    m, i = h.shape
    words = sfh.cpu()
    exps = torch.stack([(words >> (8 * j)) & 255 for j in range(4)], 1).flatten(0, 1)   # [4 slices, align4(m)]
    groups = cdiv(i, 128)
    assert not bool(exps[groups:].any()) and not bool(exps[:, m:].any()), f"{what}: unused bytes"
    pad = torch.nn.functional.pad
    by_group = pad(h.abs(), (0, groups * 128 - i)).view(m, groups, 128)
    slack = pad(tol, (0, groups * 128 - i)).view(m, groups, 128).amax(-1)
    amax = by_group.amax(-1)
    got = torch.exp2(exps[:groups, :m].t().double() - 127)
    ok = (got == scale64(amax)) | (got == scale64(amax + slack)) | (got == scale64((amax - slack).clamp_min(0)))
    assert bool(ok.all()), f"{what}: scales"
    s = got.repeat_interleave(128, 1)[:, :i]
    within(hq.cpu().double() * s, h, tol + torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -10 * s), what)


# (rows, inner width, K): one row, whole and ragged tiles, widths and K that end inside a block
# of 128 and inside a word of 4 blocks, several K ring turns, more tiles than CTA pairs
SIZES = [(1, 16, 16), (256, 128, 128), (129, 144, 80), (7, 1408, 2048), (515, 272, 400), (300, 640, 1040),
         (600, 1408, 384), (2300, 1296, 384)]


@pytest.mark.parametrize("m,i,k", SIZES)
def test_forward(m, i, k):
    torch.manual_seed(m + i + k)
    a, sfa, x = rows_operand(torch.randn(m, k))
    b, sfb, w1 = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    gu64, h64, e, tol = forward_bounds(x, w1, k)
    a, sfa, b, sfb = cuda(a, sfa, b, sfb)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gu = torch.empty(m, 2 * i, dtype=BF16, device="cuda")
    h = torch.empty(m, i, dtype=BF16, device="cuda")
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=h, gu=gu, status=status)
    within(h, h64, tol + 2.0 ** -8 * h64.abs(), "h")
    within(gu, gu64, e + 2.0 ** -8 * gu64.abs(), "gate and up")
    h2 = torch.empty_like(h)
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=h2, status=status)
    assert torch.equal(h, h2)
    hq = torch.empty(m, i, dtype=E4M3, device="cuda")
    sfh = torch.full((cdiv(i, 512), cdiv(m, 4) * 4), -1, dtype=torch.int32, device="cuda")
    gu2 = torch.empty_like(gu)
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, hq=hq, sfh=sfh, gu=gu2, status=status)
    check_quantised(hq, sfh, h64, tol, "quantised h")
    assert torch.equal(gu, gu2) and int(status) == 0


@pytest.mark.parametrize("m,i,k", SIZES)
def test_backward(m, i, k):
    torch.manual_seed(m + 2 * i + k)
    a, sfa, dy = rows_operand(torch.randn(m, k) * 1e-3)
    b, sfb, w2 = block_operand(torch.randn(k, i) * i ** -0.5, along_rows=True)
    gu = (2 * torch.randn(m, 2 * i)).to(BF16)
    ref, h64 = gated_backward64(dy, w2, gu.double())
    g, u = gu.double().split(i, 1)
    e = sum_error(dy, w2, k)
    s = torch.sigmoid(g)
    tol = torch.cat((e * (u * (s * (1 + g * (1 - s)))).abs(), e * (g * s).abs()), 1)
    # s (1 + g (1 - s)) cancels near its zero: an error of 2^-19 of its terms, s and g s (1 - s)
    dh = (dy @ w2).abs()
    tol[:, :i] += 2.0 ** -18 * dh * u.abs() * (s + (g * s).abs())
    tol += (2.0 ** -8 + 2.0 ** -18) * ref.abs()
    a, sfa, b, sfb, gu = cuda(a, sfa, b, sfb, gu)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dgu, h = torch.empty_like(gu), torch.empty(m, i, dtype=BF16, device="cuda")
    dg.dg_fp8_gated_gemm_nn_backward(a, sfa, b, sfb, gu, dgu, h=h, status=status)
    within(dgu, ref, tol, "gradient of gate and up")
    within(h, h64, (2.0 ** -8 + 2.0 ** -18) * h64.abs(), "h")
    once = gu.clone()
    dg.dg_fp8_gated_gemm_nn_backward(a, sfa, b, sfb, once, once, status=status)   # in place, without h
    assert torch.equal(once, dgu) and int(status) == 0


def test_gradient_by_differences():
    """The gradient of sum(h W2^T dY^T) by central differences of the 64-bit forward pass."""
    torch.manual_seed(5)
    m, i, k = 3, 32, 48
    a, sfa, dy = rows_operand(torch.randn(m, k))
    b, sfb, w2 = block_operand(torch.randn(k, i), along_rows=True)
    gu = torch.randn(m, 2 * i).to(BF16)

    def loss(v):
        g, u = v.split(i, 1)
        return float(((g / (1 + torch.exp(-g)) * u) @ w2.t() * dy).sum())
    base, step = gu.double(), 2.0 ** -12
    diff = torch.zeros_like(base)
    for r in range(m):
        for c in range(2 * i):
            d = torch.zeros_like(base)
            d[r, c] = step
            diff[r, c] = (loss(base + d) - loss(base - d)) / (2 * step)
    a, sfa, b, sfb, gu = cuda(a, sfa, b, sfb, gu)
    dgu = torch.empty_like(gu)
    dg.dg_fp8_gated_gemm_nn_backward(a, sfa, b, sfb, gu, dgu)
    # central differences: step^2 / 6 of the third derivative, below 1 times |dh| max(|u|, 1)
    scale = (dy.abs() @ w2.abs()).amax() * base.abs().amax().clamp_min(1)
    within(dgu, diff, 2.0 ** -8 * diff.abs() + scale * (step ** 2 / 6 + 18 * 2.0 ** -23 + 1e-10), "differences")


def grouped_inputs(e, i, k, seed):
    torch.manual_seed(seed)
    layout = torch.tensor([0, 0, -1, 2, 2, 3, -1, 3, 3][:9]).repeat_interleave(128).to(torch.int32)
    return layout, layout.numel()


@pytest.mark.parametrize("i,k", [(272, 384), (512, 128), (1040, 640)])
def test_grouped(i, k):
    e = 4                                         # expert 1 has no rows
    layout, m = grouped_inputs(e, i, k, i)
    a, sfa, x = rows_operand(torch.randn(m, k))
    w1 = [block_operand(torch.randn(2 * i, k) * k ** -0.5) for _ in range(e)]
    w2 = [block_operand(torch.randn(k, i) * i ** -0.5, along_rows=True) for _ in range(e)]
    gu_in = torch.randn(m, 2 * i).to(BF16)
    b, sfb = torch.stack([w[0] for w in w1]).cuda(), torch.stack([w[1] for w in w1]).cuda()
    c, sfc = torch.stack([w[0] for w in w2]).cuda(), torch.stack([w[1] for w in w2]).cuda()
    a, sfa, gl, gu_in = cuda(a, sfa, layout, gu_in)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mark = 77.0
    gu = torch.full((m, 2 * i), mark, dtype=BF16, device="cuda")
    h, h2 = torch.full((m, i), mark, dtype=BF16, device="cuda"), torch.full((m, i), mark, dtype=BF16, device="cuda")
    hq = torch.zeros(m, i, dtype=E4M3, device="cuda")
    sfh = torch.zeros(cdiv(i, 512), m, dtype=torch.int32, device="cuda")
    dgu = torch.full((m, 2 * i), mark, dtype=BF16, device="cuda")
    dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(a, sfa, b, sfb, gl, h=h, gu=gu, status=status)
    dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(a, sfa, b, sfb, gl, hq=hq, sfh=sfh, status=status)
    dg.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(a, sfa, c, sfc, gl, gu_in, dgu, h=h2, status=status)
    none = (layout < 0).cuda()
    for t in (gu, h, h2, dgu):
        assert bool((t[none] == mark).all()), "rows of skipped blocks are left as they were"
    assert not bool(hq.view(torch.uint8)[none].any()) and not bool(sfh[:, none].any())
    for j in range(e):
        rows = (layout == j).nonzero().flatten()
        if not len(rows):
            continue
        gu64, h64, err, tol = forward_bounds(x[rows], w1[j][2], k)
        within(h[rows.cuda()], h64, tol + 2.0 ** -8 * h64.abs(), "h")
        within(gu[rows.cuda()], gu64, err + 2.0 ** -8 * gu64.abs(), "gate and up")
        check_quantised(hq[rows.cuda()], sfh[:, rows.cuda()], h64, tol, "quantised h")
        # (backward by the same rule as the dense call, on this expert's rows alone)
        part = dgu[rows.cuda()]
        alone = torch.empty_like(part)
        q, words, _ = rows_operand(torch.zeros(len(rows), k))
        q = a[rows.cuda()].contiguous()
        words = sfa[:, rows.cuda()].contiguous()
        halone = torch.empty(len(rows), i, dtype=BF16, device="cuda")
        dg.dg_fp8_gated_gemm_nn_backward(q, words, c[j], sfc[j], gu_in[rows.cuda()].contiguous(), alone, h=halone)
        assert torch.equal(part, alone) and torch.equal(h2[rows.cuda()], halone)
    assert int(status) == 0
    layout[256:384] = e                           # no such expert
    dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(a, sfa, b, sfb, layout.cuda(), h=h, status=status)
    assert int(status) == dg.DG_DEV_BAD_GROUP and bool((h[256:384] == mark).all())


def test_strides():
    """Rows of wider buffers, and nothing written beside them."""
    torch.manual_seed(9)
    m, i, k = 140, 48, 96
    a, sfa, x = rows_operand(torch.randn(m, k))
    b, sfb, w1 = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    d, sfd, w2 = block_operand(torch.randn(k, i), along_rows=True)
    wide = torch.zeros(m, k + 32, dtype=torch.uint8)
    wide[:, 16:16 + k] = a.view(torch.uint8)
    bw = torch.zeros(2 * i, k + 16, dtype=torch.uint8)
    bw[:, :k] = b.view(torch.uint8)
    dw = torch.zeros(k, i + 64, dtype=torch.uint8)
    dw[:, 32:32 + i] = d.view(torch.uint8)
    wide, bw, dw, sfa, sfb, sfd = cuda(wide, bw, dw, sfa, sfb, sfd)
    gu_all = torch.full((m + 1, 2 * i + 16), 3.0, dtype=BF16, device="cuda")
    h_all = torch.full((m + 1, i + 8), 3.0, dtype=BF16, device="cuda")
    q_all = torch.full((m + 1, i + 32), 1, dtype=torch.uint8, device="cuda").view(E4M3)
    sfh = torch.empty(1, m, dtype=torch.int32, device="cuda")
    gu, h, hq = gu_all[:m, 8:8 + 2 * i], h_all[:m, :i], q_all[:m, 16:16 + i]
    av, bv, dv = wide.view(E4M3)[:, 16:16 + k], bw.view(E4M3)[:, :k], dw.view(E4M3)[:, 32:32 + i]
    dg.dg_fp8_gated_gemm_nt(av, sfa, bv, sfb, h=h, gu=gu)
    dg.dg_fp8_gated_gemm_nt(av, sfa, bv, sfb, hq=hq, sfh=sfh)
    gu64, h64, e, tol = forward_bounds(x, w1, k)
    within(h, h64, tol + 2.0 ** -8 * h64.abs(), "h")
    within(gu, gu64, e + 2.0 ** -8 * gu64.abs(), "gate and up")
    check_quantised(hq.contiguous(), sfh, h64, tol, "quantised h")
    back = torch.full((m + 1, 2 * i + 8), 3.0, dtype=BF16, device="cuda")
    dg.dg_fp8_gated_gemm_nn_backward(av, sfa, dv, sfd, gu, back[:m, :2 * i])
    plain = torch.empty(m, 2 * i, dtype=BF16, device="cuda")
    dg.dg_fp8_gated_gemm_nn_backward(av.contiguous(), sfa, dv.contiguous(), sfd, gu.contiguous(), plain)
    assert torch.equal(back[:m, :2 * i], plain)
    for t, cols in ((gu_all, slice(8, 8 + 2 * i)), (h_all, slice(0, i)), (back, slice(0, 2 * i))):
        rest = t.clone()
        rest[:m, cols] = 3.0
        assert bool((rest == 3.0).all())
    rest = q_all.view(torch.uint8).clone()
    rest[:m, 16:16 + i] = 1
    assert bool((rest == 1).all())


def test_rows_are_independent():
    """A row's bits do not depend on the other rows; a NaN row stays alone; a row of zeros."""
    torch.manual_seed(11)
    m, i, k = 200, 160, 256
    a, sfa, x = rows_operand(torch.randn(m, k))
    b, sfb, _ = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    a.view(torch.uint8)[17] = 0x7F
    a.view(torch.uint8)[18] = 0
    a, sfa, b, sfb = cuda(a, sfa, b, sfb)
    hq = torch.empty(m, i, dtype=E4M3, device="cuda")
    sfh = torch.empty(cdiv(i, 512), m, dtype=torch.int32, device="cuda")
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, hq=hq, sfh=sfh)
    assert bool(hq[17].float().isnan().all()) and not bool(hq.float().isnan()[torch.arange(m) != 17].any())
    assert not bool(hq[18].float().any()) and int(sfh[0, 18]) == 127 | 127 << 8
    one, sf1 = torch.empty(1, i, dtype=E4M3, device="cuda"), torch.empty(cdiv(i, 512), 4, dtype=torch.int32, device="cuda")
    words = torch.zeros(sfa.shape[0], 4, dtype=torch.int32, device="cuda")
    words[:, 0] = sfa[:, 101]
    dg.dg_fp8_gated_gemm_nt(a[101:102], words, b, sfb, hq=one, sfh=sf1)
    assert torch.equal(one.view(torch.uint8)[0], hq.view(torch.uint8)[101]) and int(sf1[0, 0]) == int(sfh[0, 101])


def test_large_gates():
    """Gates so far below zero that exp(-g) overflows give 0, far above give the product."""
    m, i, k = 4, 16, 128
    x = torch.zeros(m, k)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = -448.0, 448.0, -90.0, 0.0
    w1 = torch.zeros(2 * i, k)
    w1[:i, 0], w1[i:, 0] = 2.0, 1.0
    a, sfa, xv = rows_operand(x)
    b, sfb, wv = block_operand(w1)
    gu64, h64 = gated64(xv, wv)
    a, sfa, b, sfb = cuda(a, sfa, b, sfb)
    h = torch.empty(m, i, dtype=BF16, device="cuda")
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=h)
    # (below the smallest normal FP32, e^-g is infinite and the product 0)
    within(h, h64, 2.0 ** -7 * h64.abs() + 2.0 ** -100, "h")


def test_captured_and_on_another_stream():
    torch.manual_seed(13)
    m, i, k = 384, 256, 512
    a, sfa, _ = rows_operand(torch.randn(m, k))
    b, sfb, _ = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    c, sfc, _ = block_operand(torch.randn(k, i), along_rows=True)
    a, sfa, b, sfb, c, sfc = cuda(a, sfa, b, sfb, c, sfc)
    want = torch.empty(m, i, dtype=BF16, device="cuda")
    gu = torch.empty(m, 2 * i, dtype=BF16, device="cuda")
    wantd = torch.empty_like(gu)
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=want, gu=gu)
    dg.dg_fp8_gated_gemm_nn_backward(a, sfa, c, sfc, gu, wantd)
    h, g2, d = torch.empty_like(want), torch.empty_like(gu), torch.empty_like(gu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=h, gu=g2, stream=side)
    dg.dg_fp8_gated_gemm_nn_backward(a, sfa, c, sfc, g2, d, stream=side)
    side.synchronize()
    assert torch.equal(h, want) and torch.equal(d, wantd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=h, gu=g2)
        dg.dg_fp8_gated_gemm_nn_backward(a, sfa, c, sfc, g2, d)
    h.zero_(), d.zero_(), g2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want) and torch.equal(d, wantd)


def test_last_config():
    a, sfa, _ = rows_operand(torch.randn(300, 128))
    b, sfb, _ = block_operand(torch.randn(512, 128))
    a, sfa, b, sfb = cuda(a, sfa, b, sfb)
    dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, h=torch.empty(300, 256, dtype=BF16, device="cuda"))
    cfg = dg.last_config()
    assert cfg["kind"] == 2 and cfg["launches"] == 1 and cfg["block_m"] == 256


@pytest.mark.parametrize("backward", [False, True])
def test_lost_load_is_reported(backward):
    """A load that never comes ends in a time-out and a status; the next call is whole."""
    torch.manual_seed(17)
    m, i, k = 512, 384, 640
    a, sfa, _ = rows_operand(torch.randn(m, k))
    b, sfb, _ = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    c, sfc, _ = block_operand(torch.randn(k, i), along_rows=True)
    a, sfa, b, sfb, c, sfc = cuda(a, sfa, b, sfb, c, sfc)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gu = torch.randn(m, 2 * i, device="cuda").to(BF16)

    def call():
        if backward:
            out = torch.empty_like(gu)
            dg.dg_fp8_gated_gemm_nn_backward(a, sfa, c, sfc, gu, out, status=status)
            return out
        out = torch.empty(m, i, dtype=E4M3, device="cuda")
        dg.dg_fp8_gated_gemm_nt(a, sfa, b, sfb, hq=out, sfh=torch.empty(1, m, dtype=torch.int32, device="cuda"),
                                status=status)
        return out.view(torch.uint8)
    want = call()
    dg.set_wait_timeout_ms(20)
    dg.set_debug_flags(dg.DG_DEBUG_DROP_ONE_LOAD)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        dg.set_wait_timeout_ms(0)
        dg.set_debug_flags(0)
    assert int(status) == dg.DG_DEV_TIMEOUT
    status.zero_()
    assert torch.equal(call(), want) and int(status) == 0


def test_tiles_of_every_width():
    """A row's bits are the same in tiles of 64, 128 and 256 columns."""
    torch.manual_seed(19)
    i, k = 1296, 640
    a, sfa, _ = rows_operand(torch.randn(4096, k))
    b, sfb, _ = block_operand(torch.randn(2 * i, k) * k ** -0.5)
    c, sfc, _ = block_operand(torch.randn(k, i), along_rows=True)
    gu = torch.randn(4096, 2 * i).to(BF16)
    a, sfa, b, sfb, c, sfc, gu = cuda(a, sfa, b, sfb, c, sfc, gu)
    seen, back, want = set(), set(), None
    for m in (4096, 700, 256, 3):
        hq = torch.empty(m, i, dtype=E4M3, device="cuda")
        sfh = torch.empty(cdiv(i, 512), cdiv(m, 4) * 4, dtype=torch.int32, device="cuda")
        words = torch.zeros(sfa.shape[0], cdiv(m, 4) * 4, dtype=torch.int32, device="cuda")
        words[:, :m] = sfa[:, :m]
        g = torch.empty(m, 2 * i, dtype=BF16, device="cuda")
        h = torch.empty(m, i, dtype=BF16, device="cuda")
        dg.dg_fp8_gated_gemm_nt(a[:m], words, b, sfb, hq=hq, sfh=sfh, gu=g)
        dg.dg_fp8_gated_gemm_nt(a[:m], words, b, sfb, h=h)
        seen.add(dg.last_config()["block_n"])
        d = torch.empty(m, 2 * i, dtype=BF16, device="cuda")
        dg.dg_fp8_gated_gemm_nn_backward(a[:m], words, c, sfc, gu[:m], d)
        back.add(dg.last_config()["block_n"])
        got = (hq.view(torch.uint8), sfh[:, :m].t(), g, h, d)
        if want is None:
            want = got
        for x, y in zip(got, want):
            assert torch.equal(x, y[:m])
    assert seen == {64, 128, 256} and back == {128, 256}


def test_more_narrow_tiles_than_pairs():
    """Experts of 128 rows: each is a tile of its own, so that narrow tiles, chosen for the rows alone, are
    more than the CTA pairs, and a pair goes from one to the next."""
    e, i, k = 8, 2048, 256
    m = 128 * e
    g = torch.Generator().manual_seed(31)

    def codes(*s):
        return torch.randn(*s, generator=g).to(torch.float8_e4m3fn).cuda()

    def words(*s):
        return (torch.randint(124, 130, (*s, 4), generator=g, dtype=torch.uint8).view(torch.int32).view(*s)).cuda()
    dy, w2 = codes(m, k), codes(e, k, i)
    sfdy, sfw2 = words(1, m), words(e, 1, i)
    gu = torch.randn(m, 2 * i, generator=g).to(torch.bfloat16).cuda()
    layout = torch.arange(e, dtype=torch.int32).repeat_interleave(128).cuda()
    dgu, h = torch.empty_like(gu), torch.empty(m, i, dtype=torch.bfloat16, device="cuda")
    dg.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(dy, sfdy, w2, sfw2, layout, gu, dgu, h=h)
    assert dg.last_config()["block_n"] == 128
    want, want_h = torch.empty(128, 2 * i, dtype=torch.bfloat16, device="cuda"), torch.empty_like(h[:128])
    for j in range(e):
        r = slice(128 * j, 128 * j + 128)
        dg.dg_fp8_gated_gemm_nn_backward(dy[r], sfdy[:, r].contiguous(), w2[j], sfw2[j], gu[r], want, h=want_h)
        assert torch.equal(dgu[r], want) and torch.equal(h[r], want_h), j


def test_offsets_past_32_bits():
    """More than 2^32 elements of gate and up: rows at both ends and past 2^31 elements have the bits of a
    small call."""
    m, i, k = 263168, 8192, 128
    g = torch.Generator(device="cuda").manual_seed(5)

    def codes(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.float8_e4m3fn)

    def words(*s):
        return torch.randint(124, 130, (*s, 4), generator=g, device="cuda", dtype=torch.uint8).view(torch.int32).view(*s)
    x, sfx, w1, sf1, w2, sf2 = codes(m, k), words(1, m), codes(2 * i, k), words(1, 2 * i), codes(k, i), words(1, i)
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    gu, h = torch.empty(m, 2 * i, **bf16), torch.empty(m, i, **bf16)
    small, small_h = torch.empty(256, 2 * i, **bf16), torch.empty(256, i, **bf16)
    assert gu.numel() > 2 ** 32
    rows = [slice(r, r + 256) for r in (0, 131072, m - 256)]
    dg.dg_fp8_gated_gemm_nt(x, sfx, w1, sf1, h=h, gu=gu)
    for r in rows:
        dg.dg_fp8_gated_gemm_nt(x[r], sfx[:, r].contiguous(), w1, sf1, h=small_h, gu=small)
        assert torch.equal(small, gu[r]) and torch.equal(small_h, h[r]), r
    kept = [gu[r].clone() for r in rows]
    dg.dg_fp8_gated_gemm_nn_backward(x, sfx, w2, sf2, gu, gu, h=h)
    for r, before in zip(rows, kept):
        dg.dg_fp8_gated_gemm_nn_backward(x[r], sfx[:, r].contiguous(), w2, sf2, before, small, h=small_h)
        assert torch.equal(small, gu[r]) and torch.equal(small_h, h[r]), r
