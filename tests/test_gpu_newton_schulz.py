"""Newton-Schulz orthogonalisation against the definition in 64 bits.

Tolerance, as a share of the result's 2-norm: the operands of a step's three products have a
relative error of 2^-12 each (11 bits, half a step, near uniform: 2^-12 / sqrt(3) RMS).  Errors of X
pass through X <- a X + (b A + c A A) X, whose slope a + 3 b s^2 + 5 c s^4 is at most 3.45 for the singular
values s of these inputs, as does X itself while it is small, so relative to X they do not
grow until the last steps, where s is 0.7 to 1.2 and the slope at most 3.45 against a value of
s: each step then adds at most (|b| s^2 + 2 |c| s^4 ...) < 12 times 2^-12 / sqrt(3) of X, and
passes on the step before times at most 3.45.  Two such steps: (1 + 3.45) 12 2^-12 / sqrt(3) = 7.5e-3
as the worst case; 4e-3 is asked for here, and bf16's rounding (2^-8 / sqrt(3) = 2.3e-3) comes on top
in quadrature: 5e-3 in all.  A single element: 8 times the RMS of that, beside 2^-8 of its value."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
COEF, EPS = (3.4445, -4.7750, 2.0315), 1e-7


def plain(g, steps=5, coef=COEF, eps=EPS):
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.norm() + eps)
    a, b, c = coef
    for _ in range(steps):
        p = x @ x.t()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.t() if tall else x


def close(out, ref, share=5e-3, what=""):
    o = out.cpu().double()
    assert bool(o.isfinite().all()), what
    d, norm = o - ref, float(ref.norm())
    rms = norm / ref.numel() ** 0.5
    assert float(d.norm()) <= share * norm, f"{what}: {float(d.norm()) / norm}"
    assert bool((d.abs() <= 8 * share * rms + 2.0 ** -8 * ref.abs()).all()), f"{what}: an element"


def gradient(r, c, seed, kind="noise"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, c, generator=g)
    if kind == "decay":       # singular values over four decades
        x = torch.randn(r, r, generator=g) * torch.logspace(0, -4, r) @ x
    elif kind == "low":       # a few strong directions
        x = torch.randn(r, 8, generator=g) @ torch.randn(8, c, generator=g) + 0.01 * x
    return 1e-3 * x


# one element, one row or column, odd sizes, both orientations, one and several tiles, K that ends
# inside a stage, more tiles than CTA pairs
SIZES = [(1, 1), (1, 300), (77, 1), (5, 3), (24, 25), (64, 64), (250, 1000), (256, 512), (257, 255), (700, 333), (530, 2100)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r,c", SIZES)
def test_sizes(r, c, dtype):
    g = gradient(r, c, r + c).to(dtype)
    out = torch.full((r, c), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dg.dg_newton_schulz(g.cuda(), out, status=status)
    close(out, plain(g), what=f"{r}x{c}")
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["noise", "decay", "low"])
@pytest.mark.parametrize("r,c", [(320, 900), (900, 320), (384, 384)])
def test_spectra(r, c, kind):
    g = gradient(r, c, 3, kind)
    out = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g.cuda(), out)
    close(out, plain(g), what=kind)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_polynomials(steps):
    g = gradient(130, 400, 4)
    out = torch.empty(130, 400, dtype=torch.bfloat16, device="cuda")
    for coef in (COEF, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)):
        dg.dg_newton_schulz(g.cuda(), out, steps=steps, coef=coef, eps=1e-3)
        close(out, plain(g, steps, coef, 1e-3), what=str(coef))


def test_orthogonal():
    """With the cubic polynomial and enough steps the rows become orthonormal."""
    g = gradient(96, 600, 5).cuda()
    out = torch.empty(96, 600, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g, out, steps=14, coef=(1.5, -0.5, 0.0))
    gram = out.double() @ out.double().t()
    # rows of 600 elements with bf16 roundings of 2^-8 and the result's own 4e-3
    assert float((gram - torch.eye(96, device="cuda", dtype=torch.double)).abs().max()) < 2e-2


@pytest.mark.parametrize("r,c", [(300, 200), (200, 300)])
def test_batch_and_strides(r, c):
    b = 3
    g = torch.stack([gradient(r, c, 7 + j) * 10.0 ** j for j in range(b)])
    wide = torch.zeros(b, r + 2, c + 5)
    wide[:, 1:1 + r, 3:3 + c] = g
    view = wide.cuda()[:, 1:1 + r, 3:3 + c]
    buf = torch.full((b, r + 1, c + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :r, 1:1 + c]
    dg.dg_newton_schulz(view, out)
    for j in range(b):
        close(out[j], plain(g[j]), what=f"matrix {j}")
        one = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
        dg.dg_newton_schulz(view[j], one)
        assert torch.equal(one, out[j]), "a matrix's result does not depend on the others"
    rest = buf.clone()
    rest[:, :r, 1:1 + c] = 9.0
    assert bool((rest == 9.0).all())
    same = g[1].bfloat16().cuda()
    want = torch.empty_like(same)
    dg.dg_newton_schulz(same, want)
    dg.dg_newton_schulz(same, same)        # in place
    assert torch.equal(same, want)


def test_magnitudes():
    """Scales at which squares leave FP32, and a matrix of zeros."""
    g = gradient(60, 90, 8)
    want = plain(g, eps=0.0)
    out = torch.empty(60, 90, dtype=torch.bfloat16, device="cuda")
    for s in (2.0 ** 90, 2.0 ** -90, 1.0, 2.0 ** 40, 2.0 ** -30):
        dg.dg_newton_schulz((g * s).cuda(), out, eps=0.0)
        close(out, want, what=str(s))
    for eps in (0.0, EPS):
        dg.dg_newton_schulz(torch.zeros(60, 90, device="cuda"), out, eps=eps)
        assert not bool(out.any())


def test_not_finite():
    g = torch.stack([gradient(70, 50, 9), gradient(70, 50, 10), gradient(70, 50, 11)]).cuda()
    out = torch.empty(3, 70, 50, dtype=torch.bfloat16, device="cuda")
    want = torch.empty(70, 50, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g[1], want)
    g[0, 3, 3], g[2, 69, 49] = float("nan"), float("inf")
    dg.dg_newton_schulz(g, out)
    assert bool(out[0].isnan().all()) and bool(out[2].isnan().all()) and torch.equal(out[1], want)


def test_workspace_stream_and_capture():
    g = gradient(300, 520, 12).cuda()
    need = dg.newton_schulz_workspace_bytes(1, 300, 520)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")     # (NaN wherever it is read unwritten)
    want, out = (torch.empty(300, 520, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.dg_newton_schulz(g, want, workspace=ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    close(want, plain(g.cpu()))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dg.dg_newton_schulz(g, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], []
    for _ in range(2):                       # two graphs, each with a workspace of its own
        graph, o = torch.cuda.CUDAGraph(), torch.zeros_like(want)
        with torch.cuda.graph(graph):
            dg.dg_newton_schulz(g, o)
        graphs.append(graph), outs.append(o)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert dg.last_config()["launches"] == 3


def test_lost_load_is_reported():
    """A load that never comes ends in a time-out and a status, not in a hang."""
    g = gradient(300, 520, 12).cuda()
    out = torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dg.set_wait_timeout_ms(20)
    dg.set_debug_flags(dg.DG_DEBUG_DROP_ONE_LOAD)
    try:
        dg.dg_newton_schulz(g, out, status=status)
        torch.cuda.synchronize()
    finally:
        dg.set_wait_timeout_ms(0)
        dg.set_debug_flags(0)
    assert int(status) == dg.DG_DEV_TIMEOUT
    status.zero_()
    dg.dg_newton_schulz(g, out, status=status)
    close(out, plain(g.cpu()))
    assert int(status) == 0


@pytest.mark.parametrize("b,r,c", [(700, 40, 64), (300, 20, 33), (200, 130, 70)])
def test_many_small_matrices(b, r, c):
    """More matrices than CTA pairs, so that a pair goes from one diagonal tile to the next."""
    g = torch.stack([gradient(r, c, j) * 2.0 ** (j % 7) for j in range(b)])
    out = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g.cuda(), out)
    for j in range(0, b, 7):
        close(out[j], plain(g[j]), what=f"matrix {j}")
    one = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    for j in (0, 75, 76, 152, b - 1):
        dg.dg_newton_schulz(g[j].cuda(), one)
        assert torch.equal(one, out[j])


@pytest.mark.parametrize("b", [9, 10])
def test_two_groups(b):
    """Enough large matrices for two groups of phases, of equal and of unequal numbers."""
    r, c = 1024, 2064
    g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(b)).cuda()
    out = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dg.dg_newton_schulz(g, out, steps=3, status=status)
    assert int(status) == 0
    one = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    for j in (0, b // 2, b - 1):
        dg.dg_newton_schulz(g[j], one, steps=3)
        assert torch.equal(one, out[j])
    x = g[b - 1].double()
    x = x / (x.norm() + EPS)
    for _ in range(3):
        p = x @ x.t()
        x = COEF[0] * x + (COEF[1] * p + COEF[2] * (p @ p)) @ x
    close(out[b - 1], x.cpu())


@pytest.mark.parametrize("r,c", [(1, 24), (24, 1), (1, 20), (1, 1)])
def test_batch_of_single_rows_and_columns(r, c):
    """Matrices closer to one another than the row stride that a single row stands for."""
    g = torch.stack([gradient(r, c, 40 + j) for j in range(5)])
    out = torch.full((7, r, c), 9.0, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g.cuda(), out[1:6])
    assert bool((out[0] == 9.0).all()) and bool((out[6] == 9.0).all())
    for j in range(5):
        close(out[1 + j], plain(g[j]), what=f"matrix {j}")


@pytest.mark.parametrize("b,r,c", [(4, 1024, 1024), (6, 1024, 1024), (8, 1000, 1024), (2, 2112, 1536), (5, 1536, 1536)])
def test_groups_and_tiles_leave_the_bits(b, r, c):
    """A matrix's result does not depend on batch, and so not on the tiles and groups that a batch makes
    the call choose: narrow and wide tiles, two groups, equal and unequal."""
    g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(b + r)).cuda()
    out, one = (torch.empty(*s, r, c, dtype=torch.bfloat16, device="cuda") for s in ((b,), ()))
    for steps in (1, 5):
        dg.dg_newton_schulz(g, out, steps=steps)
        for j in range(b):
            dg.dg_newton_schulz(g[j], one, steps=steps)
            assert torch.equal(one, out[j]), (steps, j)
    close(out[b - 1], plain(g[b - 1].cpu()))


@pytest.mark.parametrize("scale", [2.0 ** -140, 2.0 ** -126, 2.0 ** -75, 1.0, 2.0 ** 64, 2.0 ** 126])
def test_norm_and_eps_of_any_magnitude(scale):
    """eps beside, below and above the norm, up to FP32's ends (values below 2^-126 have few bits left,
    which the definition is given as well)."""
    g = (torch.tensor([[1.0, -0.5, 0.25], [0.5, 1.0, 0.75]]) * scale).float()
    out = torch.empty(2, 3, dtype=torch.bfloat16, device="cuda")
    for ratio in (0.0, 2.0 ** -20, 0.5, 1.0, 4.0):
        eps = float(torch.tensor(scale * ratio).float())     # as the call takes it
        dg.dg_newton_schulz(g.cuda(), out, steps=1, eps=eps)
        close(out, plain(g, steps=1, eps=eps), what=f"{scale} {ratio}")
    dg.dg_newton_schulz(g.cuda(), out, steps=1, eps=float("inf"))
    assert not bool(out.any())


def test_last_config():
    """The products' tiles and grid as they were chosen."""
    for (b, r, c), (bn, stages, grid) in (((1, 64, 64), (64, 6, 2)), ((1, 250, 1000), (64, 6, 32)), ((4, 4096, 1024), (256, 5, None))):
        g = torch.randn(b, r, c, device="cuda")
        dg.dg_newton_schulz(g, torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda"), steps=1)
        v = dg.last_config()
        assert (v["block_m"], v["block_n"], v["stages"], v["launches"]) == (256, bn, stages, 3)
        assert v["grid"] == (grid or torch.cuda.get_device_properties(0).multi_processor_count)
