"""How near Newton-Schulz comes to its definition in 64 bits, beside the rounding of its result to bf16.

The header's figures, as shares of the result's norm: 1e-3 where the short side is 250 or more, 1.5e-3 from 24 on,
5e-3 below.  They hold only with all that the operator keeps beside its 11-bit operands: without the diagonals
in FP32 noise of 512x512 is off by 1.5e-3, without the low plane of X a decaying spectrum by 7e-3, and
small matrices with a few strong directions by 2e-3 to 7e-3 where the update's product leaves the low plane out.
(Those from the same roundings done in 64 bits.)  The rounding to bf16 is known, r: the difference of
the 64-bit result and itself rounded; it does not go with the operator's own error, so that the two add in
quadrature, up to 4 / sqrt(elements) of their product; matrices of a few elements are given their sum."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg
from tests.test_gpu_newton_schulz import gradient, plain

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def allowed(ref, short):
    own = 1e-3 if short >= 250 else 1.5e-3 if short >= 24 else 5e-3
    r = float((ref.bfloat16().double() - ref).norm() / ref.norm())
    if short < 24:
        return r + own
    return (r * r + own * own + 2 * r * own * 4 / ref.numel() ** 0.5) ** 0.5


SIZES = [(2, 2), (2, 3), (4, 4), (5, 3), (16, 16), (16, 700), (24, 25), (40, 64), (64, 64), (64, 2000), (2000, 64),
         (96, 96), (128, 128), (192, 1024), (193, 1024), (200, 200), (250, 1000), (256, 2048), (512, 512), (320, 900), (900, 320)]


@pytest.mark.parametrize("kind", ["noise", "decay", "low"])
@pytest.mark.parametrize("r,c", SIZES)
def test_share_of_the_result(r, c, kind):
    n = 8 if r * c < 10000 else 2
    g = torch.stack([gradient(r, c, 100 + j, kind) for j in range(n)])
    out = torch.empty(n, r, c, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g.cuda(), out)
    for j in range(n):
        ref = plain(g[j])
        off = float((out[j].cpu().double() - ref).norm() / ref.norm())
        assert off <= allowed(ref, min(r, c)), (j, off)
