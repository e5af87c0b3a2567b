"""A matrix's bits do not depend on where it lies: in a batch of odd sizes the matrices start at every
alignment, alone on a line of memory."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r,c", [(37, 41), (251, 333), (333, 251), (5, 3), (1, 9001), (1001, 1003)])
def test_alignment_leaves_the_bits(r, c, dtype):
    b = 9
    g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(r + c)).to(dtype).cuda()
    out = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    one = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    for steps in (1, 5):
        dg.dg_newton_schulz(g, out, steps=steps)
        for j in range(b):
            dg.dg_newton_schulz(g[j].clone(), one, steps=steps)
            assert torch.equal(one, out[j]), (steps, j)
