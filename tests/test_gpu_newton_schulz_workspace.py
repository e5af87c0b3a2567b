"""The workspaces of Newton-Schulz calls whose caller gives none: a large one does not stay with its stream."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_large_workspaces_are_not_kept():
    b, r, c = 4, 1024, 8192
    need = dg.newton_schulz_workspace_bytes(b, r, c)
    assert need > dg._MAX_KEPT_BYTES
    g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(1)).cuda()
    want = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    dg.dg_newton_schulz(g, want, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [torch.empty_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    used = torch.cuda.memory_allocated()
    for i, out in enumerate(outs):        # (nothing is waited for: memory that goes back may be in use)
        dg.dg_newton_schulz(g, out, stream=streams[i % 4])
    dg.dg_newton_schulz(g, outs[0])
    assert torch.cuda.memory_allocated() - used <= 8 << 20
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


def test_memory_that_goes_back_serves_its_stream_only():
    """What a call's workspace was may be the next tensor of its stream, whose work comes after the call."""
    b, r, c = 8, 2048, 2048
    g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(2)).cuda()
    want, out = (torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = dg.newton_schulz_workspace_bytes(b, r, c)
    assert n > dg._MAX_KEPT_BYTES
    dg.dg_newton_schulz(g, want, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        dg.dg_newton_schulz(g, out, stream=side)
        with torch.cuda.stream(side):
            torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # on the current stream: other memory
        side.synchronize()
        assert torch.equal(out, want)
