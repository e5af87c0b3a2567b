"""Newton-Schulz calls of more tiles than their counter holds are refused by the binding as by the library: before a
workspace is made, on tensors of any place."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_gb300 import build
    build.build()


@pytest.mark.parametrize("rows,cols,steps", [(1, 2 ** 20, 6), (2 ** 20, 1, 6), (300, 4096, 700)])
def test_too_many_tiles(rows, cols, steps, monkeypatch):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(a) or empty(*a, **k))
    g, out = (torch.zeros(rows * cols, dtype=t).as_strided((4096, rows, cols), (0, cols, 1))
              for t in (torch.float32, torch.bfloat16))
    with pytest.raises(binding.DGError) as e:
        binding.dg_newton_schulz(g, out, steps=steps)
    assert e.value.name == "DG_ERR_UNSUPPORTED"
    assert not made
    # one step is taken, and so asks where the tensors are
    with pytest.raises(AssertionError):
        binding.dg_newton_schulz(g, out, steps=1)
