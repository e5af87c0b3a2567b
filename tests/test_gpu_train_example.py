"""The training example runs, and its gradients are those of the step in 64 bits as near as 8-bit operands
allow: 2^-4 / sqrt(3) for each of them (y: x, W1, h, W2; the gradients at most six)."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("ffn_training", os.path.join(ROOT, "examples", "ffn_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("rows,hidden,inner", [(128, 256, 128), (384, 400, 272), (1024, 2048, 1408)])
def test_step(rows, hidden, inner):
    errors = _example().main(["--rows", str(rows), "--hidden", str(hidden), "--inner", str(inner)])
    assert errors[0] < 0.073 and max(errors[1:]) < 0.089
    assert min(errors) > 1e-3        # (8-bit operands were in fact used)


def test_a_mistake_in_the_plain_form_shows(monkeypatch):
    m = _example()
    plain = m.Block.plain

    def wrong(block):
        y, dx, dw1, dw2 = plain(block)
        return y, dx, dw1.roll(1, 0), dw2
    monkeypatch.setattr(m.Block, "plain", wrong)
    assert m.main(["--rows", "128", "--hidden", "256", "--inner", "128"])[2] > 0.5
