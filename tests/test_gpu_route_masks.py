"""Experts that a bias takes out of the routing."""
import pytest
import torch

from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [8, 40, 256, 1000])
@pytest.mark.parametrize("out", [float("-inf"), float("nan")])
def test_bias_masks_experts(scoring, e, out):
    """Of e experts three are left, two of them with a logit, for 4 slots."""
    logits = torch.randn(5, e, generator=T._gen(e))
    logits[:, e - 1], logits[:, 2] = 3.0, 1.0
    logits[:, 5] = float("-inf")
    bias = torch.full((e,), out)
    bias[[2, 5, e - 1]] = 0.25
    ids, w = T._route(logits.cuda(), 4, bias=bias.cuda(), scoring=scoring)
    assert (ids == torch.tensor([e - 1, 2, -1, -1]).int()).all()
    x = torch.tensor([3.0, 1.0], dtype=torch.float64)
    s = torch.exp(x - 3.0) if scoring == "softmax" else torch.sigmoid(x)
    # expf or sigmoid, one division: 2^-21 of a weight covers their roundings
    assert ((w[:, :2].double() - s / s.sum()).abs() <= 2.0 ** -21).all()
    assert (w[:, 2:] == 0).all()
