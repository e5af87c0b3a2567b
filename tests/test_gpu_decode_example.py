"""The example's decode step: every token counts, and a wrong result shows."""
import pytest
import torch

from tests import test_gpu_decode as T
from tests.test_gpu_decode_chain import _example

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

SMALL = ["--hidden", "512", "--inner", "256", "--vocab", "1024"]


@pytest.mark.parametrize("seed", [0, 1, 2, 3])
@pytest.mark.parametrize("tokens,experts,topk", [(1, 8, 2), (1, 16, 4), (6, 8, 3)])
def test_step(tokens, experts, topk, seed):
    """As test_example_step, whose bound this is; no token is left out of the comparison."""
    same, worst = _example().main(["--tokens", str(tokens), "--experts", str(experts), "--topk", str(topk),
                                   "--seed", str(seed), *SMALL])
    assert 0.0 < worst <= 2.0 ** -6


@pytest.mark.parametrize("part", ["w1_64", "w2_64", "head_64", "router_64"])
def test_a_mistake_in_the_plain_form_shows(part, monkeypatch):
    """One token, one part of the 64-bit weights in another order: the comparison fails."""
    example = _example()
    plain = example.Block.plain

    def wrong(block, chosen):
        w = getattr(block, part)
        setattr(block, part, w.roll(1, -1))
        return plain(block, chosen)

    monkeypatch.setattr(example.Block, "plain", wrong)
    args = ["--tokens", "1", "--experts", "8", "--topk", "2", *SMALL]
    try:
        _, worst = example.main(args)
    except AssertionError:
        return
    assert worst > 2.0 ** -6


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,topk", [(1, 1), (5, 5), (33, 4), (256, 8), (384, 1), (1000, 32)])
@pytest.mark.parametrize("bias", [False, True])
def test_one_token_of_well_separated_keys(scoring, e, topk, bias):
    """Logits of e distinct values from -4 to 4 in random order: the scores of neighbours differ by 1e-4
    of themselves at least, hundreds of times the error of an FP32 score."""
    order = torch.randperm(e, generator=T._gen(e + topk))
    logits = torch.empty(e)
    logits[order] = torch.linspace(4.0, -4.0, e) if e > 1 else torch.zeros(1)
    b = torch.full((e,), 0.125) if bias else None        # (shifts all keys alike)
    ids, w = T._route(logits[None].cuda(), topk, bias=None if b is None else b.cuda(), scoring=scoring, scale=2.0)
    assert ids[0].tolist() == order[:topk].tolist()
    x = logits[order].double()
    s = (torch.softmax(x, 0) if scoring == "softmax" else torch.sigmoid(x))[:topk]
    assert ((w[0].double() - 2 * s / s.sum()).abs() <= 2.0 ** -18 * 2 * s / s.sum()).all()
