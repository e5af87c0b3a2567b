"""The MoE layer: a token's bits do not depend on the other tokens of the call."""
import pytest
import torch

from tests import _decode as D
from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _run(s, x, ids, weights, c):
    return T._layer({**s, "x": x, "ids": ids, "weights": weights}, c=c.cuda()).cpu()


# the call sizes of one comparison; FP4 has one form of activations up to t = 8 and another above
# (the experts are few enough for that)
@pytest.mark.parametrize("fmt,sizes", [("fp8", (1, 2, 5, 8, 9, 16, 33, 64)), ("fp4", (1, 2, 3, 7, 8)), ("fp4", (9, 16, 17, 40, 64))])
@pytest.mark.parametrize("e,topk,h,i", [(4, 2, 512, 256), (6, 3, 384, 1408), (4, 4, 1152, 640), (8, 4, 256, 2048),
                                        (3, 2, 2048, 128)])
def test_layer_tokens_do_not_depend_on_the_batch(fmt, sizes, e, topk, h, i):
    """C is minus the bf16 result, so what is left is the sum's last bits: any change in the order in
    which a token's products are added shows."""
    s = T._layer_case(fmt, 64, e, topk, h, i)
    g = T._gen(i)
    full = max(sizes)
    x, ids, weights = s["x"][:full], s["ids"][:full], s["weights"][:full]
    c = -_run(s, x, ids, weights, torch.zeros(full, h).bfloat16())
    want = _run(s, x, ids, weights, c)
    assert (want != 0).any()
    for t in sizes:
        rows = torch.randperm(full, generator=g)[:t]                   # other places, another number
        assert torch.equal(_run(s, x[rows], ids[rows], weights[rows], c[rows]), want[rows]), t
        if t < 2:
            continue
        # token 0 of the permutation among tokens that all go elsewhere, or nowhere
        for other in (torch.full((topk,), -1).int(), torch.arange(topk).int(), torch.arange(e)[-topk:].int(),
                      torch.randperm(e, generator=g)[:topk].int()):
            xs, js, ws = torch.randn(t, h, generator=g).bfloat16(), other.repeat(t, 1), torch.rand(t, topk, generator=g)
            at = int(torch.randint(0, t, (1,), generator=g))
            xs[at], js[at], ws[at] = x[rows[0]], ids[rows[0]], weights[rows[0]]
            cs = torch.randn(t, h, generator=g).bfloat16()
            cs[at] = c[rows[0]]
            assert torch.equal(_run(s, xs, js, ws, cs)[at], want[rows[0]]), (t, other)
