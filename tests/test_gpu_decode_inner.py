"""The MoE layer's inner activations are held to 14 bits."""
import pytest
import torch

from tests import _decode as D
from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _plain(s):
    """(y, bound of |sum - y|) in 64 bits.  The bound: the first product's own through silu (slope at most
    1.1) and the product; h = w silu(g) u to 14 bits (2^-14 of |h|; 2^-25 of the largest of its 32), FP32
    roundings on the way to it (2^-20 of |h|: exp, the quotient and three products), and the second product's
    truncated sums."""
    x, w1, w2 = s["x"].double(), s["d1"], s["d2"]
    i = w2.shape[2]
    y, tol = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    for r in range(x.shape[0]):
        for e, w in zip(s["ids"][r].tolist(), s["weights"][r].double().tolist()):
            gu, b = w1[e] @ x[r], D.product_bound(x[r:r + 1], w1[e])[0]
            g, u = gu[:i], gu[i:]
            act = torch.nn.functional.silu(g) * u
            dact = 1.1 * b[:i] * u.abs() + torch.nn.functional.silu(g).abs() * b[i:]
            dact = dact + (2.0 ** -14 + 2.0 ** -20) * act.abs() + 2.0 ** -25 * D.group_amax(act[None])[0]
            y[r] += w * (w2[e] @ act)
            tol[r] += w * (w2[e].abs() @ (dact + act.abs() * (i / 32 + 16) * 2.0 ** -23))
    return y, tol * 1.01


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("t,e,topk,h,i", [(24, 4, 2, 512, 128), (64, 8, 2, 1024, 128), (13, 3, 3, 256, 384), (3, 8, 2, 1024, 128)])
def test_inner_activations(fmt, t, e, topk, h, i):
    """C is minus the exact result in bf16, so the output is the sum's last bits, 2^-17 of the result."""
    s = T._layer_case(fmt, t, e, topk, h, i, seed=21)
    y, tol = _plain(s)
    c = (-y).bfloat16()
    rest = y + c.double()
    got = T._layer(s, c=c.cuda())
    T._check(got, rest, tol + rest.abs() * 2.0 ** -8, f"{fmt} t{t} {h}x{i}")
