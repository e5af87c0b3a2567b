"""One token out of a buffer whose rows are any number of elements apart."""
import pytest
import torch

from tests import _decode as D
from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _row(t, odd):
    """t [1, C] as the first row of a buffer with rows of C + odd elements."""
    wide = torch.zeros(3, t.shape[1] + odd, dtype=t.dtype, device="cuda")
    wide[0, :t.shape[1]] = t[0]
    return wide[:1, :t.shape[1]]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("odd", [1, 3, 4, 10])
def test_product(fmt, f32, odd):
    g = T._gen(odd)
    n, k = 136, 384
    a = torch.randn(1, k, generator=g).bfloat16().cuda()
    codes, s, _ = D.quantize(torch.randn(n, k, generator=g), fmt)
    codes, sf = codes.cuda(), D.pack_scales(s)
    c = torch.randn(1, n, generator=g).to(torch.float32 if f32 else torch.bfloat16).cuda()
    want = T._gemv(fmt, a, codes, sf, f32, c)
    d = _row(torch.full_like(c, 7.0), odd)
    rest = d._base.clone()
    T._gemv(fmt, _row(a, odd), codes, sf, f32, _row(c, odd), d)
    assert torch.equal(d, want)
    rest[:1, :n] = want
    assert torch.equal(d._base, rest)                  # nothing else is written


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_layer(fmt):
    s = T._layer_case(fmt, 1, 4, 2, 256, 128)
    c = torch.randn(1, 256, generator=T._gen(1)).bfloat16().cuda()
    want = T._layer(s, c=c)
    y = _row(torch.full_like(c, 7.0), 5)
    T._layer(s, x=_row(s["x"].cuda(), 3), c=_row(c, 1), y=y)
    assert torch.equal(y, want)
