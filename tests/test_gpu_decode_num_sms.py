"""dg_set_num_sms and the decode kernels: no more CTAs than SMs, the same results."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding
from tests import _decode as D
from tests import test_gpu_decode as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture
def num_sms():
    yield binding.set_num_sms
    binding.set_num_sms(0)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("m,n,k", [(1, 264, 1024), (1, 20000, 256), (3, 2112, 1408), (8, 1000, 2048), (17, 520, 4096),
                                   (20, 20000, 256), (64, 776, 1152), (64, 40000, 128)])
def test_products(num_sms, fmt, m, n, k):
    g = T._gen(m + n + k)
    a = torch.randn(m, k, generator=g).bfloat16()
    codes, s, gran = D.quantize(torch.randn(n, k, generator=g), fmt)
    w = D.dequantize(codes, s, gran)
    sf = D.pack_scales(s)
    ref, tol = a.double() @ w.t(), D.product_bound(a.double(), w)
    for limit in (1, 7, 40, 100, 151):
        num_sms(limit)
        d = T._gemv(fmt, a.cuda(), codes.cuda(), sf, True)
        assert binding.last_config()["grid"] <= limit
        T._check(d, ref, tol + ref.abs() * 2.0 ** -23, f"{fmt} {m}x{n}x{k} on {limit} SMs")


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("t,e,topk,h,i", [(1, 8, 2, 1024, 256), (5, 6, 3, 384, 640), (16, 8, 4, 640, 256), (64, 8, 2, 512, 384)])
def test_layer(num_sms, fmt, t, e, topk, h, i):
    s = T._layer_case(fmt, t, e, topk, h, i)
    ref, tol = D.layer_plain(s["x"], s["ids"], s["weights"], s["d1"], s["d2"], None)
    for limit in (1, 7, 40, 151):
        num_sms(limit)
        y = T._layer(s)
        assert binding.last_config()["grid"] <= limit      # (the down kernel's)
        T._check(y, ref, tol, f"{fmt} t{t} on {limit} SMs")


def test_all_sms_are_no_limit(num_sms):
    """A setting of all SMs, or more, is the default: the same bits."""
    s = T._layer_case("fp4", 3, 8, 2, 512, 256)
    want = T._layer(s)
    config = binding.last_config()
    sms = binding.get_num_sms()
    for n in (sms, sms + 100):
        num_sms(n)
        assert torch.equal(T._layer(s), want)
        assert binding.last_config() == config
