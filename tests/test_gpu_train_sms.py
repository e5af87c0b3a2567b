"""The gated calls and Newton-Schulz run on CTA pairs: one SM is refused, two are enough."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_one_and_two_sms():
    m, i, k = 300, 256, 256
    g = torch.Generator().manual_seed(1)

    def codes(*s):
        return torch.randn(*s, generator=g).to(torch.float8_e4m3fn).cuda()

    def words(*s):
        return torch.randint(124, 130, (*s, 4), generator=g, dtype=torch.uint8).view(torch.int32).view(*s).cuda()
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    x, sfx, w1, sf1, w2, sf2 = codes(m, k), words(1, m), codes(2 * i, k), words(1, 2 * i), codes(k, i), words(1, i)
    grad = torch.randn(64, 300, generator=g).cuda()

    def calls():
        h, gu, up = torch.zeros(m, i, **bf16), torch.zeros(m, 2 * i, **bf16), torch.zeros(64, 300, **bf16)
        dgu = torch.zeros(m, 2 * i, **bf16)
        return (h, gu, dgu, up), (lambda: dg.dg_fp8_gated_gemm_nt(x, sfx, w1, sf1, h=h, gu=gu),
                                  lambda: dg.dg_fp8_gated_gemm_nn_backward(x, sfx, w2, sf2, gu, dgu),
                                  lambda: dg.dg_newton_schulz(grad, up))
    want, run = calls()
    for f in run:
        f()
    try:
        dg.set_num_sms(1)
        out, run = calls()
        for f in run:
            with pytest.raises(dg.DGError) as e:
                f()
            assert e.value.name == "DG_ERR_UNSUPPORTED"
        torch.cuda.synchronize()
        assert not any(bool(t.any()) for t in out)
        dg.set_num_sms(2)
        for f in run:
            f()
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(0)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
