"""The decode-side operators together, and their failure detection."""
import importlib.util
import os

import pytest
import torch

from block_scaled_fp8_gb300 import binding
from tests import _decode as D

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,experts,topk", [(1, 8, 2), (5, 16, 4), (20, 8, 3)])
def test_example_step(tokens, experts, topk):
    """Route, layer and products in one captured graph against the step in 64 bits.  The
    output is rounded to bf16 twice (h, whose products with the head then differ by up to
    2^-9 of their terms, and the output itself): 2^-6 of the output's RMS covers outputs of 4
    times the RMS."""
    same, worst = _example().main(["--tokens", str(tokens), "--experts", str(experts), "--topk", str(topk),
                                   "--hidden", "512", "--inner", "256", "--vocab", "1024"])
    assert same >= tokens - 1
    assert worst <= 2.0 ** -6


def _gemv(fmt, m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    codes, s, _ = D.quantize(torch.randn(n, k, generator=g), fmt)
    a, b, sf = torch.randn(m, k, generator=g).bfloat16().cuda(), codes.cuda(), D.pack_scales(s)
    fn = {"fp4": binding.dg_bf16_fp4_gemv_nt, "fp8": binding.dg_bf16_fp8_gemv_nt}[fmt]
    return lambda d, status: fn(a, b, sf, d, status=status), (m, n)


def _layer(fmt, t, e, topk, h, i):
    g = torch.Generator().manual_seed(t + h + i)
    w = [[D.quantize(torch.randn(n, k, generator=g) * k ** -0.5, fmt)[:2] for _ in range(e)] for n, k in ((2 * i, h), (h, i))]
    codes = [torch.stack([c.view(torch.uint8) for c, _ in x]).view(x[0][0].dtype).cuda() for x in w]
    sf = [torch.stack([D.pack_scales(s) for _, s in x]) for x in w]
    x = torch.randn(t, h, generator=g).bfloat16().cuda()
    ids = torch.rand(t, e, generator=g).topk(topk, -1)[1].int().cuda()
    wt = torch.rand(t, topk, generator=g).cuda()
    fn = {"fp4": binding.dg_moe_fp4_layer, "fp8": binding.dg_moe_fp8_layer}[fmt]
    return lambda d, status: fn(x, ids, wt, codes[0], sf[0], codes[1], sf[1], d, status=status), (t, h)


@pytest.mark.parametrize("make,args", [
    (_gemv, ("fp4", 1, 512, 4096)),       # split over a cluster, rows split by its CTAs
    (_gemv, ("fp8", 2, 40000, 512)),      # persistent CTAs
    (_gemv, ("fp4", 6, 512, 4096)),       # rows split beforehand
    (_gemv, ("fp4", 20, 512, 4096)),
    (_gemv, ("fp8", 40, 33000, 512)),
    (_layer, ("fp4", 2, 8, 2, 512, 256)),    # the up kernel splits the rows
    (_layer, ("fp8", 16, 4, 2, 512, 256)),
    (_layer, ("fp4", 40, 4, 2, 512, 256)),
])
def test_dropped_load_times_out_and_context_survives(make, args):
    call, shape = make(*args)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        d = torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda")
        call(d, status)
        torch.cuda.synchronize()
        return d

    first = run()
    assert int(status.item()) == 0
    binding.set_wait_timeout_ms(100)
    try:
        binding.set_debug_flags(binding.DG_DEBUG_DROP_ONE_LOAD)
        run()
        assert int(status.item()) & binding.DG_DEV_TIMEOUT
        # the drop flag cleared itself; the next call is complete and has the same bits
        status.zero_()
        again = run()
        assert int(status.item()) == 0
    finally:
        binding.set_debug_flags(0)
        binding.set_wait_timeout_ms(2000)
    assert torch.equal(first, again)


def test_calls_in_a_row_with_gemms():
    """GEMMs, few-row products and layers back to back on one stream, each starting beside the
    end of the one before (all of them allocate TMEM): every call gives the bits that it gives alone."""
    from block_scaled_fp8_gb300 import inputs
    calls = []
    for M, N, K in ((128, 512, 1024), (512, 768, 512)):
        case = inputs.dense_case(M, N, K, seed=5)
        a, b = case.a.cuda(), case.b.cuda()
        sfa, sfb = binding.transform_sf(case.sfa.cuda(), 1, M), binding.transform_sf(case.sfb.cuda(), 128, N)
        calls.append((lambda d, status, a=a, b=b, sfa=sfa, sfb=sfb: binding.dg_fp8_gemm_nt(a, sfa, b, sfb, d, status=status),
                      (M, N)))
    calls += [_gemv("fp4", 1, 1024, 2048), _gemv("fp8", 12, 2048, 1024), _gemv("fp4", 40, 20480, 512),
              _layer("fp4", 3, 8, 2, 512, 256), _layer("fp8", 24, 8, 2, 512, 256)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    alone = []
    for call, shape in calls:
        d = torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda")
        call(d, status)
        torch.cuda.synchronize()
        alone.append(d)
    order = [i for first in range(len(calls)) for second in range(len(calls)) for i in (first, second)]
    outs = [torch.full(calls[i][1], 9.0, dtype=torch.bfloat16, device="cuda") for i in order]
    torch.cuda.synchronize()
    for i, d in zip(order, outs):
        calls[i][0](d, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for i, d in zip(order, outs):
        assert torch.equal(d, alone[i]), i
