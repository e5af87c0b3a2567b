"""The limit of a bounded wait counts a kernel's own time only: a decode kernel that starts beside
the end of a kernel that outlasts the limit is none the worse for it."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _codes(*shape):
    return torch.randint(0, 120, shape, dtype=torch.uint8, device="cuda")


def _scales(*shape):
    return torch.full(shape, 0x78787878, dtype=torch.int32, device="cuda")


@pytest.fixture
def knobs():
    yield
    binding.set_num_sms(0)
    binding.set_wait_timeout_ms(2000)


@pytest.mark.parametrize("fmt,m", [("fp4", 1), ("fp8", 1), ("fp8", 5), ("fp4", 6), ("fp8", 12)])
def test_product_after_a_long_gemm(knobs, fmt, m):
    """962 GFLOP on 8 SMs take over 4 ms at the tensor cores' peak rate; the product's limit is 1 ms."""
    M, N, K = 4096, 7168, 16384
    a, b = _codes(M, K).view(torch.float8_e4m3fn), _codes(N, K).view(torch.float8_e4m3fn)
    sfa, sfb = _scales(K // 512, M), _scales(K // 512, N)
    big = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    n, k = 1024, 4096
    w = _codes(n, k // 2) if fmt == "fp4" else _codes(n, k).view(torch.float8_e4m3fn)
    sf = _scales(k // 128 if fmt == "fp4" else k // 512, n)
    x = torch.randn(m, k, device="cuda").bfloat16()
    fn = binding.dg_bf16_fp4_gemv_nt if fmt == "fp4" else binding.dg_bf16_fp8_gemv_nt
    want = fn(x, w, sf, torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
    d, status = torch.full_like(want, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    binding.set_num_sms(8)
    begin.record()
    binding.dg_fp8_gemm_nt(a, sfa, b, sfb, big)
    binding.set_num_sms(0)
    binding.set_wait_timeout_ms(1)
    fn(x, w, sf, d, status=status)
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) > 2.0      # (the GEMM did outlast the limit)
    assert int(status.item()) == 0
    assert torch.equal(d, want)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_down_kernel_after_a_long_up_kernel(knobs, fmt):
    """The layer's up kernel alone reads 268 MB of weights (FP8: twice that) on 2 SMs, which an SM
    does at less than 100 GB/s; the limit is 1 ms."""
    t, e, topk, h, i = 40, 32, 4, 4096, 2048
    per, sl = (2, 128) if fmt == "fp4" else (1, 512)
    w1, w2 = _codes(e, 2 * i, h // per), _codes(e, h, i // per)
    if fmt == "fp8":
        w1, w2 = w1.view(torch.float8_e4m3fn), w2.view(torch.float8_e4m3fn)
    sf1, sf2 = _scales(e, h // sl, 2 * i), _scales(e, i // sl, h)
    x = torch.randn(t, h, device="cuda").bfloat16()
    ids = torch.rand(t, e, device="cuda").topk(topk, -1)[1].int()
    wt = torch.rand(t, topk, device="cuda")
    fn = binding.dg_moe_fp4_layer if fmt == "fp4" else binding.dg_moe_fp8_layer
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    binding.set_num_sms(2)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for limit in (2000, 1):
        binding.set_wait_timeout_ms(limit)
        y = torch.full((t, h), 9.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        begin.record()
        fn(x, ids, wt, w1, sf1, w2, sf2, y, status=status)
        end.record()
        torch.cuda.synchronize()
        assert begin.elapsed_time(end) > 3.0
        outs.append(y)
    assert int(status.item()) == 0
    assert torch.equal(outs[0], outs[1])
