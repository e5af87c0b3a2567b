"""Decode calls on streams that the caller names, with workspaces that the binding makes."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _product(m=20, n=1024, k=2048):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    sf = torch.full((k // 128, n), 0x78787878, dtype=torch.int32, device="cuda")
    a = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    return a, w, sf, torch.empty(m, n, dtype=torch.bfloat16, device="cuda")


def test_a_named_stream_does_not_wait_for_the_current_one():
    a, w, sf, d = _product()
    assert binding.gemv_workspace_bytes(20, 1024, 2048) > 0
    want = binding.dg_bf16_fp4_gemv_nt(a, w, sf, d.clone())
    other = torch.cuda.Stream()
    binding.dg_bf16_fp4_gemv_nt(a, w, sf, d, stream=other)   # (kernels loaded, memory there)
    d.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(1 << 30)                                # half a second on the current stream
    busy = torch.cuda.Event()
    busy.record()
    binding.dg_bf16_fp4_gemv_nt(a, w, sf, d, stream=other)
    other.synchronize()
    still = not busy.query()
    got = d.clone()
    torch.cuda.synchronize()
    assert still
    assert torch.equal(got, want)


def test_calls_in_turn_on_two_streams():
    """Calls with different operands in turn on two named streams, each with a workspace of its own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    ops = [_product(20), _product(17)]
    ops[1][0].mul_(-3.0)
    want = [binding.dg_bf16_fp4_gemv_nt(*o[:3], o[3].clone()) for o in ops]
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(o[3]) for _ in range(50)] for o in ops]
    torch.cuda.synchronize()
    for r in range(50):
        for s, o, out in zip(streams, ops, outs):
            binding.dg_bf16_fp4_gemv_nt(*o[:3], out[r], stream=s)
    torch.cuda.synchronize()
    for v, out in zip(want, outs):
        assert all(torch.equal(v, d) for d in out)


def test_a_named_stream_in_a_capture():
    a, w, sf, d = _product()
    want = binding.dg_bf16_fp4_gemv_nt(a, w, sf, d.clone())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        binding.dg_bf16_fp4_gemv_nt(a, w, sf, d, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)
