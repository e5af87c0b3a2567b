"""The workspaces that the binding keeps go with their thread, and there are only so many."""
import threading

import pytest
import torch

from block_scaled_fp8_gb300 import binding
from tests.test_gpu_decode_streams import _product

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_a_thread_takes_its_workspaces_with_it():
    a, w, sf, d = _product()
    binding.dg_bf16_fp4_gemv_nt(a, w, sf, d)
    torch.cuda.synchronize()
    want, before = d.clone(), torch.cuda.memory_allocated()
    outs = [torch.zeros_like(d) for _ in range(12)]
    used = torch.cuda.memory_allocated()

    def work(out):
        binding.dg_bf16_fp4_gemv_nt(a, w, sf, out)
        torch.cuda.synchronize()

    for out in outs:
        thread = threading.Thread(target=work, args=(out,))
        thread.start()
        thread.join()
    assert torch.cuda.memory_allocated() - used < 1 << 20      # less than one kept workspace
    assert used >= before and all(torch.equal(out, want) for out in outs)


def test_many_streams_keep_few_workspaces():
    a, w, sf, d = _product()
    binding.dg_bf16_fp4_gemv_nt(a, w, sf, d)
    torch.cuda.synchronize()
    want = d.clone()
    streams = [torch.cuda.Stream() for _ in range(20)]
    outs = [torch.zeros_like(d) for _ in range(60)]
    torch.cuda.synchronize()
    used = torch.cuda.memory_allocated()
    for i, out in enumerate(outs):       # (nothing is waited for: memory that goes may be in use)
        binding.dg_bf16_fp4_gemv_nt(a, w, sf, out, stream=streams[i % 20])
    assert torch.cuda.memory_allocated() - used <= 8 << 20
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
