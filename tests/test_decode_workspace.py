"""The workspaces that the binding makes for decode calls whose caller gives none."""
import types

import pytest
import torch

from block_scaled_fp8_gb300 import binding as B
from tests.test_decode_marshal import _gemv_args

STREAM = types.SimpleNamespace(cuda_stream=0)   # (never used: every call here is refused)


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_gb300 import build
    build.build()


def _layer_args(t=3, e=4, topk=2):
    return dict(x=torch.zeros(t, 256).bfloat16(), ids=torch.zeros(t, topk, dtype=torch.int32),
                weights=torch.zeros(t, topk), w1=torch.zeros(e, 256, 128, dtype=torch.uint8),
                sf1=torch.zeros(e, 2, 256, dtype=torch.int32), w2=torch.zeros(e, 256, 64, dtype=torch.uint8),
                sf2=torch.zeros(e, 1, 256, dtype=torch.int32), y=torch.zeros(t, 256).bfloat16())


@pytest.mark.parametrize("fn,args", [
    (B.dg_bf16_fp4_gemv_nt, _gemv_args(m=65)), (B.dg_bf16_fp8_gemv_nt, _gemv_args(False, m=4096)),
    (B.dg_moe_fp4_layer, _layer_args(t=65)), (B.dg_moe_fp4_layer, _layer_args(topk=17)),
    (B.dg_moe_fp4_layer, _layer_args(e=1025)),
])
def test_refused_sizes_make_no_workspace(fn, args, monkeypatch):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(a) or empty(*a, **k))
    with pytest.raises(B.DGError) as e:
        fn(**args, stream=STREAM)
    assert e.value.name == "DG_ERR_UNSUPPORTED"
    assert not made


def test_size_functions_know_the_limits():
    assert B.gemv_workspace_bytes(64, 64, 256) > 0 and B.gemv_workspace_bytes(65, 64, 256) == -1
    assert B.moe_layer_workspace_bytes(64, 16, 256, 128, 1024) > 0
    for sizes in ((65, 2, 256, 128, 4), (3, 17, 256, 128, 4), (3, 2, 256, 128, 1025), (3, 2, (1 << 24) + 128, 128, 4),
                  (3, 2, 256, (1 << 24) + 128, 4)):
        assert B.moe_layer_workspace_bytes(*sizes) == -1, sizes
