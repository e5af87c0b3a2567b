"""The decode calls' argument checks in the binding: wrong dtypes, shapes and layouts are
refused before the library is called, what the library refuses raises DGError."""
import types

import pytest
import torch

from block_scaled_fp8_gb300 import binding as B

STREAM = types.SimpleNamespace(cuda_stream=0)   # (never used: every call here is refused)


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_gb300 import build
    build.build()


def _gemv_args(fp4=True, m=2, n=64, k=256):
    b = torch.zeros(n, k // 2, dtype=torch.uint8) if fp4 else torch.zeros(n, k).to(torch.float8_e4m3fn)
    return dict(a=torch.zeros(m, k).bfloat16(), b=b, sfb=torch.zeros(2 if fp4 else 1, n, dtype=torch.int32),
                d=torch.zeros(m, n).bfloat16())


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("change", [
    dict(a=torch.zeros(2, 256)), dict(a=torch.zeros(2, 128).bfloat16()), dict(a=torch.zeros(256).bfloat16()),
    dict(a=torch.zeros(256, 2).bfloat16().t()), dict(b=torch.zeros(64, 128)), dict(sfb=torch.zeros(2, 64)),
    dict(sfb=torch.zeros(1, 32, dtype=torch.int32)), dict(d=torch.zeros(2, 64)), dict(d=torch.zeros(3, 64).bfloat16()),
    dict(d=torch.zeros(64, 2).bfloat16().t()), dict(c=torch.zeros(2, 64)), dict(c=torch.zeros(2, 56).bfloat16()),
])
def test_gemv_arguments(fp4, change):
    fn = B.dg_bf16_fp4_gemv_nt if fp4 else B.dg_bf16_fp8_gemv_nt
    with pytest.raises(AssertionError):
        fn(**{**_gemv_args(fp4), **change}, stream=STREAM)


@pytest.mark.parametrize("fn,fp4", [(B.dg_bf16_fp4_gemv_nt_f32, True), (B.dg_bf16_fp8_gemv_nt_f32, False)])
def test_gemv_f32_wants_fp32(fn, fp4):
    with pytest.raises(AssertionError):
        fn(**_gemv_args(fp4), stream=STREAM)


def test_gemv_library_refusals():
    with pytest.raises(B.DGError) as e:   # more rows than the call takes
        B.dg_bf16_fp4_gemv_nt(**_gemv_args(m=65), workspace=torch.zeros(1 << 20, dtype=torch.uint8), stream=STREAM)
    assert e.value.name == "DG_ERR_UNSUPPORTED"
    with pytest.raises(B.DGError) as e:   # too small a workspace
        B.dg_bf16_fp4_gemv_nt(**_gemv_args(m=20), workspace=torch.zeros(16, dtype=torch.uint8), stream=STREAM)
    assert e.value.name == "DG_ERR_INVALID_ARG"


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(4, 64, dtype=torch.float64)), dict(logits=torch.zeros(5, 64)),
    dict(logits=torch.zeros(64, 4).t()), dict(ids=torch.zeros(4, 4)), dict(ids=torch.zeros(4, 8, dtype=torch.int32)[:, ::2]),
    dict(weights=torch.zeros(4, 3)), dict(weights=torch.zeros(4, 4).bfloat16()), dict(bias=torch.zeros(63)),
    dict(bias=torch.zeros(64).bfloat16()), dict(scoring="other"),
])
def test_route_arguments(change):
    args = dict(logits=torch.zeros(4, 64), ids=torch.zeros(4, 4, dtype=torch.int32), weights=torch.zeros(4, 4))
    with pytest.raises(AssertionError):
        B.dg_moe_route(**{**args, **change}, stream=STREAM)


@pytest.mark.parametrize("change", [
    dict(x=torch.zeros(3, 256)), dict(x=torch.zeros(2, 256).bfloat16()), dict(ids=torch.zeros(3, 2)),
    dict(weights=torch.zeros(3, 3)), dict(w1=torch.zeros(4, 255, 128, dtype=torch.uint8)),
    dict(w1=torch.zeros(4, 256, 128)), dict(w2=torch.zeros(3, 256, 64, dtype=torch.uint8)),
    dict(sf1=torch.zeros(4, 1, 256, dtype=torch.int32)), dict(sf2=torch.zeros(4, 1, 256)),
    dict(y=torch.zeros(3, 128).bfloat16()), dict(c=torch.zeros(3, 256)),
])
def test_layer_arguments(change):
    args = dict(x=torch.zeros(3, 256).bfloat16(), ids=torch.zeros(3, 2, dtype=torch.int32), weights=torch.zeros(3, 2),
                w1=torch.zeros(4, 256, 128, dtype=torch.uint8), sf1=torch.zeros(4, 2, 256, dtype=torch.int32),
                w2=torch.zeros(4, 256, 64, dtype=torch.uint8), sf2=torch.zeros(4, 1, 256, dtype=torch.int32),
                y=torch.zeros(3, 256).bfloat16(), workspace=torch.zeros(1 << 22, dtype=torch.uint8))
    with pytest.raises(AssertionError):
        B.dg_moe_fp4_layer(**{**args, **change}, stream=STREAM)
    with pytest.raises(AssertionError):   # FP4 weights given to the FP8 form
        B.dg_moe_fp8_layer(**args, stream=STREAM)
