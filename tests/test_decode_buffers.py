"""Status words and workspaces that the kernels could not write to as they stand: refused before the
library is called."""
import types

import pytest
import torch

from block_scaled_fp8_gb300 import binding as B
from tests.test_decode_marshal import _gemv_args
from tests.test_decode_workspace import _layer_args

STREAM = types.SimpleNamespace(cuda_stream=0)
CALLS = [(B.dg_bf16_fp4_gemv_nt, _gemv_args(m=65)), (B.dg_moe_fp4_layer, _layer_args(t=65))]


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_gb300 import build
    build.build()


# (65 rows: the library would refuse the sizes, so nothing is launched where the check is missing)
@pytest.mark.parametrize("fn,args", CALLS)
@pytest.mark.parametrize("status", [
    torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32),
    torch.zeros(8, dtype=torch.int32)[::4], torch.zeros(1)])
def test_status_words(fn, args, status):
    with pytest.raises(AssertionError):
        fn(**args, status=status, stream=STREAM)


@pytest.mark.parametrize("fn,args", CALLS)
@pytest.mark.parametrize("workspace", [
    torch.zeros(1 << 22, dtype=torch.uint8)[::2],                 # every other byte is someone else's
    torch.zeros(1, dtype=torch.uint8).expand(1 << 22)])           # one byte
def test_workspaces_are_one_range(fn, args, workspace):
    with pytest.raises(AssertionError):
        fn(**args, workspace=workspace, stream=STREAM)
