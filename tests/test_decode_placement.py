"""Where the operands of the decode calls live: all on the current CUDA device, or the call is
refused before the library is called.  (No call here reaches a launch, with a GPU or without.)"""
import types

import pytest
import torch

from block_scaled_fp8_gb300 import binding as B
from tests.test_decode_marshal import _gemv_args
from tests.test_decode_workspace import _layer_args

STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_scaled_fp8_gb300 import build
    build.build()


class On:
    """A host tensor that says it is on `device`."""

    def __init__(self, tensor, device):
        self.tensor, self.device_index = tensor, device

    def get_device(self):
        return self.device_index

    def __getattr__(self, name):
        return getattr(self.tensor, name)


def _route_args():
    return dict(logits=torch.zeros(4, 64), ids=torch.zeros(4, 4, dtype=torch.int32), weights=torch.zeros(4, 4),
                bias=torch.zeros(64))


def _with_options(args, rows, cols):
    return dict(args, c=torch.zeros(rows, cols).bfloat16(), status=torch.zeros(1, dtype=torch.int32),
                workspace=torch.zeros(1 << 20, dtype=torch.uint8))


CALLS = [(B.dg_bf16_fp4_gemv_nt, _with_options(_gemv_args(), 2, 64)),
         (B.dg_bf16_fp8_gemv_nt, _with_options(_gemv_args(False), 2, 64)),
         (B.dg_moe_route, _route_args()),
         (B.dg_moe_fp4_layer, _with_options(_layer_args(), 3, 256))]


@pytest.mark.parametrize("fn,args", CALLS)
def test_host_tensors_are_refused(fn, args):
    with pytest.raises(AssertionError):
        fn(**args, stream=STREAM)
    with pytest.raises(AssertionError):
        fn(**args)


@pytest.mark.parametrize("fn,args,name", [(f, a, n) for f, a in CALLS for n in a])
@pytest.mark.parametrize("device", [-1, 1])
def test_one_operand_elsewhere_is_refused(fn, args, name, device):
    with pytest.raises(AssertionError, match="current device"):
        fn(**{k: On(t, device if k == name else 0) for k, t in args.items()}, stream=STREAM)


@pytest.mark.parametrize("fn,args", CALLS)
def test_another_device_than_the_current_one_is_refused(fn, args):
    with pytest.raises(AssertionError, match="current device"):
        fn(**{k: On(t, 1) for k, t in args.items()}, stream=STREAM)


def test_weights_of_no_width_need_no_workspace():
    assert B.moe_layer_workspace_bytes(3, 2, 256, 0, 4) == 0
    assert B.moe_layer_workspace_bytes(3, 2, 0, 128, 4) == 0
