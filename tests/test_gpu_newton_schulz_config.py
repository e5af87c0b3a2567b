"""A Newton-Schulz call that launches nothing does not pass for the last configuration launched."""
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

# The runtime refuses launches on the legacy default stream while a blocking stream is captured: an error on the
# host, after which that capture is void.  (In a process of its own, which ends there.)
SCRIPT = """
import ctypes
import os
import torch
from block_scaled_fp8_gb300 import binding as dg
g = torch.randn(64, 64, device="cuda")
out = torch.empty(64, 64, dtype=torch.bfloat16, device="cuda")
ws = torch.empty(dg.newton_schulz_workspace_bytes(1, 64, 64), dtype=torch.uint8, device="cuda")
dg.dg_newton_schulz(g, out, workspace=ws)
torch.cuda.synchronize()
before = dg.last_config()
assert before["launches"] == 3
name = [line.split("/")[-1].strip() for line in open("/proc/self/maps") if "libcudart.so" in line][0]
cudart, blocking = ctypes.CDLL(name), ctypes.c_void_p()
assert cudart.cudaStreamCreate(ctypes.byref(blocking)) == 0
assert cudart.cudaStreamBeginCapture(blocking, 0) == 0
try:
    dg.dg_newton_schulz(g, out, workspace=ws)
    name = "none"
except dg.DGError as e:
    name = e.name
print(name, dg.last_config() == before, flush=True)
os._exit(0)
"""


def test_a_refused_launch_is_not_recorded():
    r = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["DG_ERR_CUDA", "True"], r.stdout + r.stderr
