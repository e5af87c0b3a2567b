"""Sizes at the end of the int range: refused on the host, before any device access."""
import ctypes

import pytest

from block_scaled_fp8_gb300 import binding

P = ctypes.c_void_p
UNSUP = 4
LIMIT = 2 ** 31 - 256


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_gb300 import build
    build.build()
    return binding.lib()


@pytest.mark.parametrize("fn", ["dg_bf16_fp4_gemv_nt", "dg_bf16_fp8_gemv_nt_f32"])
def test_products(lib, fn):
    """n rounded up to 128 rows, k to 256: 2^31 - 8 and 2^31 - 128 would leave the range."""
    def call(n=64, k=256):
        return getattr(lib, fn)(P(16 * 2), 1 << 32, P(64), 1 << 32, P(16), None, 0, P(16), 1 << 32, 1, n, k, P(16), 1 << 40,
                                None, None)
    assert call(n=2 ** 31 - 8) == UNSUP and call(k=2 ** 31 - 128) == UNSUP
    assert lib.dg_bf16_gemv_workspace_bytes(12, 2 ** 31 - 8, 256) == -1
    assert lib.dg_bf16_gemv_workspace_bytes(12, 64, 2 ** 31 - 128) == -1
    assert lib.dg_bf16_gemv_workspace_bytes(12, LIMIT, LIMIT) > 0


def test_routing(lib):
    """8 tokens to a block."""
    assert lib.dg_moe_route(P(16), 64, 0, None, P(16), P(16), 2 ** 31 - 1, 64, 4, 0, 1, 1.0, None) == UNSUP
