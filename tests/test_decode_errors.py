"""Refusals of the decode-side entry points: answered on the host, before any device
access (the pointers here are never dereferenced)."""
import ctypes

import pytest

from block_scaled_fp8_gb300 import binding

P = ctypes.c_void_p
OK, ARG, ALIGN, UNSUP = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_gb300 import build
    build.build()
    return binding.lib()


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("f32", [False, True])
def test_gemv_refusals(lib, fp4, f32):
    fn = getattr(lib, f"dg_bf16_{'fp4' if fp4 else 'fp8'}_gemv_nt" + ("_f32" if f32 else ""))

    def call(a=16, lda=256, b=64, ldb=256, sfb=16, c=0, ldc=64, d=16, ldd=64, m=3, n=64, k=256,
             ws=16, nbytes=1 << 20):
        return fn(P(a), lda, P(b), ldb, P(sfb), P(c), ldc, P(d), ldd, m, n, k, P(ws), nbytes, None, None)
    assert call(m=-1) == ARG and call(n=-8) == ARG and call(k=-128) == ARG
    assert call(m=0) == OK and call(n=0) == OK
    assert call(m=65) == UNSUP
    assert call(d=0) == ARG and call(a=0) == ARG and call(b=0) == ARG and call(sfb=0) == ARG
    assert call(d=24) == ALIGN and call(a=24) == ALIGN and call(sfb=24) == ALIGN and call(c=24) == ALIGN
    assert call(n=60) == ALIGN and call(ldd=66) == ALIGN and call(c=16, ldc=66) == ALIGN
    assert call(ldd=56) == ARG and call(c=16, ldc=56) == ARG
    assert call(k=192) == ALIGN and call(lda=260) == ALIGN and call(lda=248) == ARG
    assert call(b=72) == ALIGN and call(ldb=264) == ALIGN
    assert call(ldb=96 if fp4 else 240) == ARG
    need = lib.dg_bf16_gemv_workspace_bytes(64, 64, 256)
    assert need > 0 and lib.dg_bf16_gemv_workspace_bytes(-1, 64, 256) == -1
    assert call(m=64, ws=0, nbytes=need) == ARG and call(m=64, nbytes=need - 1) == ARG and call(m=64, ws=24) == ALIGN
    if fp4:
        assert call(b=48) == ALIGN and call(ldb=144) == ALIGN     # FP4 rows: 32 bytes


def test_route_refusals(lib):
    def call(logits=16, ld=64, fmt=0, bias=0, ids=16, w=16, t=4, e=64, topk=4, scoring=0):
        return lib.dg_moe_route(P(logits), ld, fmt, P(bias), P(ids), P(w), t, e, topk, scoring, 1, 1.0, None)
    assert call(t=-1) == ARG and call(e=0) == ARG and call(topk=0) == ARG and call(topk=65) == ARG
    assert call(fmt=2) == ARG and call(scoring=2) == ARG and call(ld=63) == ARG
    assert call(e=1025, ld=1025) == UNSUP and call(topk=33) == UNSUP
    assert call(logits=0) == ARG and call(ids=0) == ARG and call(w=0) == ARG
    assert call(logits=18) == ALIGN and call(bias=18) == ALIGN and call(w=18) == ALIGN
    assert call(t=0, logits=0) == OK


@pytest.mark.parametrize("fp4", [True, False])
def test_layer_refusals(lib, fp4):
    fn = lib.dg_moe_fp4_layer if fp4 else lib.dg_moe_fp8_layer

    def call(x=16, ldx=256, ids=16, w=16, w1=64, sf1=16, w2=64, sf2=16, c=0, ldc=256, y=16, ldy=256, t=3, h=256, i=128,
             e=4, topk=2, ws=16, nbytes=None):
        nbytes = 1 << 24 if nbytes is None else nbytes
        return fn(P(x), ldx, P(ids), P(w), P(w1), P(sf1), P(w2), P(sf2), P(c), ldc, P(y), ldy, t, h, i, e, topk, P(ws),
                  nbytes, None, None)
    need = lib.dg_moe_layer_workspace_bytes(3, 2, 256, 128, 4)
    assert need > 0 and lib.dg_moe_layer_workspace_bytes(-1, 2, 256, 128, 4) == -1
    assert call(t=-1) == ARG and call(h=-128) == ARG and call(i=-128) == ARG and call(e=0) == ARG and call(topk=0) == ARG
    assert call(t=0) == OK and call(h=0) == OK
    assert call(t=65) == UNSUP and call(topk=17) == UNSUP and call(e=1025) == UNSUP
    assert call(h=192) == ALIGN and call(i=64) == ALIGN
    for name in ("x", "ids", "w", "w1", "sf1", "w2", "sf2", "y", "ws"):
        assert call(**{name: 0}) == ARG, name
    for name in ("x", "w1", "w2", "sf1", "sf2", "y", "ws", "c"):
        assert call(**{name: 72}) == ALIGN, name
    assert call(ids=18) == ALIGN and call(w=18) == ALIGN
    assert call(ldx=248) == ARG and call(ldy=248) == ARG and call(c=16, ldc=248) == ARG
    assert call(ldx=260) == ALIGN and call(ldy=260) == ALIGN and call(c=16, ldc=260) == ALIGN
    assert call(nbytes=need - 1) == ARG
    if fp4:
        assert call(w1=48) == ALIGN and call(w2=48) == ALIGN
