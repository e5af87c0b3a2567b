"""What the gated feed-forward calls refuse, on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

from block_scaled_fp8_gb300 import binding

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_gb300 import build
    build.build()
    return binding.lib()


def forward(lib, grouped=False, **kw):
    v = dict(a=16, lda=256, sfa=16, b=16, ldb=256, sfb=16, gu=None, ldgu=0, h=16, ldh=128, hq=None, ldhq=0, sfh=None,
             layout=16, m=256, i=128, k=256, e=2)
    v.update(kw)
    args = [P(v["a"]), v["lda"], P(v["sfa"]), P(v["b"]), v["ldb"], P(v["sfb"]), P(v["gu"]), v["ldgu"], P(v["h"]),
            v["ldh"], P(v["hq"]), v["ldhq"], P(v["sfh"])]
    if grouped:
        return lib.dg_m_grouped_fp8_gated_gemm_nt_contiguous(*args, P(v["layout"]), v["m"], v["i"], v["k"], v["e"],
                                                             None, None)
    return lib.dg_fp8_gated_gemm_nt(*args, v["m"], v["i"], v["k"], None, None)


def backward(lib, grouped=False, **kw):
    v = dict(dy=16, lddy=256, sfdy=16, w2=16, ldw2=128, sfw2=16, gu=16, ldgu=256, dgu=16, lddgu=256, h=None, ldh=0,
             layout=16, m=256, i=128, k=256, e=2)
    v.update(kw)
    args = [P(v["dy"]), v["lddy"], P(v["sfdy"]), P(v["w2"]), v["ldw2"], P(v["sfw2"]), P(v["gu"]), v["ldgu"],
            P(v["dgu"]), v["lddgu"], P(v["h"]), v["ldh"]]
    if grouped:
        return lib.dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(*args, P(v["layout"]), v["m"], v["i"], v["k"],
                                                                      v["e"], None, None)
    return lib.dg_fp8_gated_gemm_nn_backward(*args, v["m"], v["i"], v["k"], None, None)


OK, ARG, ALIGN, LAYOUT, UNSUPPORTED = 0, 1, 2, 3, 4
BOTH = [  # refused (or nothing to do) in each of the four calls
    (dict(m=-1), ARG), (dict(i=-16), ARG), (dict(k=-1), ARG), (dict(m=0), OK), (dict(i=0), OK),
    (dict(k=0), UNSUPPORTED), (dict(i=120), ALIGN), (dict(k=250, lda=256, lddy=256), ALIGN),
    (dict(i=2 ** 30 - 64, ldgu=2 ** 31, lddgu=2 ** 31, ldh=2 ** 31, ldw2=2 ** 31, ldhq=2 ** 31, m=2 ** 24), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BOTH)
def test_both_directions(lib, kw, want):
    for fn in (forward, backward):
        assert fn(lib, **kw) == want, fn.__name__
        if kw.get("m", 0) <= 256:
            assert fn(lib, grouped=True, **kw) == want, fn.__name__


def test_int_range(lib):
    top = 2 ** 31 - 1
    assert forward(lib, m=top) == UNSUPPORTED and backward(lib, m=top) == UNSUPPORTED
    assert forward(lib, k=top - 15, lda=2 ** 31, ldb=2 ** 31) == UNSUPPORTED
    assert forward(lib, i=2 ** 30, ldh=2 ** 31) == UNSUPPORTED
    assert forward(lib, grouped=True, e=2 ** 24, m=128) == UNSUPPORTED          # e * 2 I, and e itself
    assert forward(lib, grouped=True, m=131072 + 256) == UNSUPPORTED
    assert backward(lib, grouped=True, e=32767, k=2 ** 20, lddy=2 ** 20) == UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(a=0), ARG), (dict(b=0), ARG), (dict(sfa=0), ARG), (dict(sfb=0), ARG), (dict(h=None), ARG),
    (dict(h=16, hq=16, ldhq=128, sfh=16), ARG), (dict(h=None, hq=16, ldhq=128), ARG), (dict(lda=240), ARG),
    (dict(ldb=240), ARG), (dict(ldh=120), ARG), (dict(gu=16, ldgu=248), ARG), (dict(h=None, hq=16, ldhq=112, sfh=16), ARG),
    (dict(a=24), ALIGN), (dict(b=8), ALIGN), (dict(sfa=20), ALIGN), (dict(sfb=4), ALIGN), (dict(lda=264), ALIGN),
    (dict(ldb=260), ALIGN), (dict(ldh=132), ALIGN), (dict(h=20), ALIGN), (dict(gu=18, ldgu=256), ALIGN),
    (dict(gu=16, ldgu=260), ALIGN), (dict(h=None, hq=20, ldhq=128, sfh=16), ALIGN),
    (dict(h=None, hq=16, ldhq=136, sfh=16), ALIGN), (dict(h=None, hq=16, ldhq=128, sfh=8), ALIGN)])
def test_forward_refusals(lib, kw, want):
    assert forward(lib, **kw) == want
    assert forward(lib, grouped=True, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), ARG), (dict(w2=0), ARG), (dict(sfdy=0), ARG), (dict(sfw2=0), ARG), (dict(gu=0), ARG), (dict(dgu=0), ARG),
    (dict(lddy=240), ARG), (dict(ldw2=112), ARG), (dict(ldgu=248), ARG), (dict(lddgu=248), ARG), (dict(h=16, ldh=120), ARG),
    (dict(dy=8), ALIGN), (dict(w2=24), ALIGN), (dict(lddy=264), ALIGN), (dict(ldw2=136), ALIGN), (dict(gu=24), ALIGN),
    (dict(ldgu=260), ALIGN), (dict(dgu=8), ALIGN), (dict(lddgu=258), ALIGN), (dict(h=24, ldh=128), ALIGN),
    (dict(h=16, ldh=130), ALIGN)])
def test_backward_refusals(lib, kw, want):
    assert backward(lib, **kw) == want
    assert backward(lib, grouped=True, **kw) == want


def test_grouped_refusals(lib):
    for fn in (forward, backward):
        assert fn(lib, grouped=True, m=300) == LAYOUT
        assert fn(lib, grouped=True, layout=0) == ARG
        assert fn(lib, grouped=True, layout=18) == ALIGN
        assert fn(lib, grouped=True, e=0) == ARG
    assert backward(lib, grouped=True, k=240, lddy=256) == ALIGN     # experts along K: whole blocks


def test_binding_checks():
    e4, bf, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32

    def t(*shape, dtype=e4):
        return torch.zeros(*shape, dtype=torch.uint8).view(e4) if dtype is e4 else torch.zeros(*shape, dtype=dtype)
    ok = dict(a=t(8, 256), sfa=t(1, 8, dtype=i32), b=t(64, 256), sfb=t(1, 64, dtype=i32), h=t(8, 32, dtype=bf))

    def call(**kw):
        v = {**ok, **kw}
        binding.dg_fp8_gated_gemm_nt(v.pop("a"), v.pop("sfa"), v.pop("b"), v.pop("sfb"), **v)
    for kw in (dict(a=t(8, 256, dtype=bf)), dict(a=t(8, 512)[:, ::2]), dict(sfa=t(1, 7, dtype=i32)), dict(sfa=t(2, 8, dtype=i32)),
               dict(sfb=t(1, 60, dtype=i32)), dict(b=t(64, 128)), dict(h=None), dict(h=t(8, 64, dtype=bf)),
               dict(hq=t(8, 32), sfh=t(1, 8, dtype=i32)), dict(h=None, hq=t(8, 32), sfh=t(1, 4, dtype=i32)),
               dict(gu=t(8, 32, dtype=bf)), dict(status=t(1, dtype=torch.int64)), dict()):   # (the last: CPU tensors)
        with pytest.raises(AssertionError):
            call(**kw)
    with pytest.raises(AssertionError):
        binding.dg_m_grouped_fp8_gated_gemm_nt_contiguous(t(128, 256), t(1, 128, dtype=i32), t(2, 64, 256),
                                                          t(2, 1, 64, dtype=i32), t(128, dtype=torch.int64).long(),
                                                          h=t(128, 32, dtype=bf))
    with pytest.raises(AssertionError):
        binding.dg_fp8_gated_gemm_nn_backward(t(8, 256), t(1, 8, dtype=i32), t(256, 32), t(1, 32, dtype=i32),
                                              t(8, 32, dtype=bf), t(8, 64, dtype=bf))
