"""What the quantiser and the Newton-Schulz call refuse, on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

from block_scaled_fp8_gb300 import binding

P = ctypes.c_void_p
OK, ARG, ALIGN, LAYOUT, UNSUPPORTED = 0, 1, 2, 3, 4
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_gb300 import build
    build.build()
    return binding.lib()


def quantize(lib, **kw):
    v = dict(x=16, fmt=0, ldx=256, q=16, ldq=256, sf=16, qk=None, ldqk=256, sfk=None, rows=128, cols=256, ks=None, groups=0)
    v.update(kw)
    ks = None if v["ks"] is None else (ctypes.c_int * max(1, len(v["ks"])))(*v["ks"])
    return lib.dg_quantize_fp8(P(v["x"]), v["fmt"], v["ldx"], P(v["q"]), v["ldq"], P(v["sf"]), P(v["qk"]), v["ldqk"],
                               P(v["sfk"]), v["rows"], v["cols"], ks, v["groups"] if ks is None else len(v["ks"]), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(fmt=2), ARG), (dict(q=None), ARG), (dict(rows=0), OK),
    (dict(cols=0, ldx=0, ldq=0), OK), (dict(x=0), ARG), (dict(sf=0), ARG), (dict(q=None, qk=16), ARG), (dict(ldx=252), ARG),
    (dict(ldq=240), ARG), (dict(q=None, qk=16, sfk=16, ldqk=240), ARG), (dict(x=8), ALIGN), (dict(ldx=258), ALIGN),
    (dict(fmt=1, ldx=260), ALIGN), (dict(q=24), ALIGN), (dict(ldq=264), ALIGN), (dict(sf=8), ALIGN),
    (dict(qk=16, sfk=20), ALIGN), (dict(qk=18, sfk=16), ALIGN), (dict(qk=16, sfk=16, ldqk=272 + 8), ALIGN),
    (dict(rows=TOP), UNSUPPORTED), (dict(cols=TOP, ldx=2 ** 32, ldq=2 ** 32), UNSUPPORTED),
    (dict(ks=[128]), ARG), (dict(qk=16, sfk=16, ks=[100]), ARG), (dict(qk=16, sfk=16, ks=[-128, 256]), ARG),
    (dict(qk=16, sfk=16, ks=[256]), LAYOUT), (dict(qk=16, sfk=16, ks=[128], cols=254), LAYOUT),
    (dict(qk=16, sfk=16, ks=[0] * 256), ARG), (dict(qk=16, sfk=16, ks=[0, 0], rows=0), OK)])
def test_quantize(lib, kw, want):
    assert quantize(lib, **kw) == want


def blocks(lib, **kw):
    v = dict(x=16, fmt=0, ldx=256, xb=32768, q=16, ldq=256, qb=32768, sf=16, sft=16, batch=2, rows=128, cols=256)
    v.update(kw)
    return lib.dg_quantize_fp8_blocks(P(v["x"]), v["fmt"], v["ldx"], v["xb"], P(v["q"]), v["ldq"], v["qb"], P(v["sf"]),
                                      P(v["sft"]), v["batch"], v["rows"], v["cols"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), ARG), (dict(rows=-1), ARG), (dict(fmt=7), ARG), (dict(batch=0), OK), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(x=0), ARG), (dict(q=0), ARG), (dict(sf=0, sft=0), ARG), (dict(ldx=128), ARG), (dict(ldq=128), ARG),
    (dict(xb=-4), ARG), (dict(qb=16), ARG), (dict(qb=0), ARG), (dict(qb=32776), ALIGN), (dict(xb=32766), ALIGN),
    (dict(x=20), ALIGN), (dict(q=8), ALIGN), (dict(sf=4), ALIGN), (dict(sft=8), ALIGN), (dict(ldx=257), ALIGN),
    (dict(ldq=260, qb=65536), ALIGN), (dict(batch=65536), UNSUPPORTED), (dict(rows=TOP), UNSUPPORTED)])
def test_blocks(lib, kw, want):
    assert blocks(lib, **kw) == want


def schulz(lib, **kw):
    v = dict(g=16, fmt=0, ldg=64, gb=2048, out=16, ldo=64, ob=2048, batch=2, rows=32, cols=64, steps=5, eps=0.0, ws=128,
             bytes=1 << 24)
    v.update(kw)
    return lib.dg_newton_schulz(P(v["g"]), v["fmt"], v["ldg"], v["gb"], P(v["out"]), v["ldo"], v["ob"], v["batch"], v["rows"],
                                v["cols"], v["steps"], 3.0, -4.0, 2.0, v["eps"], P(v["ws"]), v["bytes"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), ARG), (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(steps=0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(fmt=3), ARG), (dict(batch=0), OK), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(g=0), ARG), (dict(out=0), ARG), (dict(ws=0), ARG), (dict(ldg=63), ARG), (dict(ldo=63), ARG), (dict(gb=-1), ARG),
    (dict(ob=2047), ARG), (dict(bytes=1000), ARG), (dict(g=18), ALIGN), (dict(fmt=1, g=17), ALIGN), (dict(out=17), ALIGN),
    (dict(ws=64), ALIGN), (dict(steps=1001), UNSUPPORTED), (dict(batch=4097), UNSUPPORTED),
    (dict(rows=2 ** 20 + 1), UNSUPPORTED), (dict(rows=2 ** 16, cols=2 ** 16, ldg=2 ** 16, ldo=2 ** 16), UNSUPPORTED),
    (dict(cols=TOP, ldg=2 ** 31, ldo=2 ** 31), UNSUPPORTED)])
def test_newton_schulz(lib, kw, want):
    assert schulz(lib, **kw) == want


def test_newton_schulz_workspace(lib):
    assert binding.newton_schulz_workspace_bytes(-1, 4, 4) == -1
    assert binding.newton_schulz_workspace_bytes(1, 2 ** 20 + 1, 4) == -1
    assert binding.newton_schulz_workspace_bytes(5000, 4, 4) == -1
    a, b = binding.newton_schulz_workspace_bytes(1, 250, 1000), binding.newton_schulz_workspace_bytes(3, 250, 1000)
    # three planes of 250 x 1024, two matrices of 250 x 256, of 2 bytes; sums and diagonals beside them
    assert a >= 2 * 250 * (3 * 1024 + 2 * 256) and b - 3 * a <= 0 and b % 128 == 0 and a % 128 == 0
    assert binding.newton_schulz_workspace_bytes(1, 1000, 250) == a


@pytest.mark.parametrize("over", [254, 512, 1022])
def test_quantize_sizes_near_the_int_range(lib, over):
    """A tile's columns and rows past the matrix still have to be ints: 512 of them, and 8 beside."""
    n = TOP - over
    assert quantize(lib, cols=n, ldx=2 ** 32, ldq=2 ** 32) == UNSUPPORTED
    assert quantize(lib, rows=n) == UNSUPPORTED
    assert blocks(lib, rows=n, qb=2 ** 40, batch=1) == UNSUPPORTED
    assert blocks(lib, cols=n, ldx=2 ** 32, ldq=2 ** 32, batch=1) == UNSUPPORTED


def test_nothing_to_do_needs_no_pointers(lib):
    """Tensors without elements have null pointers."""
    none = dict(x=None, q=None, sf=None, qk=None, sfk=None)
    assert quantize(lib, rows=0, **none) == OK and quantize(lib, cols=0, ldx=0, ldq=0, ldqk=0, **none) == OK
    assert quantize(lib, rows=0, ks=[0, 0], **none) == OK
    assert quantize(lib, rows=0, ks=[128], **none) == LAYOUT      # (the sizes are checked all the same)
    assert blocks(lib, batch=0, x=None, q=None, sf=None, sft=None) == OK
    assert schulz(lib, batch=0, g=None, out=None, ws=None, bytes=0) == OK


def test_newton_schulz_tiles_and_steps(lib):
    """The finished tiles of a call are counted in 31 bits: 6 a step and tile of 256 x 64."""
    one = dict(batch=4096, rows=1, cols=2 ** 20, ldg=2 ** 20, gb=2 ** 20, ldo=2 ** 20, ob=2 ** 20, ws=128, bytes=2 ** 50)
    assert schulz(lib, steps=6, **one) == UNSUPPORTED                  # 6 * 6 * 4096 * 2^14 tiles: 2.4e9
    assert schulz(lib, steps=5, **{**one, "ws": 64}) == ALIGN          # 2.0e9: refused for its workspace alone
    assert schulz(lib, steps=1000, rows=4096, cols=4096, ldg=4096, ldo=4096, gb=2 ** 24, ob=2 ** 24, bytes=2 ** 50,
                  ws=64) == ALIGN
    tall = dict(one, rows=2 ** 20, cols=1, ldg=8, ldo=8, gb=2 ** 23, ob=2 ** 23)
    assert schulz(lib, steps=6, **tall) == UNSUPPORTED and schulz(lib, steps=5, **{**tall, "ws": 64}) == ALIGN


def f8(*s):
    return torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)


def test_binding_checks():
    x, i32 = torch.zeros(128, 256), torch.int32

    def w(*s):
        return torch.zeros(*s, dtype=i32)
    good = dict(q=f8(128, 256), sf=w(1, 128))
    for kw in (dict(q=None), dict(q=f8(128, 128)), dict(q=torch.zeros(128, 256)), dict(sf=w(1, 64)), dict(sf=None),
               dict(qk=f8(128, 256), sfk=w(1, 128)), dict(qk=f8(128, 256), sfk=w(2, 256), ks=[128]),
               dict(qk=f8(128, 256), sfk=w(1, 256), ks=[100]), dict()):      # (the last: CPU tensors)
        with pytest.raises((AssertionError, TypeError, AttributeError)):
            binding.dg_quantize_fp8(x, **{**good, **kw})
    for bad in (x.half(), x[:, ::2], x[0]):
        with pytest.raises((AssertionError, ValueError)):
            binding.dg_quantize_fp8(bad, **good)
    for kw in (dict(), dict(sf=w(2, 1, 64)), dict(sft=w(2, 1, 128)), dict(sf=w(2, 1, 128))):
        with pytest.raises(AssertionError):
            binding.dg_quantize_fp8_blocks(torch.zeros(2, 128, 256), f8(2, 128, 256), **kw)
    o = torch.zeros(128, 256, dtype=torch.bfloat16)
    for args, kw in (((x, o.float()), {}), ((x, o[:64]), {}), ((x.double(), o), {}), ((x[None], o), {}), ((x, o), {}),
                     ((x, o), dict(workspace=torch.zeros(4, 4)[:, ::2])), ((x, o), dict(status=torch.zeros(1)))):
        with pytest.raises(AssertionError):
            binding.dg_newton_schulz(*args, **kw)


def test_refused_sizes_make_no_workspace():
    """What the library refuses by its sizes is its own error, on tensors of any place."""
    x, o = torch.zeros(4, 4), torch.zeros(4, 4, dtype=torch.bfloat16)
    for kw in (dict(steps=0), dict(eps=-1.0), dict(steps=1001)):
        with pytest.raises(binding.DGError):
            binding.dg_newton_schulz(x, o, **kw)
