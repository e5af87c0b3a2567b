"""The tiles and groups that Newton-Schulz calls choose, as DG_DEBUG_PRINT_CONFIGS prints them, and that batches
in two groups, of equal and unequal numbers and in more than one width of tile, give the bits of single calls."""
import re

import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture
def printed(capfd):
    def call(*args, **kw):
        capfd.readouterr()
        dg.set_debug_flags(dg.DG_DEBUG_PRINT_CONFIGS)
        try:
            dg.dg_newton_schulz(*args, **kw)
        finally:
            dg.set_debug_flags(0)
        lines = [t for t in capfd.readouterr().err.splitlines() if t.startswith("[dg] newton-schulz")]
        assert len(lines) == 1
        v = [int(x) for x in re.findall(r"\d+", lines[0])]
        return dict(zip(("batch", "rows", "cols", "block_m", "sym", "update", "first", "second", "stages", "grid"), v))
    return call


def test_printed_as_recorded(printed):
    g = torch.randn(3, 250, 1000, device="cuda")
    v = printed(g, torch.empty(3, 250, 1000, dtype=torch.bfloat16, device="cuda"), steps=1)
    last = dg.last_config()
    assert (v["batch"], v["rows"], v["cols"], v["first"] + v["second"]) == (3, 250, 1000, 3)
    assert (v["block_m"], v["update"], v["stages"], v["grid"]) == tuple(last[n] for n in ("block_m", "block_n", "stages", "grid"))


def test_two_groups_are_chosen_and_leave_the_bits(printed):
    equal, unequal, widths = 0, 0, set()
    for b, r, c in ((9, 1024, 2064), (10, 1024, 2064), (4, 1024, 1024), (6, 1024, 1024), (2, 2112, 1536), (5, 1536, 1536),
                    (3, 2048, 2048), (61, 166, 773), (40, 387, 1262)):
        g = torch.randn(b, r, c, generator=torch.Generator().manual_seed(b + r)).cuda()
        out, one = (torch.empty(*s, r, c, dtype=torch.bfloat16, device="cuda") for s in ((b,), ()))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        v = printed(g, out, steps=2, status=status)
        if v["second"]:
            equal += v["first"] == v["second"]
            unequal += v["first"] != v["second"]
            widths.add((v["sym"], v["update"]))
        for j in (range(b) if b <= 10 else (0, 1, b // 2, b // 2 + 1, b - 1)):
            assert printed(g[j], one, steps=2, status=status)["second"] == 0
            assert torch.equal(one, out[j]), (b, r, c, j)
        assert int(status) == 0
    assert equal and unequal and len(widths) >= 3
