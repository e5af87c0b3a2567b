"""The gated forward pass in narrow tiles, whose CTA pairs exchange scales over a cluster, where a cluster
takes several tiles: experts of one block of 128 rows each, so that there are twice as many tiles as
the rows alone suggest (on as many SMs as make the call choose tiles of 64 and of 128 columns).  Codes, scale words, gate and up are the bits of dense calls, a cluster's one tile each."""
import pytest
import torch

from block_scaled_fp8_gb300 import binding as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _codes(g, *s):
    return torch.randn(*s, generator=g).to(torch.float8_e4m3fn).cuda()


def _words(g, *s):
    return torch.randint(124, 130, (*s, 4), generator=g, dtype=torch.uint8).view(torch.int32).view(*s).cuda()


def _outputs(m, i):
    return (torch.full((m, i), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
            torch.full(((i + 511) // 512, m), -1, dtype=torch.int32, device="cuda"),
            torch.full((m, 2 * i), 9.0, dtype=torch.bfloat16, device="cuda"))


@pytest.fixture
def sms():
    yield dg.set_num_sms
    dg.set_num_sms(0)


@pytest.mark.parametrize("e,i,k,skipped,limit,columns", [
    (8, 512, 256, (), 64, 128), (16, 512, 256, (), 0, 128), (8, 528, 640, (2, 3), 96, 128),
    (16, 384, 1024, (0, 5, 15), 96, 128), (8, 256, 256, (), 64, 64), (8, 208, 1152, (1,), 64, 64)])
def test_several_tiles_a_cluster(e, i, k, skipped, limit, columns, sms):
    sms(limit)
    g = torch.Generator().manual_seed(e + i + k)
    m = 128 * e
    x, sfx = _codes(g, m, k), _words(g, (k + 511) // 512, m)
    w1, sf1 = _codes(g, e, 2 * i, k), _words(g, e, (k + 511) // 512, 2 * i)
    which = torch.arange(e, dtype=torch.int32)
    which[list(skipped)] = -1
    layout = which.repeat_interleave(128).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _outputs(m, i)
    for j in range(e):
        if j in skipped:
            continue
        r = slice(128 * j, 128 * j + 128)
        hq, sfh, gu = _outputs(128, i)
        dg.dg_fp8_gated_gemm_nt(x[r], sfx[:, r].contiguous(), w1[j], sf1[j], hq=hq, sfh=sfh, gu=gu, status=status)
        cfg = dg.last_config()
        assert (i + 127) // 128 == cfg["grid"] // (512 // cfg["block_n"])     # (every cluster has one tile)
        want[0][r], want[1][:, r], want[2][r] = hq, sfh, gu
    for _ in range(20):
        got = _outputs(m, i)
        dg.dg_m_grouped_fp8_gated_gemm_nt_contiguous(x, sfx, w1, sf1, layout, hq=got[0], sfh=got[1], gu=got[2],
                                                     status=status)
        cfg = dg.last_config()
        tiles, clusters = (e - len(skipped)) * ((i + 127) // 128), cfg["grid"] // (512 // cfg["block_n"])
        assert cfg["block_n"] == columns and tiles > clusters
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(status) == 0
