"""One training step of a gated feed-forward block on FP8 operands, captured in a CUDA graph.

    codes and scales of x, W1, W2          dg_quantize_fp8, dg_quantize_fp8_blocks
    h  = silu(x Wg^T) * (x Wu^T)           dg_fp8_gated_gemm_nt           (quantised; gate and up kept)
    y  = h W2^T                            dg_fp8_gemm_nt
    d(gate, up), h again                   dg_fp8_gated_gemm_nn_backward  (from dy and W2)
    dx = d(gate, up) W1                    dg_fp8_gemm_nn
    dW1 = d(gate, up)^T x, dW2 = dy^T h    dg_k_grouped_fp8_gemm_tn_contiguous (FP32)
    W -= lr * update(dW)                   dg_newton_schulz               (gate, up and down each)

Run from the repository's root: python examples/ffn_training.py [--rows 1024] [--hidden 2048] ...
The values are random; the gradients are compared with those of the step in FP64 without quantisation.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp8_gb300 import binding as dg  # noqa: E402


def codes(*shape):
    return torch.empty(*shape, dtype=torch.float8_e4m3fn, device="cuda")


def words(groups, mn, *lead):
    """Packed scale words: four groups of 128 to a word, rows padded to whole fours."""
    return torch.empty(*lead, (groups + 511) // 512, (mn + 3) // 4 * 4, dtype=torch.int32, device="cuda")


class Block:
    """The weights of one block and the buffers of a step of `rows` rows (whole 128s)."""

    def __init__(self, rows, hidden, inner, lr=0.02, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lr, self.ks = lr, [rows]
        m, k, i = rows, hidden, inner
        f32, bf16 = dict(device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        self.w1 = torch.randn(2 * i, k, generator=gen, **f32) * k ** -0.5
        self.w2 = torch.randn(k, i, generator=gen, **f32) * i ** -0.5
        self.x = torch.randn(m, k, generator=gen, **f32).bfloat16()
        self.dy = (1e-3 * torch.randn(m, k, generator=gen, **f32)).bfloat16()
        # operands along their columns (q) and along their rows (k)
        self.w1q, self.w1s, self.w1t = codes(2 * i, k), words(k, 2 * i), words(2 * i, k)
        self.w2q, self.w2s, self.w2t = codes(k, i), words(i, k), words(k, i)
        self.xq, self.xs, self.xk, self.xt = codes(m, k), words(k, m), codes(m, k), words(m, k)
        self.yq, self.ys, self.yk, self.yt = codes(m, k), words(k, m), codes(m, k), words(m, k)
        self.gq, self.gs, self.gk, self.gt = codes(m, 2 * i), words(2 * i, m), codes(m, 2 * i), words(m, 2 * i)
        self.hq, self.hs, self.hk, self.ht = codes(m, i), words(i, m), codes(m, i), words(m, i)
        self.gu, self.dgu, self.h = torch.empty(m, 2 * i, **bf16), torch.empty(m, 2 * i, **bf16), torch.empty(m, i, **bf16)
        self.y, self.dx = torch.empty(m, k, **bf16), torch.empty(m, k, **bf16)
        self.dw1, self.dw2 = torch.empty(1, 2 * i, k, **f32), torch.empty(1, k, i, **f32)
        self.up1, self.up2 = torch.empty(2, i, k, **bf16), torch.empty(k, i, **bf16)
        self.ks_dev = torch.tensor(self.ks, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # one workspace serves both updates, which run one after another
        need = max(dg.newton_schulz_workspace_bytes(2, i, k), dg.newton_schulz_workspace_bytes(1, k, i))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(self):
        s, st = self, dict(status=self.status)
        dg.dg_quantize_fp8_blocks(s.w1, s.w1q, sf=s.w1s, sft=s.w1t)
        dg.dg_quantize_fp8_blocks(s.w2, s.w2q, sf=s.w2s, sft=s.w2t)
        dg.dg_quantize_fp8(s.x, q=s.xq, sf=s.xs, qk=s.xk, sfk=s.xt)
        dg.dg_fp8_gated_gemm_nt(s.xq, s.xs, s.w1q, s.w1s, hq=s.hq, sfh=s.hs, gu=s.gu, **st)
        dg.dg_fp8_gemm_nt(s.hq, s.hs, s.w2q, s.w2s, s.y, **st)
        dg.dg_quantize_fp8(s.dy, q=s.yq, sf=s.ys, qk=s.yk, sfk=s.yt)
        dg.dg_fp8_gated_gemm_nn_backward(s.yq, s.ys, s.w2q, s.w2t, s.gu, s.dgu, h=s.h, **st)
        dg.dg_quantize_fp8(s.dgu, q=s.gq, sf=s.gs, qk=s.gk, sfk=s.gt)
        dg.dg_quantize_fp8(s.h, qk=s.hk, sfk=s.ht)
        dg.dg_fp8_gemm_nn(s.gq, s.gs, s.w1q, s.w1t, s.dx, **st)
        s.dw1.zero_()
        s.dw2.zero_()
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(s.gk, s.gt, s.xk, s.xt, s.dw1, s.ks, ks_dev=s.ks_dev, c=s.dw1, **st)
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(s.yk, s.yt, s.hk, s.ht, s.dw2, s.ks, ks_dev=s.ks_dev, c=s.dw2, **st)
        dg.dg_newton_schulz(s.dw1.view(s.up1.shape), s.up1, workspace=s.workspace, **st)
        dg.dg_newton_schulz(s.dw2[0], s.up2, workspace=s.workspace, **st)
        s.w1.sub_(s.up1.view(s.w1.shape), alpha=s.lr)
        s.w2.sub_(s.up2, alpha=s.lr)

    def plain(self):
        """y and the gradients of x, W1 and W2 in FP64, with the weights as they are now."""
        x, dy, w1, w2 = (t.double() for t in (self.x, self.dy, self.w1, self.w2))
        g, u = (x @ w1.t()).chunk(2, 1)
        s = torch.sigmoid(g)
        h, dh = g * s * u, dy @ w2
        dgu = torch.cat((dh * u * (s + g * s * (1 - s)), dh * g * s), 1)
        return h @ w2.t(), dgu @ w1, dgu.t() @ x, dy.t() @ h


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1408)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    if a.rows < 1 or a.rows % 128 or a.hidden % 16 or a.inner % 16:
        p.error("rows: whole 128s (the weight gradient's groups); hidden, inner: whole 16s")
    block = Block(a.rows, a.hidden, a.inner, seed=a.seed)
    want = block.plain()
    block.step()
    torch.cuda.synchronize()
    assert int(block.status.item()) == 0, f"device status {int(block.status.item())}"
    got = (block.y, block.dx, block.dw1[0], block.dw2[0])
    errors = [float((g.double() - w).norm() / w.norm()) for g, w in zip(got, want)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step()
    graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert int(block.status.item()) == 0, f"device status {int(block.status.item())}"
    print(f"{a.rows} rows, {a.hidden} x {a.inner}: {begin.elapsed_time(end) / 20 * 1e3:.1f} us a step; error beside the "
          "step in FP64: " + ", ".join(f"{n} {e:.3f}" for n, e in zip(("y", "dx", "dW1", "dW2"), errors)))
    return errors


if __name__ == "__main__":
    main()
