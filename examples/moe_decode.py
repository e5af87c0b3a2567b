"""One decode step of a mixture-of-experts block, captured in a CUDA graph.

    logits = x @ router^T              dg_bf16_fp8_gemv_nt_f32  (FP8 weights, FP32 logits)
    ids, w = top-k of sigmoid(logits)  dg_moe_route             (a bias shifts the choice)
    h      = x + sum_e w_e expert_e(x) dg_moe_fp4_layer         (FP4 weights, the residual as C)
    out    = h @ head^T                dg_bf16_fp4_gemv_nt      (FP4 weights)

Run from the repository's root: python examples/moe_decode.py [--tokens 4] [--hidden 2048] ...
The weights are random; the result is compared with the same step in FP64 on the device.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp8_gb300 import binding, inputs  # noqa: E402


def fp4_weights(n, k, gen):
    """Random weights [n, k]: (packed E2M1 codes, packed scales, the weights in FP64), on the device."""
    codes, s = inputs.quantize_e2m1_1x32(torch.randn(n, k, generator=gen) * k ** -0.5)
    mags = torch.tensor(inputs.E2M1_MAGNITUDES, dtype=torch.float64)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    w = mags[c & 7] * torch.where(c >= 8, -1.0, 1.0).double() * s.double().repeat_interleave(32, 1)
    return codes.cuda(), binding.transform_sf(s.cuda(), 1, n), w.cuda()


def fp8_weights(n, k, gen):
    """The same for E4M3 with one scale per 128 x 128."""
    codes, s = inputs.quantize_128x128(torch.randn(n, k, generator=gen) * k ** -0.5)
    rows = s.repeat_interleave(128, 0)[:n].contiguous()
    w = codes.double() * rows.double().repeat_interleave(128, 1)
    return codes.cuda(), binding.transform_sf(rows.cuda(), 1, n), w.cuda()


class Block:
    """The weights of one block and the buffers of a decode step of `tokens` tokens."""

    def __init__(self, tokens, hidden, inner, experts, topk, vocab, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.topk = topk
        self.router, self.router_sf, self.router_64 = fp8_weights(experts, hidden, gen)
        self.bias = 0.1 * torch.randn(experts, generator=gen).cuda()
        up = [fp4_weights(2 * inner, hidden, gen) for _ in range(experts)]
        down = [fp4_weights(hidden, inner, gen) for _ in range(experts)]
        self.w1, self.sf1, self.w1_64 = (torch.stack(v) for v in zip(*up))
        self.w2, self.sf2, self.w2_64 = (torch.stack(v) for v in zip(*down))
        self.head, self.head_sf, self.head_64 = fp4_weights(vocab, hidden, gen)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.x = torch.randn(tokens, hidden, generator=gen).bfloat16().cuda()
        self.logits = torch.empty(tokens, experts, device="cuda")
        self.ids = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
        self.weights = torch.empty(tokens, topk, device="cuda")
        self.h = torch.empty(tokens, hidden, **bf16)
        self.out = torch.empty(tokens, vocab, **bf16)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # one workspace serves the calls of a stream, which run one after another
        need = max(binding.gemv_workspace_bytes(tokens, experts, hidden),
                   binding.gemv_workspace_bytes(tokens, vocab, hidden),
                   binding.moe_layer_workspace_bytes(tokens, topk, hidden, inner, experts))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(self):
        kw = dict(status=self.status, workspace=self.workspace)
        binding.dg_bf16_fp8_gemv_nt_f32(self.x, self.router, self.router_sf, self.logits, **kw)
        binding.dg_moe_route(self.logits, self.ids, self.weights, bias=self.bias, scoring="sigmoid")
        binding.dg_moe_fp4_layer(self.x, self.ids, self.weights, self.w1, self.sf1, self.w2, self.sf2, self.h,
                                 c=self.x, **kw)
        binding.dg_bf16_fp4_gemv_nt(self.h, self.head, self.head_sf, self.out, **kw)
        return self.out

    def plain(self, chosen):
        """The step in FP64 (rounded to bf16 where the step stores bf16) with the experts `chosen` (near
        ties may be chosen in either order), and how far their keys are below the largest ones."""
        x = self.x.double()
        score = torch.sigmoid(x @ self.router_64.t())
        key = score + self.bias.double()
        best, ids = key.topk(self.topk, -1)
        behind = (best - key.gather(1, chosen)).abs().max()
        same = (chosen.sort(-1)[0] == ids.sort(-1)[0]).all(-1)
        ids = chosen
        w = score.gather(1, ids)
        w = w / w.sum(-1, keepdim=True)
        h = x.clone()
        for t in range(x.shape[0]):
            for j in range(self.topk):
                g, u = (x[t] @ self.w1_64[ids[t, j]].t()).chunk(2)
                h[t] += (w[t, j] * torch.nn.functional.silu(g) * u) @ self.w2_64[ids[t, j]].t()
        return same, float(behind), h.bfloat16().double() @ self.head_64.t()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inner", type=int, default=1024)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--vocab", type=int, default=8192)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    if not 1 <= a.tokens <= 64:
        p.error("1 to 64 tokens (more go through the grouped GEMMs)")
    block = Block(a.tokens, a.hidden, a.inner, a.experts, a.topk, a.vocab, a.seed)
    block.step()   # sizes are checked, kernels loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step()
    graph.replay()
    torch.cuda.synchronize()
    assert int(block.status.item()) == 0, f"device status {int(block.status.item())}"
    assert ((block.ids >= 0) & (block.ids < a.experts)).all() and all(len(set(r)) == a.topk for r in block.ids.tolist())
    same, behind, ref = block.plain(block.ids.long())
    # the logits are FP32 sums of some thousand products; a key is a sigmoid (slope 1/4 at most) and a sum
    assert behind <= 1e-4, f"an expert was chosen whose key is {behind} behind"
    err = (block.out.double() - ref).abs().amax(-1) / ref.pow(2).mean(-1).sqrt()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    worst = float(err.max())
    print(f"{a.tokens} tokens, {a.experts} experts top {a.topk}, {a.hidden} x {a.inner}, vocabulary {a.vocab}: "
          f"{begin.elapsed_time(end) / 20 * 1e3:.1f} us a step, {int(same.sum())} of {a.tokens} tokens routed as in "
          f"FP64, largest error {worst:.2e} of the output's RMS")
    return int(same.sum()), worst


if __name__ == "__main__":
    main()
