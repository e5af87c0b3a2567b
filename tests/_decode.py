"""Plain 64-bit forms of the decode-side operators, and their inputs."""
from __future__ import annotations

import torch

from block_scaled_fp8_gb300 import binding, inputs

MAGS = torch.tensor(inputs.E2M1_MAGNITUDES, dtype=torch.float64)


def quantize(w: torch.Tensor, fmt: str):
    """FP32 weights [N, K] -> (codes, FP32 scales per row and group, group)."""
    if fmt == "fp4":
        codes, s = inputs.quantize_e2m1_1x32(w)
        return codes, s, 32
    codes, s = inputs.quantize_128x128(w)
    return codes, s.repeat_interleave(128, 0)[:w.shape[0]].contiguous(), 128


def dequantize(codes: torch.Tensor, s: torch.Tensor, gran: int) -> torch.Tensor:
    """The weights [N, K] in 64 bits."""
    if codes.dtype == torch.uint8:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        v = MAGS[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    else:
        v = codes.double()
    return v * s.double().repeat_interleave(gran, 1)


def pack_scales(s: torch.Tensor) -> torch.Tensor:
    """FP32 scales [..., N, groups] -> packed words on the device (by the library's transform)."""
    n = s.shape[-2]
    return binding.transform_sf(s.contiguous().cuda(), 1, n)


def padded(t: torch.Tensor, pad: int) -> torch.Tensor:
    """t [R, C] on the device as a view of rows `pad` elements longer."""
    if not pad:
        return t.cuda()
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype).cuda()
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def group_amax(x: torch.Tensor) -> torch.Tensor:
    """|x| replaced by the largest magnitude of its 32 consecutive K."""
    g = x.abs().unflatten(-1, (-1, 32))
    return g.amax(-1, keepdim=True).expand_as(g).flatten(-2)


def product_bound(a: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """Bound of |computed - exact| of a @ w^T before any output rounding, for
    products that are exact and sums of 32 products that lose less than a unit
    in the last place of an FP32 sum no larger than sum |a||w| (K/32 steps, and 16
    for joining partial sums), with activations held to 2^-20 of the largest
    magnitude of their group of 32."""
    k = a.shape[-1]
    s = a.abs() @ w.abs().t()
    return s * (k / 32 + 16) * 2.0 ** -23 + (group_amax(a) @ w.abs().t()) * 2.0 ** -20


def route_plain(logits, bias, topk, scoring, renormalize, scale):
    """(ids, weights, rows whose order 32-bit arithmetic decides alike) in 64 bits."""
    x = logits.double()
    ok = x > float("-inf")
    if scoring == "softmax":
        xs = torch.where(ok, x, float("-inf"))
        top = xs.amax(-1, keepdim=True)
        s = torch.where(ok, torch.exp(x - top), 0.0)
        s = s / s.sum(-1, keepdim=True)
        key = x if bias is None else s + bias.double()
    else:
        s = torch.sigmoid(x)
        key = s if bias is None else s + bias.double()
    key = torch.where(ok, key, float("-inf"))
    val, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    near = val[:, :-1] - val[:, 1:]
    near = near[:, :topk]
    eps = 0.0 if (scoring == "softmax" and bias is None) else 2e-6
    clear = ~((near > 0) & (near < eps)).any(-1)
    val, ids = val[:, :topk], ids[:, :topk]
    empty = val == float("-inf")
    w = torch.where(empty, 0.0, s.gather(-1, ids))
    if renormalize:
        w = w / w.sum(-1, keepdim=True).clamp_min(2.0 ** -126)
    return torch.where(empty, -1, ids).int(), w * scale, clear


def layer_plain(x, ids, weights, w1, w2, c=None):
    """(y, bound of |bf16 y - y|) in 64 bits; w1 [E, 2I, H] and w2 [E, H, I] 64-bit weights.

    The bound: one rounding to bf16 (half a unit, 2^-9 of |y|, and as much for a
    result next to a power of two), h = silu(g) u held to 9 bits in groups of 32 by two
    4-bit pieces (2^-10 of |h|; 2^-20 of the group's largest), FP32 sums, and the
    first product's own bound through silu (slope at most 1.1) and the product."""
    t, h = x.shape
    i = w2.shape[2]
    y = torch.zeros(t, h, dtype=torch.float64)
    tol = torch.zeros_like(y)
    xd = x.double()
    if c is not None:
        y += c.double()
    for r in range(t):
        for j in range(ids.shape[1]):
            e = int(ids[r, j])
            if e < 0 or e >= w1.shape[0]:
                continue
            gu = w1[e] @ xd[r]
            b = product_bound(xd[r:r + 1], w1[e])[0]
            g, u = gu[:i], gu[i:]
            act = torch.nn.functional.silu(g) * u
            dact = 1.1 * b[:i] * u.abs() + torch.nn.functional.silu(g).abs() * b[i:] + 2.0 ** -22 * act.abs()
            w = abs(float(weights[r, j]))
            y[r] += float(weights[r, j]) * (w2[e] @ act)
            a2 = w2[e].abs()
            tol[r] += w * (a2 @ (dact + 2.0 ** -10 * act.abs() + 2.0 ** -20 * group_amax(act[None])[0])
                           + (a2 @ act.abs()) * (i / 32 + 16) * 2.0 ** -23)
    # sums over the experts run on in FP32
    return y, tol * 1.01 + y.abs() * 2.0 ** -8
