"""Inputs and 64-bit forms shared by the tests of the feed-forward training operators."""
import torch

from block_scaled_fp8_gb300 import inputs


def cdiv(a, b):
    return (a + b - 1) // b


def exponents(scale):
    """Biased exponents of power-of-two FP32 scales."""
    return (scale.contiguous().view(torch.int32) >> 23) & 255


def pack(exps, mn):
    """[.., groups, mn] exponents -> int32 words [.., ceil(groups/4), align4(mn)]."""
    groups = exps.shape[-2]
    w = torch.zeros(*exps.shape[:-2], cdiv(groups, 4) * 4, cdiv(mn, 4) * 4, dtype=torch.int32)
    w[..., :groups, :mn] = exps
    w = w.unflatten(-2, (-1, 4))
    return (w[..., 0, :] | (w[..., 1, :] << 8) | (w[..., 2, :] << 16) | (w[..., 3, :] << 24)).contiguous()


def rows_operand(x):
    """FP32 [m, k] -> codes, packed words, values in FP64 (a scale for each 1 x 128)."""
    q, s = inputs.quantize_1x128(x)
    values = q.double() * s.double().repeat_interleave(128, 1)[:, :x.shape[1]]
    return q, pack(exponents(s).t(), x.shape[0]), values


def block_operand(w, along_rows=False):
    """FP32 [n, k] -> codes, packed words, values in FP64 (a scale for each 128 x 128); the words
    are for products along k, or along n (the operand's rows)."""
    n, k = w.shape
    q, s = inputs.quantize_128x128(w)
    values = q.double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    if along_rows:
        return q, pack(exponents(s).repeat_interleave(128, 1)[:, :k], k), values
    return q, pack(exponents(s).repeat_interleave(128, 0)[:n].t(), n), values


def scale64(amax):
    """2^ceil(log2(amax / 448)) in FP64, 1 for 0, as the quantiser defines it."""
    mant, e = torch.frexp(amax.double())
    p = e - 9 + (mant > 0.875).int()
    return torch.where(amax == 0, torch.ones_like(mant), torch.ldexp(torch.ones_like(mant), p.clamp(-126, 127)))


def gated64(x, w1):
    """x [m, k], w1 [2i, k] in FP64 -> (gate and up, h)."""
    gu = x @ w1.t()
    g, u = gu.split(w1.shape[0] // 2, 1)
    return gu, torch.nn.functional.silu(g) * u


def gated_backward64(dy, w2, gu):
    """dy [m, k], w2 [k, i], gu [m, 2i] in FP64 -> (gradient of gate and up, h)."""
    dh = dy @ w2
    g, u = gu.split(w2.shape[1], 1)
    s = torch.sigmoid(g)
    return torch.cat((dh * u * (s * (1 + g * (1 - s))), dh * g * s), 1), g * s * u
