"""Plain 64-bit forms of the softmax-attention operators, and the error bounds of the kernels' arithmetic."""
from __future__ import annotations

import math

import torch

# Half a unit in the last place of 1: the relative error of one rounding.
ROUNDING = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FP32 = 2.0 ** -24


def rope_tables(positions, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def pair_index(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(z, cos, sin, interleaved):
    """z [rows, heads, d] turned by the angles cos, sin [rows, rot/2] (None: not at all)."""
    if cos is None:
        return z
    one, two = pair_index(2 * cos.shape[1], interleaved)
    c, s = cos.to(z.dtype)[:, None], sin.to(z.dtype)[:, None]
    y = z.clone()
    y[..., one] = z[..., one] * c - z[..., two] * s
    y[..., two] = z[..., two] * c + z[..., one] * s
    return y


def norm_rope(x, w, cos, sin, eps, interleaved, normed=True):
    """x [rows, heads, d] in 64 bits."""
    z = x
    if normed:
        z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            z = z * w.double()
    return rotate(z, cos, sin, interleaved)


def norm_rope_backward(x, dy, w, cos, sin, eps, interleaved):
    """The formula: dz = R^T dy, dw = sum dz x r, dx = r (t - x r^2 mean(t x)) with t = dz w; also the sum of
    |dz x r| and the size of dx's terms, for the error bounds."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dz = rotate(dy, cos, None if sin is None else -sin, interleaved)
    t = dz if w is None else dz * w.double()
    dx = r * (t - x * r * r * (t * x).mean(-1, keepdim=True))
    terms = dz * x * r
    size = r * (t.abs() + x.abs() * r * r * (t * x).abs().mean(-1, keepdim=True))
    if cos is not None:  # a rotated value is the difference of two
        both = rotate_sizes(dy, cos.shape[1] * 2, interleaved)
        ww = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double().abs()
        size = size + r * both * ww
    return dx, terms.sum((0, 1)), terms.abs().sum((0, 1)), size


def rotate_sizes(z, rot, interleaved):
    """|z_i| + |z_j| over each pair: what rounding errors of a rotated value scale with."""
    one, two = pair_index(rot, interleaved)
    y = z.abs().clone()
    y[..., one] = z[..., one].abs() + z[..., two].abs()
    y[..., two] = y[..., one]
    return y


def sees(ctx, n, mask, i):
    """Which of a sequence's ctx + n tokens its new row i sees; mask: bool [n, n] or None (up to itself)."""
    v = torch.zeros(ctx + n, dtype=torch.bool)
    v[:ctx] = True
    v[ctx:] = torch.arange(n) <= i if mask is None else mask[i]
    return v


def attention(q, k, v, ctx, mask, scale):
    """One sequence: q [n, nq, d], k, v [ctx + n, nkv, d] in 64 bits. Returns the output and, for every value of
    it, the bound of the error that the kernels may make, as functions of the output type's rounding u:
    (out, spread, slack) with |error| <= u |out| + (u + slack) spread."""
    n, nq, d = q.shape
    nkv = k.shape[1]
    out, spread = torch.zeros(n, nq, d, dtype=torch.float64), torch.zeros(n, nq, d, dtype=torch.float64)
    size = torch.zeros(n, nq, dtype=torch.float64)
    for i in range(n):
        see = sees(ctx, n, mask, i)
        if not bool(see.any()):
            continue
        for h in range(nq):
            kk, vv = k[see, h // (nq // nkv)], v[see, h // (nq // nkv)]
            x = scale * (kk @ q[i, h])
            p = torch.softmax(x, 0)
            out[i, h] = p @ vv
            spread[i, h] = p @ vv.abs()
            # fp32 scores: d products, their sum, the scaling and the exponential's argument
            size[i, h] = abs(scale) * ((d + 4) * (kk.abs() @ q[i, h].abs())).max() + 4 * x.abs().max()
    # the sums over the tokens in fp32, and 2^x to 2^-22
    slack = 2 * FP32 * (size[..., None] + (ctx + n) + 16)
    return out, spread, slack


def attention_bound(out, spread, slack, dtype, tokens, vmax):
    """u for the rounded output, u for the rounded weights; fp16 weights below 2^-14 are off by up to 2^-25 each."""
    u = ROUNDING[dtype]
    bound = u * out.abs() + (u + slack) * spread * (1 + 2 * u)
    if dtype == torch.float16:
        bound = bound + (tokens + 1) * 2.0 ** -25 * vmax + 2.0 ** -25
    return bound + 1e-30


def pack_mask(mask):
    """bool [rows, bits] -> int64 [rows, words]."""
    rows, bits = mask.shape
    words = max(1, math.ceil(bits / 64))
    out = torch.zeros(rows, words, dtype=torch.int64)
    for j in range(bits):
        bit = 1 << (j % 64)
        out[:, j // 64] |= torch.where(mask[:, j], bit - (1 << 64) if bit >= 1 << 63 else bit, 0)
    return out
