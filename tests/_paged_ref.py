"""Plain 64-bit forms of a decoder layer's attention over a cache in pages, and the bounds that kernels with fp32
arithmetic have to keep."""
from __future__ import annotations

import torch


def norm_rope(x, gamma, eps, cos, sin):
    """x [N, heads, D], cos / sin [N, D / 2] or None; returns (y, size): the result in 64 bits and the size of its terms."""
    x = x.double()
    D = x.shape[-1]
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    if cos is None:
        return x, x.abs()
    c, s = cos.double()[:, None], sin.double()[:, None]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return (torch.cat([a * c - b * s, b * c + a * s], -1),
            torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1))


def norm_rope_bound(size, D):
    """How far an fp32 evaluation may be from norm_rope's y: in units of 2^-24 relative to the terms' size, the mean square takes
    D / 8 products and sums a lane and four sums of lanes, D + 8 with room, which the root halves; the mean's quotient,
    eps, the root and its inverse (2 each: not all of them need be rounded to nearest) and the two factors 8 more; a product and the final
    sum 3; 1e-38 for what is flushed or rounded near zero."""
    return size * ((D + 8) / 2 + 8 + 3) * 2.0 ** -24 + 1e-38


def place(lengths, new, page):
    """(stream, page index, row) of every new token, stream after stream."""
    return [(b, (n - k + t) // page, (n - k + t) % page) for b, (n, k) in enumerate(zip(lengths, new)) for t in range(k)]


def prompt(q, k, v, offsets, kv_offsets, scale):
    """Attention over packed prompts in 64 bits, sequence by sequence and key head by key head: (out, mag, noise, spread) with mag = sum p |v| /
    sum p, noise = sqrt(sum p^2 v^2) / sum p and the largest sum |q k| scale of a row.  Rows of no sequence are NaN."""
    N, QH, D = q.shape
    H = k.shape[1]
    out = torch.full((N, QH, D), float("nan"), dtype=torch.float64, device=q.device)
    mag, noise, spread = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out[..., :1])
    for b in range(len(offsets) - 1):
        i0, i1, j0, j1 = offsets[b], offsets[b + 1], kv_offsets[b], kv_offsets[b + 1]
        n, m = i1 - i0, j1 - j0
        if n <= 0:
            continue
        seen = torch.arange(m, device=q.device) < (m - n + 1 + torch.arange(n, device=q.device))[:, None]
        for h in range(H):
            heads = slice(h * (QH // H), (h + 1) * (QH // H))
            x, kk, vv = q[i0:i1, heads].double().transpose(0, 1), k[j0:j1, h].double(), v[j0:j1, h].double()
            s = (x @ kk.T * scale).masked_fill(~seen, float("-inf"))
            top = s.amax(-1, keepdim=True) if m else torch.zeros_like(x[..., :1])
            p = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
            total = p.sum(-1, keepdim=True)
            by = torch.where(total > 0, 1 / total, torch.zeros_like(total))
            out[i0:i1, heads] = (p @ vv * by).transpose(0, 1)
            mag[i0:i1, heads] = (p @ vv.abs() * by).transpose(0, 1)
            noise[i0:i1, heads] = ((p * p) @ (vv * vv)).sqrt().mul(by).transpose(0, 1)
            if m:
                spread[i0:i1, heads] = ((x.abs() @ kk.abs().T).masked_fill(~seen, 0).amax(-1, keepdim=True) * abs(scale)).transpose(0, 1)
    return out, mag, noise, spread


def prompt_bound(out, mag, spread, most, D):
    """How far a result may be from `out`: the output's rounding, half a step of 2^-8; each probability's rounding to bf16, half a step
    (in the product alone: the sum is of the unrounded ones); the fp32 sum of D exact products in the score (2^-23 a product, for a
    truncating adder) and 8 more roundings, e-fold in p, in numerator and denominator; 2^-20 for the exponential and the quotient; and at most
    `most` + 64 additions of 2^-23 in both sums."""
    ds = spread * (D + 8) * 2.0 ** -23
    rel = 2.0 ** -8 + 2 * torch.expm1(2 * ds) + 2.0 ** -20 + 2 * (most + 64) * 2.0 ** -23
    return 2.0 ** -8 * (out.abs() + mag * rel) + mag * rel + 1e-30


def prompt_norm_bound(out, noise):
    """2-norm: rounding errors are at most 2^-8 relative, so 2^-8 / sqrt(3) in the mean where they spread evenly (less where values
    crowd at a step's upper end), and independent from key to key; a tenth of room for chance and the fp32 arithmetic."""
    return 1.1 * 2.0 ** -8 / 3 ** 0.5 * (out.norm() ** 2 + noise.norm() ** 2).sqrt()
