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
