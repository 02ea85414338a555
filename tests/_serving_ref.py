"""Plain 64-bit forms of the operators over caller-held caches, and the bounds that a
kernel with fp32 scores and sums, and products of rounded parts, has to keep."""
from __future__ import annotations

import math

import numpy as np
import torch


def quantise_rows(x: np.ndarray):
    """fp32 rows -> (int8 codes, fp32 scales) by the definition in qd.h."""
    x = np.asarray(x, np.float32)
    bits = np.abs(x).view(np.uint32).max(-1)
    top = bits.view(np.float32)
    bad = bits >= 0x7F800000
    tiny = bits < np.array(2.0 ** -116, np.float32).view(np.uint32)
    safe = np.where(bad | tiny, np.float32(1), top).astype(np.float32)
    scale = np.where(bad, np.float32(np.nan), np.where(tiny, np.float32(0), safe / np.float32(127)))
    by = np.float32(127) / safe
    with np.errstate(invalid="ignore"):
        codes = np.rint(x * by[..., None])
    codes = np.where((bad | tiny)[..., None], 0, codes).astype(np.int8)
    return codes, scale.astype(np.float32)


def attend(q, k, v, lengths, n_new, scale, pk=None, pv=None):
    """q [B, T, QH, D]; k, v [B, H, S, D] (values, 64 bit); returns (out, mag, spread): the result, sum p |v| / sum p (its
    last axis one longer: the largest p max|v| of a position / sum p) and the largest sum |q k| scale of a row, for the bounds.  Rows t >= n_new[b] are NaN."""
    B, T, QH, D = q.shape
    H = k.shape[1]
    G = QH // H
    q = q.double()
    out = torch.full((B, T, QH, D), math.nan, dtype=torch.float64)
    mag, spread = torch.zeros((B, T, QH, D + 1), dtype=torch.float64), torch.zeros((B, T, QH, 1), dtype=torch.float64)
    P = 0 if pk is None else pk.shape[1]
    for b in range(B):
        for t in range(n_new[b]):
            n = max(0, lengths[b] - (n_new[b] - 1 - t))
            for h in range(QH):
                kk, vv = k[b, h // G, :n], v[b, h // G, :n]
                if P:
                    kk, vv = torch.cat([pk[h // G], kk]), torch.cat([pv[h // G], vv])
                if kk.shape[0] == 0:
                    out[b, t, h] = 0.0
                    continue
                s = kk @ q[b, t, h] * scale
                p = torch.exp(s - s.max())
                out[b, t, h] = (p @ vv) / p.sum()
                mag[b, t, h, :D] = (p @ vv.abs()) / p.sum()
                mag[b, t, h, D] = (p * vv.abs().amax(1)).max() / p.sum()
                spread[b, t, h] = (kk.abs() @ q[b, t, h].abs()).max() * abs(scale)
    return out, mag, spread


def attend_bound(out, mag, spread, n, D, dtype, q8, wide=False):
    """How far a result may be from `out`:

    - the output's rounding, half a step;
    - each probability's rounding, twice (it stands in both sums, or in one of them): parts of fp16
      (half a step 2^-11 a part, 8-bit cache) or bf16 (2^-8 a part, bf16 cache: two parts for bf16 rows, or
      one where `wide`: many rows over a prefix);
    - q's parts and the fp32 sum of D products in the score (2^-23 a product, for a truncating adder), e-fold in p,
      in numerator and denominator; 4 more roundings for the scale factors, and the argument's
      own rounding is a part of the same;
    - 2^-21 for the exponential (2^-22) and the logarithm of the scale's side, and n + 64 additions of 2^-23;
    - 8-bit cache: the weights p_j s_j (s_j the row's scale) go into the product as fp16 numbers, the largest
      at 2^10 or above, so the spacing 2^-24 of fp16's smallest numbers costs each of them up to 2^-25, which is
      2^-35 of the largest.  Times codes of at most 127 and n positions: n 2^-35 max(p_j s_j 127) / sum p, and
      s_j 127 is the row's largest |v|.  Where the heavy positions hold zeros this is all that is left of an element.
      `wide` sets the largest at 2^2 or above: 2^-27."""
    mag, top = mag[..., :D], mag[..., D:]
    bf16 = dtype == torch.bfloat16
    step = torch.finfo(dtype).eps / 2
    if q8:
        part_p, part_q = (2.0 ** -11, 0.0) if bf16 else (2.0 ** -22, 2.0 ** -22)
    else:
        part_p, part_q = (2.0 ** (-8 if wide else -16), 0.0) if bf16 else (2.0 ** -24, 2.0 ** -24)
    ds = spread * (part_q + (D + 8) * 2.0 ** -23)
    rel = 2 * part_p + 2 * torch.expm1(2 * ds) + 2.0 ** -20 + 2 * (n + 64) * 2.0 ** -23
    floor = n * 2.0 ** (-27 if wide else -35) * top if q8 else 0.0
    return step * (out.abs() + mag * rel) + mag * rel + floor * 1.01 + 1e-30


def verify(p, ids, u, q=None, n_draft=None):
    """Whole-number reference of qd_verify_drafts on host arrays."""
    B, T = ids.shape
    V = p.shape[2]
    out, passed = np.full((B, T + 1), -1, np.int32), np.zeros(B, np.int32)

    def whole(w):
        w = np.nan_to_num(np.asarray(w, np.float32), nan=0.0, posinf=1.0, neginf=0.0)
        return np.floor(np.clip(w, 0, 1).astype(np.float64) * 2.0 ** 44).astype(np.uint64)

    for b in range(B):
        n = T if n_draft is None else min(max(int(n_draft[b]), 0), T)
        a = 0
        while a < n:
            x = int(ids[b, a])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(q[b, a, x])
            if not float(u[b, a]) * qx < float(p[b, a, x]):
                break
            out[b, a] = x
            a += 1
        passed[b] = a
        w = p[b, a].copy()
        if a < n:
            if q is not None:
                with np.errstate(invalid="ignore"):
                    w = w - q[b, a]
            elif 0 <= ids[b, a] < V:
                w[ids[b, a]] = 0
        w = whole(w)
        if w.sum() == 0:
            w = whole(p[b, a])
        total = int(w.sum())
        if total:
            mark = math.floor(float(u[b, T]) * float(total))
            out[b, a] = int(np.searchsorted(np.cumsum(w), np.uint64(mark), side="right"))
    return out, passed
