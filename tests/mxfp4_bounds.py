"""A bound on the error of the 4-bit attention that goes by what a row's keys contribute,
weight times value, and not by the values alone."""

from __future__ import annotations

import numpy as np
import torch

from oracle import mxfp4


def _scales(step, r):
    """Exponents e - 127 of the V scales of request r, [keys, KV heads, groups]; NaN: -1000."""
    slots, d = step.slots[r], step.d
    e = np.empty((len(slots), step.hkv, d // 32))
    for b in range(d // 32):
        place = np.array([mxfp4.scale_place(t, b, d, False) for t in range(16)])
        for h in range(step.hkv):
            e[:, h, b] = step.pools.v[slots // 16, place[slots % 16] + h * mxfp4.chunk_bytes(d)]
    return torch.from_numpy(np.where(e == 255, -1000.0, e - 127.0))


def _decode_floor(p, v, e):
    """Of one row: p [H, n] weights that sum to one, v [n, D], e [n, D / 32] -> [H, D].

    Weights are f16 with the largest at 2^11 or above, so one is off by 2^-36 of the largest
    where it is below f16's normal numbers (2^-25 of a step of 2^-24, halved).  A scale
    multiplies them by 2^(e - base - 14), rounded once more at 2^-25, base at or below every
    scale of the 32 tokens and 11 below some scale of the request's: together
      2^-25 pmax |code| (2^(base + 3) + 2^(e - 11)).
    16 tokens whose scales are more than 15 apart go another way, without a floor above 2^-100
    of their largest product of weight and scale."""
    n, nb = e.shape
    pmax = p.amax(1)
    floor = torch.zeros(p.shape[0], v.shape[1], dtype=torch.float64)
    top = e.amax(0)
    for b in range(nb):
        cols = slice(32 * b, 32 * b + 32)
        below = float(top[b]) - 11 if float(top[b] - e[:, b].amin()) < 60 else float("inf")
        for j in range(0, n, 16):
            eb, vb = e[j:j + 16, b], v[j:j + 16, cols].abs()
            if float(eb.amax() - eb.amin()) <= 15:
                base = torch.minimum(eb, torch.full_like(eb, below))
                each = 2.0 ** -25 * (torch.exp2(base - eb + 3) + 2.0 ** -11)
                floor[:, cols] += pmax[:, None] * (each[:, None] * vb).sum(0)
            else:
                most = (p[:, j:j + 16] * torch.exp2(eb)).amax(1)
                floor[:, cols] += 2.0 ** -100 * most[:, None] * (vb * torch.exp2(-eb)[:, None]).sum(0)
    return floor


def _prefill_floor(p, v, e):
    """The same of a prefill row.  With x = weight times the largest scale of a key's groups:
    weights are f16 with 2 or more for the largest x so far, off by 2^-25 each below f16's
    normal numbers, over a base that keys share, up to 2^8 above a key's own scale (up to 2^14
    with 2^8 or more for the largest x: 2^7 from x either way).  A row that sees a key whose
    groups (those with a code that is not zero) are more than 2^8 apart has weights of two
    bfloat16, without a floor."""
    most = e.amax(1)
    some = (v.nan_to_num(0.0).unflatten(1, (-1, 32)).abs().amax(2) > 0) & (e > -500)
    apart = torch.where(some, e, -1000.0).amax(1) - torch.where(some, e, 1000.0).amin(1)
    floor = torch.zeros(p.shape[0], v.shape[1], dtype=torch.float64)
    if bool((apart > 8).any()):
        return floor
    x = p * torch.exp2(most)
    so_far = torch.zeros(p.shape[0], dtype=torch.float64)
    for j in range(0, e.shape[0], 128):
        m, keys = most[j:j + 128], slice(j, j + 128)
        so_far = torch.maximum(so_far, x[:, keys].amax(1))
        floor += 2.0 ** -18 * so_far[:, None] * (v[keys].abs() * torch.exp2(-m)[:, None]).sum(0)
    return floor


def reference(step):
    """(float64 output, bound) per row of a step.  With p the weights, u = 2^-24, S the sum
    scale |q| |k| of a row's worst key, A = sum p |v|:
      score: D products and a few scalings in float32, u S each; a weight is off by
        2 (D + 32) u S of itself, numerator and denominator;
      weight: f16 twice, or a pair of bfloat16, 2^-11 of A (and an exponential, 2^-21);
        what is below f16's normal numbers: the floors above, and 2^-100 of the row's
        largest weight times scale for each key;
      sums: 2 n u A of n keys;
      the result: 2^-8 of it, or 2^-134."""
    ref = torch.zeros(step.T, step.H, step.d, dtype=torch.float64)
    tol = torch.zeros_like(ref)
    G, u = step.H // step.hkv, 2.0 ** -24
    for r in range(step.R):
        a, rows = int(step.qsl[r]), step.q_len[r]
        if rows == 0:
            continue
        k, v = step.history(r)
        e = _scales(step, r)
        for i in range(rows):
            n = step.past[r] + i + 1
            for g in range(step.hkv):
                heads = slice(g * G, g * G + G)
                q, kg, vg = step.q[a + i, heads].double(), k[:n, g], v[:n, g]
                p = torch.softmax(q @ kg.T * step.scale, 1)
                worst = (q.abs() @ kg.abs().T * abs(step.scale)).amax(1, keepdim=True)
                floor = (_decode_floor if rows == 1 else _prefill_floor)(p, vg, e[:n, g])
                # of products 2^100 below the row's largest nothing is kept
                most = (p * torch.exp2(e[:n, g].amax(1))).amax(1, keepdim=True)
                floor = floor + 2.0 ** -100 * most * 6 * n
                out = p @ vg
                ref[a + i, heads] = out
                tol[a + i, heads] = (2.0 ** -8 * out.abs() + 2.0 ** -134 + floor + (p @ vg.abs()) * (
                    2.0 ** -11 + 2.0 ** -20 + 4 * (step.d + 32) * u * worst + 2 * n * u))
    return ref, tol


def check(got, ref, tol, tight=0.75):
    """got is within the bound, and the bound is one that zeros and twice the result break
    (in the given part of the elements)."""
    assert (tol < ref.abs() / 4).double().mean() >= tight
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    at = np.unravel_index(int(over.argmax()), tuple(over.shape))
    assert over[at] <= 0, (at, float(got[at]), float(ref[at]), float(tol[at]))
