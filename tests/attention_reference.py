"""Plain 64-bit implementations of an attention layer's operators, written from
their formulas on the CPU, with bounds of what the library's arithmetic may differ.

u = 2^-24 is a rounding to fp32, t = 2^-23 a step of a tensor core's accumulator
(which truncates), h = 2^-8 a rounding to bf16, each relative to the value.

rope. The norm is within (D + 8) u of its value (a sum of D squares, then a mean, a
sum, a root, a quotient and two products). A turned element is a sum of two
products of such values with a cosine and a sine that are within 2^-24 of a turn
(2 pi 2^-24 radians) and 4 u: the error is at most ((D + 16) u + 8 * 2^-24) (|a| + |b|).
The result is rounded once.

attend. A score is a sum of D products in at most D accumulator steps, scaled and
multiplied by log2(e): within ((D + 4) t) S, S the largest sum |q k| |scale| of the row.
It enters as a power of two with that much absolute error (times ln 2 log2(e) = 1), as do the
maximum and the joining of parts, so a weight is within e = (D + 16) t S + 16 u of its value
relatively. Weighted values pass at most L accumulator steps and the weights' rounding w
(2^-8 where prompts are computed, 2^-15 for a few tokens, which keep 16 bits), the total
likewise without it. With A = sum p |v| / sum p:

    |out - y| <= (2 e + w + (L + 64) t) A + h |y|,      |lse - z| <= e + (L + 64) t.
"""

from __future__ import annotations

import math

import numpy as np
import torch

U, T, H = 2.0 ** -24, 2.0 ** -23, 2.0 ** -8


def norm(x, w, eps, one):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + one)


def turn(x, angle, neighbours):
    """x [.., D], angle [.., rot / 2]."""
    half = angle.shape[-1]
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        c, s = np.cos(angle[..., i]), np.sin(angle[..., i])
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def rope(x, q_norm, k_norm, positions, inv_freq, axis, heads, kv_heads, eps, one, neighbours):
    """x [T, heads + 2 kv_heads, D] -> queries, keys, values and the bound of each before its rounding."""
    Tn, _, D = x.shape
    axis = np.zeros(len(inv_freq), int) if axis is None else np.minimum(axis, len(positions) - 1)
    angle = positions[axis].T.astype(np.float64) * inv_freq  # [T, rot / 2]
    out, err = [], []
    for lo, hi, w in ((0, heads, q_norm), (heads, heads + kv_heads, k_norm)):
        part = x[:, lo:hi]
        if w is not None:
            part = norm(part, w, eps, one)
        y = turn(part, angle[:, None, :], neighbours) if len(inv_freq) else part.copy()
        big = np.abs(part).max(-1, keepdims=True) * 2 if len(inv_freq) else np.abs(part)
        out.append(y)
        err.append(((D + 16) * U + 8 * 2.0 ** -24) * big + H * np.abs(y))
    out.append(x[:, heads + kv_heads:])
    err.append(H * np.abs(out[-1]))
    return out, err


def attend(q, k_cache, v_cache, table, q_start, kv_len, kv_heads, scale, window=0, sinks=0, max_new=None, few=16):
    """q [T, heads, D], caches [pages, page_size, kv_heads, D] as float64 tensors; out, lse (nan where no row is
    written) and their bounds."""
    Tn, heads, D = q.shape
    pages, P = k_cache.shape[:2]
    G = heads // kv_heads
    out = torch.full((Tn, heads, D), math.nan, dtype=torch.float64)
    lse = torch.full((Tn, heads), math.nan, dtype=torch.float64)
    oerr, lerr = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        L = min(max(int(kv_len[b]), 0), len(table[b]) * P)
        key = torch.arange(L)
        page = torch.as_tensor(table[b], dtype=torch.int64)[key // P] if L else key
        there = (page >= 0) & (page < pages)
        page = page.clamp(0, pages - 1)
        k, v = (c[page, key % P] for c in (k_cache, v_cache))  # [L, kv_heads, D]
        for i in range(min(n, max_new or n)):
            pos, t = L - n + i, q_start[b] + i
            seen = there & (key <= pos)
            if window:
                seen = seen & ((key > pos - window) | (key < sinks))
            at = seen.nonzero().flatten()
            if not len(at):
                out[t], lse[t] = 0.0, -math.inf
                continue
            kk, vv = k[at].repeat_interleave(G, 1), v[at].repeat_interleave(G, 1)  # [l, heads, D]
            s = torch.einsum("hd,lhd->hl", q[t], kk) * scale
            S = (torch.einsum("hd,lhd->hl", q[t].abs(), kk.abs()) * abs(scale)).amax(-1)
            lse[t] = torch.logsumexp(s, -1)
            w = torch.exp(s - lse[t][:, None])
            out[t] = torch.einsum("hl,lhd->hd", w, vv)
            A = torch.einsum("hl,lhd->hd", w, vv.abs())
            e = (D + 16) * T * S + 16 * U
            steps = (len(at) + 64) * T
            oerr[t] = (2 * e + steps + (2.0 ** -15 if n <= few else 2.0 ** -8))[:, None] * A + H * out[t].abs()
            lerr[t] = e + steps + 4 * U * lse[t].abs()
    return out, lse, oerr, lerr
