"""Plain 64-bit implementations of the decode-step operators, written from
their formulas on the CPU, with bounds of what fp32 arithmetic may differ.

Bounds (u = 2^-24, the fp32 rounding; t = 2^-23, a tensor core's truncation):
a factored group sum passes at most 10 accumulator steps (t each) and 4
roundings inside the group, then one rounding per group and a few for joining
partial sums, each relative to at most the sum of the magnitudes. A row of G
groups is therefore within  (10 t + (2 G + 32) u) * sum(|s q x| + |b x|).
A bf16 output adds its own rounding, at most 2^-8 of the value.
"""

from __future__ import annotations

import math

import numpy as np
import torch

import synth

U = 2.0 ** -24


def bf(bits: np.ndarray) -> np.ndarray:
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def to_bf16(a) -> np.ndarray:
    """float array -> bf16 bit patterns."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16).copy()


class Matrix:
    """A seeded group-quantized matrix and its 64-bit form."""

    def __init__(self, rows, K, bits, gs, seed):
        self.q, self.scales, self.biases, _ = synth.make_weights(rows, K, bits, gs, seed)
        self.bits, self.gs, self.K = bits, gs, K
        s, b = np.repeat(bf(self.scales), gs, 1), np.repeat(bf(self.biases), gs, 1)
        self.w = s * self.q + b
        self.mag = np.abs(s * self.q) + np.abs(b)

    def product(self, x):
        """x [.., K] W^T and the bound of an fp32 result's error."""
        G = self.K // self.gs
        return x @ self.w.T, (20 + 2 * G + 32) * U * (np.abs(x) @ self.mag.T)


def lora(m: Matrix, x, a, b, ids, c):
    y, err = m.product(x)
    R, K = a.shape[1], a.shape[2]
    for i, ad in enumerate(ids):
        if 0 <= ad < len(c):
            v = a[ad] @ x[i]
            verr = (K + 2) * U * (np.abs(a[ad]) @ np.abs(x[i]))
            y[i] += c[ad] * (b[ad] @ v)
            err[i] += abs(c[ad]) * (np.abs(b[ad]) @ (verr + (R + 4) * U * np.abs(v))) + 4 * U * np.abs(y[i])
    return y, err


def route(l, k, softmax_all):
    """ids and weights of one token's router logits."""
    l = np.where(np.isnan(l), -math.inf, l)
    ids = sorted(range(len(l)), key=lambda e: (-l[e], e))[:k]
    e = np.exp(l - l.max())
    w = e[ids] / (e.sum() if softmax_all else e[ids].sum())
    return ids, w


def moe(x, router, gu, dn, inter, k, gelu, softmax_all):
    """y, its error bound, ids, weights, and the least gap between a chosen and the next logit over its fp32 error."""
    M, K = x.shape
    logits = x @ router.T
    y, err = np.zeros((M, K)), np.zeros((M, K))
    ids, weights, margin = np.zeros((M, k), int), np.zeros((M, k)), math.inf
    for m in range(M):
        ids[m], weights[m] = route(logits[m], k, softmax_all)
        s = np.sort(logits[m])[::-1]
        lerr = (K + 2) * U * float((np.abs(router) @ np.abs(x[m])).max())
        if len(s) > 1:
            margin = min(margin, np.min(s[:min(k, len(s) - 1)] - s[1:k + 1]) / (2 * lerr * K ** -0.5))
        werr = np.expm1(2 * lerr) + 16 * U
        for e, w in zip(ids[m], weights[m]):
            hh, herr = gu[e].product(x[m])
            g, up, ge, ue = hh[:inter], hh[inter:], herr[:inter], herr[inter:]
            act = 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) if gelu else g / (1 + np.exp(-g))
            # both activations have slopes below 1.13; expf and tanhf are within a few units in the last place
            ae = 1.13 * ge + 16 * U * np.abs(g)
            h = act * up
            he = ae * (np.abs(up) + ue) + np.abs(act) * ue + (2.0 ** -17 + 4 * U) * np.abs(h)
            d, derr = dn[e].product(h)
            y[m] += w * d
            err[m] += w * (derr * (1 + 1e-3) + he @ dn[e].mag.T) + w * np.abs(d) * (werr + (k + 4) * U)
    return y, err, ids, weights, margin


def verify(target, draft, toks, lens, temp, uniform, noise, big):
    """tokens, accepted, logprob, and for each sequence whether a decision is too close for fp32 (within 1e-5)."""
    B, S1, V = target.shape
    S = S1 - 1
    tokens, accepted, logprob, close = np.full((B, S1), -1), np.zeros(B, int), np.zeros((B, S1)), np.zeros(B, bool)

    def soft(row, t):
        row = np.where(np.isnan(row), -math.inf, np.minimum(row, big))
        if not (row > -math.inf).any():
            return np.full(V, -math.inf), np.zeros(V)
        z = (row - row.max()) / t
        lp = z - math.log(np.exp(z).sum())
        return lp, np.exp(lp)

    for b in range(B):
        greedy = not temp[b] > 0
        t = 1.0 if greedy else temp[b]
        n = min(max(int(lens[b]), 0), S)
        for i in range(S1):
            lp, p = soft(target[b, i], t)
            none = not (lp > -math.inf).any()
            x = int(toks[b, i]) if i < n else None
            if x is not None:
                px = p[x] if 0 <= x < V else 0.0
                if greedy:
                    take = not none and x == int(np.argmax(lp))
                else:
                    q = np.zeros(V)
                    if draft is None:
                        if 0 <= x < V:
                            q[x] = 1.0
                        qx = 1.0
                    else:
                        q = soft(draft[b, i], t)[1]
                        qx = q[x] if 0 <= x < V else 0.0
                    close[b] |= 0 < abs(uniform[b, i] * qx - px) < 1e-5 * px
                    take = uniform[b, i] * qx < px
                if take:
                    tokens[b, i], logprob[b, i] = x, lp[x]
                    accepted[b] += 1
                    continue
            if none:
                logprob[b, i] = -math.inf
                break
            if greedy:
                tok = int(np.argmax(lp))
            else:
                rest = np.maximum(p - q, 0) if x is not None else p
                if not (rest > 0).any():
                    rest = p
                ratio = rest / np.maximum(noise[b], 2.0 ** -126)
                tok = int(np.argmax(ratio))
                second = np.partition(ratio, -2)[-2] if V > 1 else 0.0
                # a difference of near-equal probabilities carries their rounding
                blur = 1e-5 * (1 + (p[tok] / rest[tok] if rest[tok] > 0 else 0))
                close[b] |= second > ratio[tok] * (1 - blur)
            tokens[b, i], logprob[b, i] = tok, lp[tok]
            break
    return tokens, accepted, logprob, close
