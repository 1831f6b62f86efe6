"""Plain 64-bit oracle of the operators around the products: RMS norm, low-rank adapters, routing by a rule.

Straight from the definitions, row by row where that is simplest; nothing here follows the kernels' order of work.
"""
from __future__ import annotations

import numpy as np

from .attention import e4m3_encode
from .formats import bf16_value, round_to_bf16

SCALE_MIN = 2.0 ** -100


def rms_norm(x, residual, weight, eps, offset):
    """(h, y) in float64 from bf16 values x, residual (or None) [m, k] and weight [k]; h is rounded to bf16."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = round_to_bf16(h + np.asarray(residual, np.float64))
    with np.errstate(all="ignore"):
        y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    return h, y


def quantise(y, group):
    """(q, scales): y [m, k] over its groups' scales [m, groups], neither rounded; group 0: a row."""
    m, k = y.shape
    g = group or k
    scales = np.empty((m, -(-k // g)))
    q = np.empty_like(y)
    with np.errstate(all="ignore"):
        for i in range(scales.shape[1]):
            part = y[:, i * g:(i + 1) * g]
            amax = np.max(np.where(np.isfinite(part), np.abs(part), 0.0), axis=1)
            scales[:, i] = np.maximum(amax / 448.0, SCALE_MIN)
            q[:, i * g:(i + 1) * g] = part / scales[:, i:i + 1]
    return q, scales


def codes_between(q, rel):
    """The lowest and highest E4M3 code value that rounding q times 1 - rel .. 1 + rel can give (by value)."""
    from .attention import e4m3_decode
    a, b = e4m3_decode(e4m3_encode(q * (1 - rel))), e4m3_decode(e4m3_encode(q * (1 + rel)))
    return np.minimum(a, b), np.maximum(a, b)


def lora(ids, x, y, a, b, scales, ranks):
    """(out, h, mag) in float64: out [m, n] unrounded, h [m, max_rank] without the scale and mag [m, max_rank] the sums of
    |a x| behind it (zeros past the rank and in rows without an adapter)."""
    out, h, mag = np.array(y, np.float64), np.zeros((len(ids), a.shape[1])), np.zeros((len(ids), a.shape[1]))
    for i, e in enumerate(ids):
        if 0 <= e < len(a):
            r = ranks[e]
            h[i, :r] = a[e, :r] @ x[i]
            mag[i, :r] = np.abs(a[e, :r]) @ np.abs(x[i])
            out[i] += scales[e] * (b[e, :, :r] @ h[i, :r])
    return out, h, mag


def route_by(logits, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_best=2, renormalise=True, scale=1.0):
    """(ids [t, topk], weights [t, topk] in float64) by a rule, token by token.

    A softmax is over the logits that are numbers: a NaN one adds nothing to its sum, comes after every number and has the weight NaN.
    Scores in 64 bits order the experts.  Without a bias, and with groups valued by one expert if there are any, the scores meant are
    exact ones: two that 64 bits round to one value (a sigmoid of 40 and of 50) are in their logits' order."""
    lg = np.asarray(logits, np.float32).astype(np.float64)
    t, n = lg.shape
    ids, weights = np.zeros((t, topk), np.int64), np.zeros((t, topk))
    exact = bias is None and (groups == 1 or group_best == 1)
    for i in range(t):
        l = lg[i]
        num = ~np.isnan(l)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                e = np.exp(l - np.max(l[num], initial=-np.inf))
                s = e / np.sum(e[num])
            c = s + (0.0 if bias is None else np.asarray(bias, np.float32).astype(np.float64))

            def place(e):  # smaller comes first: by value, then by the logit where exact scores are meant, then by the index
                nan = np.isnan(l[e]) if exact else np.isnan(c[e])
                return nan, 0.0 if np.isnan(c[e]) else -c[e], -l[e] if exact and not nan else 0.0, e
            out = np.zeros(n, bool)
            if groups > 1:
                per = n // groups
                if exact:  # a group's value is its first expert's
                    value = [min(place(e) for e in range(g * per, g * per + per)) for g in range(groups)]
                    value = [(False, 0.0, np.inf) if v[0] else v[:3] for v in value]  # no number in it: as minus infinity
                    keep = sorted(range(groups), key=lambda g: value[g] + (g,))
                else:
                    value = np.full(groups, -np.inf)
                    for g in range(groups):
                        part = np.sort(c[g * per:(g + 1) * per][~np.isnan(c[g * per:(g + 1) * per])])[::-1][:group_best]
                        value[g] = np.sum(part) if len(part) == group_best else -np.inf
                        value[g] = -np.inf if np.isnan(value[g]) else value[g]
                    keep = sorted(range(groups), key=lambda g: (-value[g], g))
                for g in keep[topk_groups:]:
                    out[g * per:(g + 1) * per] = True
            ids[i] = sorted(np.flatnonzero(~out), key=place)[:topk]
            w = s[ids[i]]
            weights[i] = scale * (w / np.sum(w) if renormalise else w)
    return ids, weights


__all__ = ["rms_norm", "quantise", "codes_between", "lora", "route_by", "bf16_value", "round_to_bf16"]
