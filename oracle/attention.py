"""Plain 64-bit oracle of the cache append and of attention over the 8-bit paged cache.

One loop per sequence, head and page, straight from the definitions; nothing here follows the
kernels' order of work.  A batch is (news, lens): new tokens and length (with them) per sequence.
"""
from __future__ import annotations

import numpy as np

_GRID = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)][:127])  # magnitudes of E4M3 codes 0 .. 126 (127: NaN)


def e4m3_decode(codes):
    """Values of E4M3 bytes (0x7F and 0xFF are NaN)."""
    codes = np.asarray(codes, dtype=np.uint8)
    mag = np.append(_GRID, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def e4m3_encode(x):
    """The nearest E4M3 code of each value, ties to the even code, saturating at 448; NaN gives 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(_GRID, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - _GRID[lo], _GRID[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def page_scale(amax):
    """The smallest power of two s, 2^-100 to 2^120, with amax <= 448 s."""
    s = 2.0 ** -100
    while amax > 448.0 * s and s < 2.0 ** 120:
        s *= 2.0
    return s


def norm_rope(x, weight, eps, offset, cos_sin, interleaved, pos):
    """x [heads, d] of one token at position pos -> normed and rotated, in float64."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    if cos_sin is not None:
        r = cos_sin.shape[1]
        out = y.copy()
        for j in range(r // 2):
            c, s = float(cos_sin[pos, j]), float(cos_sin[pos, r // 2 + j])
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)
            out[:, a] = y[:, a] * c - y[:, b] * s
            out[:, b] = y[:, b] * c + y[:, a] * s
        y = out
    return y


def append(x, news, lens, pages, page_tokens, codes, scales):
    """Write the new tokens x [n, heads, d] (float64) into copies of codes [pages, heads, tokens, d] (uint8) and
    scales [pages, heads]; returns (codes, scales, exact) with exact [pages, heads, tokens, d] the values the new
    tokens' codes stand for before rounding (NaN elsewhere)."""
    codes, scales = codes.copy(), np.array(scales, dtype=np.float64)
    exact = np.full(codes.shape, np.nan)
    row = 0
    for b, (t, length) in enumerate(zip(news, lens)):
        first = length - t
        for i in range(first // page_tokens, -(-length // page_tokens) if t else 0):
            lo, hi, pg = max(first, i * page_tokens), min(length, (i + 1) * page_tokens), int(pages[b][i])
            held = lo - i * page_tokens
            for h in range(codes.shape[1]):
                new = x[row + lo - first:row + hi - first, h]
                fin = np.abs(new[np.isfinite(new)])
                s = page_scale(fin.max() if fin.size else 0.0)
                if held:
                    old = scales[pg, h]
                    s = max(s, old)
                    if s > old:
                        codes[pg, h, :held] = e4m3_encode(e4m3_decode(codes[pg, h, :held]) * (old / s))
                scales[pg, h] = s
                at = slice(held, held + hi - lo)
                codes[pg, h, at] = e4m3_encode(new / s)
                exact[pg, h, at] = new
        row += t
    return codes, scales, exact


def attention(q, news, lens, pages, page_tokens, kc, ks, vc, vs, scale, window=0):
    """out [n, hq, d] in float64 for q [n, hq, d] and, for the tests' bounds, per row and head: the sum of
    p |v| [n, hq, d], the largest sum over d of |q k| scale [n, hq] and the largest |v|.  Tokens of a page whose
    key scale is 0 do not enter."""
    q = np.asarray(q, dtype=np.float64)
    n, hq, d = q.shape
    hkv = kc.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    load, vmax = np.zeros((n, hq)), np.zeros((n, hq))
    row = 0
    for b, (t, length) in enumerate(zip(news, lens)):
        ids = [int(i) for i in pages[b][:-(-length // page_tokens)]]
        for g in range(hkv if length else 0):
            k, v = (np.concatenate([e4m3_decode(c[i, g]) * float(s[i, g]) for i in ids])[:length]
                    for c, s in ((kc, ks), (vc, vs)))
            live = np.repeat([ks[i, g] != 0 for i in ids], page_tokens)[:length]
            for i in range(t):
                pos = length - t + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0:
                    continue
                kk, vv = k[lo:pos + 1][live[lo:pos + 1]], v[lo:pos + 1][live[lo:pos + 1]]
                if not len(kk):
                    continue
                for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    s = kk @ q[row + i, h] * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[row + i, h] = p @ vv
                    mag[row + i, h] = p @ np.abs(vv)
                    load[row + i, h] = np.max(np.abs(kk) @ np.abs(q[row + i, h])) * scale
                    vmax[row + i, h] = np.max(np.abs(vv))
        row += t
    return out, mag, load, vmax
