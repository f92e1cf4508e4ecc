"""Plain numpy implementations in 64 bits of the softmax-attention layer's operators, from their
definitions, with loops over sequences, pages and tokens.  They share no code with the library."""

import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """The 256 values of e4m3 by code (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m / 8.0, -6) if e == 0 else math.ldexp(1.0 + m / 8.0, e - 7)
        out[c] = math.nan if (c & 0x7f) == 0x7f else x
    return np.where(np.arange(256) >= 128, -out, out)


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]                     # 0 .. 448, ascending with the code


def e4m3_encode(x):
    """Codes of x, rounded to nearest with ties to the even code; beyond +-448 the nearest; NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), E4M3_MAX)
    hi = np.searchsorted(_POSITIVE, a)        # first code whose value is >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_POSITIVE[hi] == a, hi, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7f, code).astype(np.uint8)


def e4m3_decode(codes):
    return _VALUES[np.asarray(codes, dtype=np.uint8)]


def power_scale(amax):
    """The smallest power of two s with amax <= 448 s, its exponent held to [-60, 60]."""
    if not amax > 0:
        return 2.0 ** -60
    if math.isinf(amax):
        return 2.0 ** 60
    e = -60
    while amax > E4M3_MAX * 2.0 ** e and e < 60:
        e += 1
    return 2.0 ** e


def rope(x, positions, frequencies, amplitude, layout, inverse):
    """x [T, H, d] rotated, and the size |a| + |b| of each channel's pair (0 where it is copied)."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.zeros_like(x)
    half = len(frequencies)
    for t in range(x.shape[0]):
        for i in range(half):
            ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            angle = float(positions[t]) * float(frequencies[i]) * (-1.0 if inverse else 1.0)
            c, s = amplitude * math.cos(angle), amplitude * math.sin(angle)
            a, b = x[t, :, ia], x[t, :, ib]
            y[t, :, ia], y[t, :, ib] = a * c - b * s, b * c + a * s
            size[t, :, ia] = size[t, :, ib] = np.abs(a) + np.abs(b)
    return y, size


def append(x, cache, scale, table, lens, counts):
    """Codes and scales (new copies) after the append of x [tokens, Hkv, d] (sequences back to back);
    cache [pages, Hkv, P, d] uint8, scale [pages, Hkv]."""
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    pages, heads, P, _ = cache.shape
    row0 = 0
    for n, count in enumerate(counts):
        length, cap = int(lens[n]), table.shape[1] * P
        groups = {}
        for t in range(count):
            pos = length - count + t
            if 0 <= pos < cap and 0 <= table[n, pos // P] < pages:
                groups.setdefault(pos // P, []).append((pos, row0 + t))
        row0 += count
        for page, items in groups.items():
            at, kept = table[n, page], items[0][0] - page * P
            for h in range(heads):
                rows = np.stack([x[r, h] for _, r in items]).astype(np.float64)
                finite = np.abs(rows[~np.isnan(rows)])
                s = power_scale(finite.max() if finite.size else 0.0)
                if kept:
                    old = scale[at, h]
                    s = max(old, s)
                    if s != old:
                        cache[at, h, :kept] = e4m3_encode(e4m3_decode(cache[at, h, :kept]) * (old / s))
                cache[at, h, kept:kept + len(items)] = e4m3_encode(rows / s)
                scale[at, h] = s
    return cache, scale


def attend(q, k_codes, v_codes, k_scale, v_scale, table, lens, scale):
    """q [N, T, Hq, d].  Returns o, lse, and for the tolerance per row: the weighted mean of |v|
    (as o) and the largest scale * sum |q_i k_i| over the tokens seen (as lse)."""
    q = np.asarray(q, dtype=np.float64)
    N, T, Hq, d = q.shape
    pages, Hk, P, _ = k_codes.shape
    o, mean_v = np.zeros_like(q), np.zeros_like(q)
    lse, size = np.full((N, T, Hq), -np.inf), np.zeros((N, T, Hq))
    kv, vv = e4m3_decode(k_codes), e4m3_decode(v_codes)
    for n in range(N):
        length = min(max(int(lens[n]), 0), table.shape[1] * P)
        at = np.array([table[n, j // P] for j in range(length)], dtype=np.int64).reshape(-1)
        good = (at >= 0) & (at < pages)
        slot = np.arange(length) % P
        for hk in range(Hk):
            pg = np.where(good, at, 0)
            k = kv[pg, hk, slot] * k_scale[pg, hk].astype(np.float64)[:, None]
            v = vv[pg, hk, slot] * v_scale[pg, hk].astype(np.float64)[:, None]
            for t in range(T):
                see = good & (np.arange(length) <= length - T + t)
                if not see.any():
                    continue
                for hq in range(hk * (Hq // Hk), (hk + 1) * (Hq // Hk)):
                    s = scale * (k[see] @ q[n, t, hq])
                    top = s.max()
                    w = np.exp(s - top)
                    o[n, t, hq] = (w @ v[see]) / w.sum()
                    mean_v[n, t, hq] = (w @ np.abs(v[see])) / w.sum()
                    lse[n, t, hq] = top + np.log(w.sum())
                    size[n, t, hq] = abs(scale) * (np.abs(k[see]) @ np.abs(q[n, t, hq])).max()
    return o, lse, mean_v, size
