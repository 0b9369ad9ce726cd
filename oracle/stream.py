"""Plain fp64 statement of the streaming operators: rotary positions over
several axes, writing a paged 8-bit cache, and attention over it. Test
infrastructure, like the rest of this package: numpy only, nothing from the
product. Pinned by tests/test_oracle_stream.py."""
from __future__ import annotations

import numpy as np

PAGE = 128
MIN_EXP = -117


def rope_frequencies(dims, theta, ladder):
    """(frequency, axis) of every rotated channel pair."""
    total = sum(dims)
    freq, axis = [], []
    for a, d in enumerate(dims):
        for j in range(d // 2):
            e = 2.0 * j / d if ladder == "axis" else 2.0 * len(freq) / total
            freq.append(theta ** -e)
            axis.append(a)
    return np.array(freq), np.array(axis)


def rope(x, pos, dims, theta=10000.0, pairing="interleaved", ladder="axis", inverse=False):
    """x [n][heads][d] (fp64), pos [n][3]: every pair turned by position * frequency."""
    freq, axis = rope_frequencies(dims, theta, ladder)
    pairs = len(freq)
    y = np.array(x, np.float64, copy=True)
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if pairing == "interleaved" else (i, i + pairs)
        w = np.asarray(pos, np.float64)[:, axis[i]] * freq[i] * (-1.0 if inverse else 1.0)
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def e4m3_values():
    """The value of every e4m3 bit pattern."""
    v = np.empty(256)
    for i in range(256):
        e, m = (i >> 3) & 15, i & 7
        x = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[i] = np.nan if i & 127 == 127 else (-x if i & 128 else x)
    return v


_VALUES = e4m3_values()


def round_e4m3(x):
    """Bit patterns of the e4m3 values nearest to x (ties to the even pattern; |x| <= 448, what is not finite
    becomes NaN)."""
    x = np.asarray(x, np.float64)
    pos = _VALUES[:127]  # ascending
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a == pos[hi], hi, pick)
    bits = pick | np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), bits, 127).astype(np.uint8)


def page_exponent(amax):
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def cache_write(x, c, scale, tok_start, kv_len, table):
    """Appends x [n][heads][d] (fp64 values) to c uint8 [pages][heads][128][d] and scale [pages][heads], in place."""
    for b in range(len(kv_len)):
        t0, t1 = tok_start[b], tok_start[b + 1]
        begin = kv_len[b] - (t1 - t0)
        for pg in range(begin // PAGE, -(-kv_len[b] // PAGE)):
            lo, hi = max(begin - pg * PAGE, 0), min(kv_len[b] - pg * PAGE, PAGE)
            page = table[b][pg]
            for h in range(x.shape[1]):
                new = x[t0 + pg * PAGE + lo - begin: t0 + pg * PAGE + hi - begin, h]
                fin = np.abs(new[np.isfinite(new)])
                s = 2.0 ** page_exponent(fin.max() if fin.size else 0.0)
                if lo > 0:
                    old = float(scale[page, h])
                    s = max(s, old)
                    if s != old:
                        held = _VALUES[c[page, h, :lo]]
                        bits = round_e4m3(held * (old / s))
                        c[page, h, :lo] = np.where(np.isnan(held), 127 | (c[page, h, :lo] & 128), bits)
                scale[page, h] = s
                c[page, h, lo:hi] = round_e4m3(new / s)


def cache_attention(q, c_k, c_v, s_k, s_v, tok_start, kv_len, table, scale, unit=0, shift=0):
    """(o, lse, sum p |v|) [heads_q][n].. of every packed token; NaN where a token belongs to no stream. shift: tokens
    before the cached ones that count for positions and are not attended to."""
    hq, n, d = q.shape
    group = hq // c_k.shape[1]
    o, av = np.full((hq, n, d), np.nan), np.full((hq, n, d), np.nan)
    lse = np.full((hq, n), np.nan)
    for b in range(len(kv_len)):
        t0, t1, length = tok_start[b], tok_start[b + 1], kv_len[b]
        for h in range(hq):
            g = h // group
            pages = table[b][: -(-length // PAGE)]
            k = (_VALUES[c_k[pages, g]] * s_k[pages, g].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            v = (_VALUES[c_v[pages, g]] * s_v[pages, g].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            for i in range(t0, t1):
                pos = shift + length - (t1 - t0) + i - t0
                end = length if unit == 0 else min(length, max(0, (pos // unit + 1) * unit - shift))
                if end == 0:
                    o[h, i], av[h, i], lse[h, i] = 0.0, 0.0, -np.inf
                    continue
                s = k[:end] @ q[h, i] * scale
                m = s.max()
                p = np.exp(s - m)
                o[h, i], av[h, i] = p @ v[:end] / p.sum(), p @ np.abs(v[:end]) / p.sum()
                lse[h, i] = m + np.log(p.sum())
    return o, lse, av
