"""Plain float64 oracle of the quantised key-value cache (test infrastructure).

Written from the definitions, one token and head at a time where that keeps
it plain; it shares no code with the HIP path. A cache is a dict of numpy
arrays: k_codes, v_codes uint32 [pages, heads, page_size, words], k_grid,
v_grid uint32 [pages, heads, page_size], and the integers head_dim and bits.
"""

from __future__ import annotations

import numpy as np

NAN_WORD = 0x7FC00000


def round16(s):
    """fp32 numbers s > 0 to 16 significant bits, ties to even."""
    frac, power = np.frexp(np.asarray(s, dtype=np.float64))
    return np.ldexp(np.rint(frac * 65536.0), power - 16)


def quantize(x, bits):
    """(codes int64 [..., dim], grid words uint32 [...]) of x [..., dim]: the
    range and the step are rounded to fp32, the step to 16 significant bits,
    everything else is float64."""
    x = np.asarray(x, dtype=np.float64)
    top = 2**bits - 1
    finite = np.isfinite(x).all(-1)
    y = np.where(finite[..., None], x, 0.0)
    lo, hi = np.minimum(y.min(-1), 0.0), np.maximum(y.max(-1), 0.0)
    with np.errstate(over="ignore"):
        span = np.float32(hi - lo)
    good = finite & np.isfinite(span)
    span = np.where(good, span, np.float32(1.0)).astype(np.float64)
    s = np.float32(span / top).astype(np.float64)
    flat = s < 2.0**-126
    s = np.where(flat, np.float64(np.float32(2.0 / top)), s)
    lo = np.where(flat, -1.0, lo)
    s = round16(s)
    z = np.rint(-np.where(good, lo, 0.0) / s)
    c = np.clip(np.rint(np.where(good[..., None], y, 0.0) / s[..., None]) + z[..., None], 0, top).astype(np.int64)
    word = s.astype(np.float32).view(np.uint32) | z.astype(np.uint32)
    return np.where(good[..., None], c, 0), np.where(good, word, np.uint32(NAN_WORD)).astype(np.uint32)


def pack(codes, bits):
    """Words [..., dim * bits / 32] of codes [..., dim], first code lowest."""
    per = 32 // bits
    c = codes.reshape(*codes.shape[:-1], -1, per).astype(np.uint64)
    return (c << (np.arange(per, dtype=np.uint64) * np.uint64(bits))).sum(-1).astype(np.uint32)


def unpack(words, bits):
    sh = np.arange(0, 32, bits, dtype=np.uint32)
    return ((words[..., None] >> sh) & np.uint32(2**bits - 1)).reshape(*words.shape[:-1], -1).astype(np.int64)


def values(words, grid, bits):
    """float64 values [..., dim]."""
    s = (grid & np.uint32(0xFFFFFF00)).view(np.float32).astype(np.float64)
    return s[..., None] * (unpack(words, bits) - (grid & np.uint32(2**bits - 1)).astype(np.int64)[..., None])


def places(cache, table, lens, starts, n_tokens):
    """Per row of the call: None (behind the last sequence), "absent", or
    (page, offset); and whether a position was on no page."""
    pages, _, size = cache["k_grid"].shape
    out, bad = [None] * n_tokens, False
    if starts is None:
        starts = range(len(lens) + 1)
    for b in range(len(lens)):
        n = int(starts[b + 1]) - int(starts[b])
        for i in range(n):
            pos = int(lens[b]) - n + i
            out[starts[b] + i] = "absent"
            if pos < 0:
                continue
            if pos // size >= table.shape[1] or not 0 <= table[b, pos // size] < pages:
                bad = True
                continue
            out[starts[b] + i] = (int(table[b, pos // size]), pos % size)
    return out, bad


def write(cache, k, v, table, lens, starts=None):
    """The cache after the call (a copy) and its info."""
    new = {n: (a.copy() if isinstance(a, np.ndarray) else a) for n, a in cache.items()}
    at, bad = places(cache, table, lens, starts, len(k))
    for t, p in enumerate(at):
        if isinstance(p, tuple):
            for name, x in (("k", k[t]), ("v", v[t])):
                c, w = quantize(x, cache["bits"])
                new[name + "_codes"][p[0], :, p[1]] = pack(c, cache["bits"])
                new[name + "_grid"][p[0], :, p[1]] = w
    return new, bad


def read(cache, table, lens, starts, n_tokens):
    """([k, v] float64 [n_tokens, heads, dim], row written or not, info)."""
    at, bad = places(cache, table, lens, starts, n_tokens)
    heads = cache["k_grid"].shape[1]
    out = [np.zeros((n_tokens, heads, cache["head_dim"])) for _ in range(2)]
    for t, p in enumerate(at):
        if isinstance(p, tuple):
            for o, name in zip(out, "kv"):
                o[t] = values(cache[name + "_codes"][p[0], :, p[1]], cache[name + "_grid"][p[0], :, p[1]], cache["bits"])
    return out, np.array([p is not None for p in at]), bad


def attention(q, cache, table, lens, starts=None, scale=1.0, slopes=None):
    """(out float64 [n_tokens, q_heads, dim], the largest |v| weight sum a row
    had (the size its rounding errors go by), row written or not, info)."""
    pages, heads, size = cache["k_grid"].shape
    n_tokens, q_heads, dim = q.shape
    q = np.asarray(q, dtype=np.float64)
    out, mag = np.zeros(q.shape), np.zeros((n_tokens, q_heads, dim))
    written, bad = np.zeros(n_tokens, bool), False
    if starts is None:
        starts = range(len(lens) + 1)
    cap = table.shape[1] * size
    for b in range(len(lens)):
        n = int(starts[b + 1]) - int(starts[b])
        written[starts[b] : starts[b + 1]] = True
        end = min(int(lens[b]), cap) if n else 0
        bad |= n > 0 and int(lens[b]) > cap
        if end <= 0:
            continue
        pos = np.arange(end)
        ids = table[b, pos // size].astype(np.int64)
        on = (ids >= 0) & (ids < pages)
        bad |= not on.all()
        ids = np.where(on, ids, 0)
        k = values(cache["k_codes"][ids, :, pos % size], cache["k_grid"][ids, :, pos % size], cache["bits"])
        v = values(cache["v_codes"][ids, :, pos % size], cache["v_grid"][ids, :, pos % size], cache["bits"])
        for i in range(n):
            at = int(lens[b]) - n + i
            seen = on & (pos <= at)
            if not seen.any():
                continue
            for h in range(q_heads):
                g = h // (q_heads // heads)
                s = scale * (k[seen, g] @ q[starts[b] + i, h])
                if slopes is not None:
                    s = s + float(slopes[h]) * (pos[seen] - at)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[starts[b] + i, h] = p @ v[seen, g]
                mag[starts[b] + i, h] = p @ np.abs(v[seen, g])
    return out, mag, written, bool(bad)
