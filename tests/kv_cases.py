"""Seeded inputs of the key-value cache tests, shared by the CPU and GPU runs."""

import numpy as np

import oracle.kv_oracle as K

# Half an ulp of each type, relative to the value, and its smallest step.
EPS = {"f16": 2.0**-11, "bf16": 2.0**-8, "f32": 2.0**-24}
TINY = {"f16": 2.0**-25, "bf16": 2.0**-134, "f32": 2.0**-150}
CODE = {"f16": 0, "f32": 1, "bf16": 2}


def bf16_bits(x):
    """bf16 bit patterns (uint16) of float32 values, round to nearest even."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def cast(x, name):
    """(values as float32, array in the type's storage) of float values x."""
    with np.errstate(over="ignore"):
        x = np.asarray(x, dtype=np.float32)
    if name == "f16":
        with np.errstate(over="ignore"):
            h = x.astype(np.float16)
        return h.astype(np.float32), h
    if name == "bf16":
        b = bf16_bits(x)
        return bf16_values(b), b
    return x, x


def batch(rng, lens, news, page, width=None, ragged=None, spare=3):
    """(table, lens, starts or None, n_pages): pages in random order, entries
    past a sequence's length -7 (never to be read)."""
    need = [max(0, -(-m // page)) for m in lens]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    width = max(need + [1]) + 1 if width is None else width
    table = np.full((len(lens), width), -7, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, : min(k, width)] = order[at : at + k][:width]
        at += k
    starts = None
    if ragged or (ragged is None and any(n != 1 for n in news)):
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return table, np.asarray(lens, dtype=np.int32), starts, n_pages


def cache(rng, n_pages, heads, page, dim, bits, garbage=False):
    """A cache of quantised random tokens. garbage: any bits at all."""
    c = {"head_dim": dim, "bits": bits}
    for n in "kv":
        if garbage:
            c[n + "_codes"] = rng.integers(0, 2**32, (n_pages, heads, page, dim * bits // 32), dtype=np.uint64).astype(np.uint32)
            c[n + "_grid"] = rng.integers(0, 2**32, (n_pages, heads, page), dtype=np.uint64).astype(np.uint32)
        else:
            x = rng.standard_normal((n_pages, heads, page, dim)) * np.exp(0.3 * rng.standard_normal((n_pages, 1, page, 1)))
            x += 0.5 * rng.standard_normal((1, heads, 1, dim))
            codes, c[n + "_grid"] = K.quantize(x, bits)
            c[n + "_codes"] = K.pack(codes, bits)
    return c


# Values far from 1, as v = factor (3 + N(0, 1)), with the same weight for
# every key. The smaller factor is above the bound's least error of longest *
# 2^-121 by far. (head_dim, bits, q dtype, out dtype, factor)
FAR_VALUES = [(64, 4, "bf16", "bf16", 2.0**-110), (64, 8, "f32", "f32", 2.0**-110), (64, 4, "f32", "f32", 2.0**100),
              (64, 8, "bf16", "bf16", 2.0**100)]


def far_cache(rng, n_pages, heads, page, dim, bits, factor):
    c = cache(rng, n_pages, heads, page, dim, bits)
    codes, c["v_grid"] = K.quantize(factor * (3 + rng.standard_normal((n_pages, heads, page, dim))), bits)
    c["v_codes"] = K.pack(codes, bits)
    return c


def poison(c, table, lens):
    """Every place past a sequence's length, and every page that no sequence
    has, gets a NaN or infinite scale and all code bits set."""
    size = c["k_grid"].shape[2]
    live = np.zeros((c["k_grid"].shape[0], size), bool)
    for b, m in enumerate(lens):
        for p in range(max(0, m)):
            if p // size < table.shape[1] and 0 <= table[b, p // size] < live.shape[0]:
                live[table[b, p // size], p % size] = True
    for n in "kv":
        g = c[n + "_grid"]
        bad = np.where((np.arange(size) % 2 == 0)[None, None], np.uint32(0x7FC000FF), np.uint32(0xFF8000FF))
        c[n + "_grid"] = np.where(live[:, None, :], g, np.broadcast_to(bad, g.shape)).astype(np.uint32)
        c[n + "_codes"] = np.where(live[:, None, :, None], c[n + "_codes"], np.uint32(0xFFFFFFFF))


def span(cache, name):
    """Largest s (2^bits - 1) of the finite grids of the cache."""
    s = (cache[name + "_grid"] & np.uint32(0xFFFFFF00)).view(np.float32).astype(np.float64)
    return float(s[np.isfinite(s)].max()) * (2 ** cache["bits"] - 1)


def attention_bound(ref, mag, q, cache, scale, slopes, q_dtype, out_dtype, longest):
    """Largest error of an attention output element, with every rounding of
    the method counted. mag is the weighted mean of |v|.

    * A weight is rounded to fp16: 2^-11 of it (two parts: 2^-22). One below
      fp16's normal range is off by at most 2^-25 while the largest is at
      least 2^8: 2^-33 of the range of v a key. Steps of v below 2^-96 count
      as that when the reference is chosen (so that 2^(x - M) stays finite):
      the sum of the weights is then at least 2^(8 + 96), a key is off by at
      most 2^-25 (2^bits - 1) over that.
    * A score's error moves its weight by as much, numerator and denominator:
      twice. Its terms sum to at most `size` = scale * sum |q| * range of k (and the
      position bias); the matrix core rounds once for 4 products, so head_dim
      / 4 times; the one-part form adds the offset of the codes to its terms
      (79 / 15 or 1279 / 255 of their range: offsets of 64 and 1024); scaling, bias, difference to the
      reference and the parts of q add up to 16 roundings more.
    * The sums over the keys: a wave of four takes every fourth tile, one
      rounding for 4 keys; joins and rescalings at most 300.
    * The output's own rounding."""
    bits, dim = cache["bits"], cache["head_dim"]
    two = "f32" in (q_dtype, out_dtype)
    size = abs(scale) * np.abs(q).sum(-1, keepdims=True) * span(cache, "k")
    if slopes is not None:
        size = size + np.abs(slopes)[None, :, None] * longest
    offset = 1.0 if two else 79 / 15 if bits == 4 else 1279 / 255
    weight = 2.0**-22 if two else 2.0**-11
    scores = 2.0**-24 * size * offset * (dim / 4 + 16)
    sums = 2.0**-24 * (longest / 16 + 300)
    reach = max(span(cache, "v"), (2**bits - 1) * 2.0**-96)
    return (mag * (weight + 2 * scores + sums) + longest * 2.0**-33 * reach
            + np.abs(ref) * EPS[out_dtype] * 1.01 + TINY[out_dtype])
