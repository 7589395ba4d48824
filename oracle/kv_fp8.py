"""Oracle: a paged K/V cache in 8 bits (fp64; codes as unsigned bytes).

No counterpart on the pages.  Definitions:

* ``E4M3[c]``: the value of byte c: sign, four exponent bits (bias 7), three fraction bits; exponent 0 holds the
  subnormals (c & 7) * 2^-9; 0x7f and 0xff are NaN; no infinities, the largest value is 448.
* ``encode(x)``: the byte whose value is nearest, of two equally near ones that with an even fraction; magnitudes above 448
  (infinities too) give 448; NaN gives a NaN byte.
* ``exponent(values)``: the smallest e in [-40, 40] with |x| <= 448 * 2^e for every x that is not NaN.
* ``write``: the rows become positions start .. of a sequence; every block of sb positions that gets a row is quantised over
  its kept rows (below start) and its new ones.
* ``commit``: the accepted rows' values are written at the prefix's end; tables and released pages as
  :func:`oracle.kv_commit`.
* ``values`` / ``tree_attention_fp8``: codes times scales, and the attention over them.

Pins (tests/test_oracle_kv_fp8.py): the byte table against hand values and torch's float8_e4m3fn, encode against
every midpoint, the exponent against its definition by search, write and commit against row-by-row statements, the
attention against :func:`oracle.tree_attention` on the values.
"""
from __future__ import annotations

import numpy as np

LO, HI = -40, 40


def _value(c: int) -> float:
    sign, e, f = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
    if e == 15 and f == 7:
        return float("nan")
    return sign * (f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))


E4M3 = np.array([_value(c) for c in range(256)])
_POS = E4M3[:127]  # 0 .. 448, ascending


def encode(x) -> np.ndarray:
    """Bytes of the nearest codes."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)          # first code whose value is >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(x), 127, c)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(values) -> int:
    v = np.abs(np.asarray(values, dtype=np.float64))
    v = v[~np.isnan(v)]
    big = v.max() if v.size else 0.0
    e = LO
    while e < HI and big > 448.0 * 2.0 ** e:
        e += 1
    return e


def clamp_scale(s) -> np.ndarray:
    s = np.asarray(s, dtype=np.float64)
    return np.clip(np.where(np.isnan(s), 2.0 ** LO, s), 2.0 ** LO, 2.0 ** HI)


def values(cache, scale) -> np.ndarray:
    """cache uint8 [NB, Hkv, bs, d], scale [NB, Hkv, bs / sb] -> fp64 values."""
    sb = cache.shape[2] // scale.shape[2]
    return E4M3[cache] * np.repeat(clamp_scale(scale), sb, axis=2)[..., None]


def _quantise(cache, scale, page, h, row, rows):
    """Rows (values, kept ones and new) become rows ``row`` .. of one page's block."""
    sb = cache.shape[2] // scale.shape[2]
    e = exponent(rows)
    with np.errstate(invalid="ignore"):
        cache[page, h, row:row + len(rows)] = encode(rows * 2.0 ** -e)
    scale[page, h, row // sb] = 2.0 ** e


def write_one(cache, scale, rows, table_row, start: int) -> None:
    """rows [len, Hkv, d] become positions start .. of one sequence, in place."""
    bs, sb = cache.shape[2], cache.shape[2] // scale.shape[2]
    old = values(cache, scale)
    end = start + len(rows)
    if len(rows) == 0:
        return
    for first in range(start // sb * sb, end, sb):
        page, row = table_row[first // bs], first % bs
        kept = max(0, start - first)
        stop = min(sb, end - first)
        for h in range(cache.shape[1]):
            new = rows[max(first, start) - start: first + stop - start, h]
            _quantise(cache, scale, page, h, row, np.concatenate([old[page, h, row:row + kept], new]))


def write(cache, scale, x, table, start, length) -> None:
    """x [B, n, Hkv, d]; cache (uint8) and scale change in place."""
    for b in range(x.shape[0]):
        write_one(cache, scale, np.asarray(x[b, :length[b]], dtype=np.float64), table[b], int(start[b]))


def read(cache, scale, table, prefix, start, n: int) -> np.ndarray:
    v, bs = values(cache, scale), cache.shape[2]
    out = np.zeros((len(prefix), n, cache.shape[1], cache.shape[3]))
    for b in range(len(prefix)):
        for t in range(max(0, min(n, prefix[b] - start[b]))):
            pos = start[b] + t
            out[b, t] = v[table[b][pos // bs], :, pos % bs]
    return out


def commit(caches, scales, table, prefix, path, length, m: int):
    """In place on the caches and scales; returns (table, prefix, freed, freed_count)."""
    table, bs = np.array(table), caches[0].shape[2]
    out, freed = table.copy(), np.full(table.shape, -1, dtype=table.dtype)
    count = np.zeros(len(prefix), dtype=np.int32)
    for b, (L, a) in enumerate(zip(prefix, length)):
        for cache, scale in zip(caches, scales):
            v = values(cache, scale)
            rows = np.stack([v[table[b][(L + p) // bs], :, (L + p) % bs] for p in path[b][:a]])
            write_one(cache, scale, rows, table[b], int(L))
        keep, used = -(-(L + a) // bs), -(-(L + m) // bs)
        count[b] = used - keep
        freed[b, :used - keep] = table[b, keep:used]
        out[b, keep:used] = -1
    return out, np.asarray(prefix) + np.asarray(length), freed, count


def tree_attention_fp8(q, k, v, table, prefix, mask, scale: float):
    """q [B, m, Hq, d]; k, v: values [NB, Hkv, bs, d]; mask bool [B, m, m] -> (out, lse), fp64."""
    q = np.asarray(q, dtype=np.float64)
    B, m, Hq, d = q.shape
    bs, g = k.shape[2], Hq // k.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, m, Hq), -np.inf)
    for b in range(B):
        L = int(prefix[b])
        pos = np.arange(L + m)
        pages = np.asarray(table[b])[pos // bs]
        ks, vs = k[pages, :, pos % bs], v[pages, :, pos % bs]
        for i in range(m):
            seen = np.concatenate([np.ones(L, dtype=bool), mask[b, i]])
            for h in range(Hq):
                if not seen.any():
                    continue
                with np.errstate(all="ignore"):
                    s = scale * (ks[seen, h // g] @ q[b, i, h])
                    top = s.max()
                    w = np.exp(s - top)
                    out[b, i, h] = (w[:, None] * vs[seen, h // g]).sum(0) / w.sum()
                    lse[b, i, h] = top + np.log(w.sum())
    return out, lse
