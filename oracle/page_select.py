"""Oracle: page bounds, the choice of pages and tree attention over it (TEST INFRASTRUCTURE ONLY).

The pages (web sources) have no counterpart.  Definitions, in fp64:

* bounds of a complete page, KV head and channel: the largest and the smallest key (NaN ignored,
  0 if there is nothing else, magnitudes clamped to 255 * 2^40), rounded outwards to whole multiples
  of 2^e, e the smallest exponent in [-40, 40] with 255 * 2^e covering the page and head;
* a query row is rounded (half to even) to whole multiples of its own 2^e; the score of a page for a node
  and KV head is the maximum over the group's heads of sum_c max(q_c hi_c, q_c lo_c);
* a node keeps the first and the most recent complete pages and the best others by
  (score descending, index ascending), n in all;
* attention as in :mod:`oracle.tree_attention`, over the kept pages, the incomplete page's prefix
  rows and the node's ancestors; a node without keys gives 0 and -inf.

Pins (tests/test_oracle_page_select.py): the score bounds every grid-rounded q . k of the page from
above; brute force over all orderings; every page kept equals dense tree attention.
"""
from __future__ import annotations

import math

import numpy as np

from .tree_attention import _f64

LO, HI, TOP = -40, 40, 255
LIMIT = TOP * 2.0 ** HI


def grid_exponent(amax: float) -> int:
    e = LO
    while e < HI and TOP * 2.0 ** e < amax:
        e += 1
    return e


def page_bounds(k_cache, block_table, prefix_len, start_len, bounds):
    """New bounds [num_blocks, Hkv, 2, d] (fp64): those of the pages complete at prefix_len but not
    at start_len are computed, the others copied from ``bounds``."""
    out = _f64(bounds).copy()
    k = _f64(k_cache)
    bs = k.shape[2]
    for b in range(len(prefix_len)):
        for p in range(int(start_len[b]) // bs, int(prefix_len[b]) // bs):
            page = int(block_table[b][p])
            for h in range(k.shape[1]):
                rows = k[page, h]
                hi = np.array([max([x for x in c if not math.isnan(x)], default=0.0) for c in rows.T])
                lo = np.array([min([x for x in c if not math.isnan(x)], default=0.0) for c in rows.T])
                hi, lo = np.clip(hi, -LIMIT, LIMIT), np.clip(lo, -LIMIT, LIMIT)
                g = 2.0 ** grid_exponent(max(np.abs(hi).max(), np.abs(lo).max()))
                out[page, h, 0] = np.ceil(hi / g) * g
                out[page, h, 1] = np.floor(lo / g) * g
    return out


def grid_query(q):
    """[..., d] -> the same on each row's grid."""
    q = np.clip(np.where(np.isnan(q), 0.0, q), -LIMIT, LIMIT)
    flat = q.reshape(-1, q.shape[-1])
    out = np.empty_like(flat)
    for i, row in enumerate(flat):
        g = 2.0 ** grid_exponent(np.abs(row).max())
        out[i] = np.rint(row / g) * g
    return out.reshape(q.shape)


def page_scores(q, bounds, table_row, n_full):
    """[Hkv, m, n_full] scores of one sequence; q [m, Hq, d]; an id out of range scores 0."""
    bnd = _f64(bounds)
    m, Hq, d = q.shape
    Hkv = bnd.shape[1]
    g = Hq // Hkv
    qg = grid_query(_f64(q)).reshape(m, Hkv, g, d)
    out = np.zeros((Hkv, m, n_full))
    for p in range(n_full):
        page = int(table_row[p])
        if not 0 <= page < bnd.shape[0]:
            continue
        hi, lo = bnd[page, :, 0], bnd[page, :, 1]
        out[:, :, p] = np.maximum(qg * hi[None, :, None], qg * lo[None, :, None]).sum(-1).max(-1).T
    return out


def page_select(q, bounds, block_table, prefix_len, n, first, recent, block_size, C):
    """Returns (pages [B, Hkv, C], count [B, Hkv], node_mask uint64 [B, Hkv, C, W], kept bool [B, Hkv, m, C])."""
    q = _f64(q)
    B, m = q.shape[:2]
    Hkv = bounds.shape[1]
    W = (m + 63) // 64
    kept = np.zeros((B, Hkv, m, C), dtype=bool)
    for b in range(B):
        nf = int(prefix_len[b]) // block_size
        s = page_scores(q[b], bounds, block_table[b], nf)
        for h in range(Hkv):
            for i in range(m):
                forced = [p for p in range(nf) if p < first or p >= nf - recent]
                rest = sorted((p for p in range(nf) if p not in set(forced)), key=lambda p: (-s[h, i, p], p))
                kept[b, h, i, (forced + rest)[:max(n, len(forced))]] = True
    pages, count, words = pack(kept, W)
    return pages, count, words, kept


def pack(kept, W):
    B, Hkv, m, C = kept.shape
    pages = np.full((B, Hkv, C), -1, dtype=np.int32)
    count = np.zeros((B, Hkv), dtype=np.int32)
    words = np.zeros((B, Hkv, C, W), dtype=np.uint64)
    for b in range(B):
        for h in range(Hkv):
            for u, p in enumerate(np.nonzero(kept[b, h].any(0))[0]):
                pages[b, h, u] = p
                count[b, h] += 1
                for i in np.nonzero(kept[b, h, :, p])[0]:
                    words[b, h, u, i // 64] |= np.uint64(1 << (int(i) % 64))
    return pages, count, words


def tree_attention_sparse(q, k_cache, v_cache, block_table, prefix_len, mask, kept, scale):
    """(out, lse, spread): fp64 [B, m, Hq, d], [B, m, Hq] and sum_j p_j |v_j| [B, m, Hq, d].

    kept: bool [B, Hkv, m, C]; mask: bool [B, m, m]."""
    qd = _f64(q)
    B, m, Hq, d = qd.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    g = Hq // Hkv
    out, spread = np.zeros((B, m, Hq, d)), np.zeros((B, m, Hq, d))
    lse = np.full((B, m, Hq), -np.inf)
    for b in range(B):
        L = int(prefix_len[b])
        nf = L // bs
        for h in range(Hkv):
            for i in range(m):
                pos = [p * bs + r for p in np.nonzero(kept[b, h, i])[0] for r in range(bs)]
                pos += list(range(nf * bs, L)) + [L + t for t in np.nonzero(mask[b, i])[0]]
                if not pos:
                    continue
                pos = np.array(pos)
                blocks = np.asarray(block_table[b])[pos // bs]
                k = _f64(k_cache[blocks, h, pos % bs])
                v = _f64(v_cache[blocks, h, pos % bs])
                s = qd[b, i, h * g:(h + 1) * g] @ k.T * scale
                top = s.max(1, keepdims=True)
                e = np.exp(s - top)
                z = e.sum(1, keepdims=True)
                out[b, i, h * g:(h + 1) * g] = e @ v / z
                spread[b, i, h * g:(h + 1) * g] = e @ np.abs(v) / z
                lse[b, i, h * g:(h + 1) * g] = (top + np.log(z))[:, 0]
    return out, lse, spread
