"""Oracle: the page pool (TEST INFRASTRUCTURE ONLY): reserve, fork and compact, one page at a time.

Source: "lesty.tech — EAGLE-2 vs. Medusa", section 8 has pages that are reserved before the verify pass
and go back to a free pool after it; sharing by counts, copies on the first write and compaction have no
counterpart on the pages.  State: block_table [B, max_blocks] (-1: none), prefix_len [B], refs [num_blocks]
= table entries that name a page plus whatever else is counted (0: free).  The functions return new arrays.

Pins (tests/test_oracle_page_pool.py): counts equal the tables' entries after any sequence of calls, no page
is both free and named, a forked sequence reads the same rows as its source, and writes to one fork
never reach another.
"""
from __future__ import annotations

import numpy as np


def reserve(k_cache, v_cache, block_table, prefix_len, refs, n, freed=()):
    """(k, v, table, refs, granted, errors): errors holds "bad" and / or "short"."""
    k, v = np.array(k_cache), np.array(v_cache)
    table, refs = np.array(block_table, dtype=np.int64), np.array(refs, dtype=np.int64)
    bs, errors = k.shape[2], set()
    for p in np.asarray(freed).reshape(-1):
        if p < 0:
            continue
        if p >= len(refs) or refs[p] <= 0:
            errors.add("bad")
        else:
            refs[p] -= 1
    free = [p for p in range(len(refs)) if refs[p] == 0]
    granted, exhausted = [], False
    for b in range(len(prefix_len)):
        L = int(prefix_len[b])
        span = range(max(L, 0) // bs, -(-(L + n) // bs))
        if L < 0 or L + n > table.shape[1] * bs or any(not -1 <= table[b, i] < len(refs) for i in span):
            errors.add("bad")
            granted.append(-1)
            continue
        want = [i for i in span
                if table[b, i] == -1 or (i == L // bs and L % bs > 0 and refs[table[b, i]] > 1)]
        if want and (exhausted or len(want) > len(free)):
            exhausted = True
            errors.add("short")
            granted.append(-1)
            continue
        for i in want:
            old, new = table[b, i], free.pop(0)
            if old >= 0:
                k[new, :, :L % bs] = k[old, :, :L % bs]
                v[new, :, :L % bs] = v[old, :, :L % bs]
                refs[old] -= 1
            table[b, i], refs[new] = new, 1
        granted.append(len(want))
    return k, v, table, refs, np.array(granted), errors


def fork(block_table, prefix_len, refs, src, block_size):
    """(table, prefix_len, refs, bad)."""
    table, refs = np.asarray(block_table, dtype=np.int64), np.array(refs, dtype=np.int64)
    B, width = table.shape
    new = np.full((len(src), width), -1, dtype=np.int64)
    lens, bad = np.zeros(len(src), dtype=np.int64), False
    for r, s in enumerate(src):
        if s == -1:
            continue
        if not 0 <= s < B or not 0 <= prefix_len[s] <= width * block_size:
            bad = True
            continue
        lens[r] = prefix_len[s]
        for i in range(-(-int(lens[r]) // block_size)):
            p = table[s, i]
            if 0 <= p < len(refs):
                new[r, i] = p
            else:
                bad = True
    for t, step in ((table, -1), (new, 1)):
        for p in t.reshape(-1):
            if 0 <= p < len(refs):
                refs[p] += step
            elif p != -1:
                bad = True
    return new, lens, refs, bad or bool((refs < 0).any())


def compact(block_table, refs, *buffers):
    """(table, refs, remap, live, bad, moved buffers)."""
    table, refs = np.array(block_table, dtype=np.int64), np.array(refs, dtype=np.int64)
    used = [p for p in range(len(refs)) if refs[p] > 0]
    live = len(used)
    holes = [p for p in range(live) if refs[p] <= 0]
    remap = np.full(len(refs), -1, dtype=np.int64)
    new, bufs = refs.copy(), [np.array(x) for x in buffers]
    for p in used:
        to = p if p < live else holes.pop(0)
        remap[p] = to
        if to != p:
            new[to], new[p] = refs[p], 0
            for x in bufs:
                x[to] = x[p]
    bad = False
    for cell in np.ndindex(*table.shape):
        p = table[cell]
        table[cell] = remap[p] if 0 <= p < len(refs) else -1
        bad |= p != -1 and table[cell] == -1
    return table, new, remap, live, bool(bad), bufs
