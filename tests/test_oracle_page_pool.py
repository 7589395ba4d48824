"""Pins of oracle/page_pool.py: conservation of pages and the independence of forked sequences."""
import numpy as np

import oracle

pool = oracle.page_pool


def _counts(table, nb):
    c = np.zeros(nb, dtype=np.int64)
    for p in table[table >= 0]:
        c[p] += 1
    return c


def _rows(cache, table, b, n):
    bs = cache.shape[2]
    return np.stack([cache[table[b, i // bs], :, i % bs] for i in range(n)]) if n else np.zeros(0)


def test_a_long_run_keeps_the_counts_and_the_rows():
    rng = np.random.default_rng(0)
    nb, H, bs, d, width = 40, 2, 4, 3, 8
    k, v = np.zeros((2, nb, H, bs, d))
    table, L, refs = np.full((3, width), -1), np.zeros(3, dtype=np.int64), np.zeros(nb, dtype=np.int64)
    told = [[] for _ in range(3)]  # what each sequence has been told to hold
    for step in range(60):
        B = len(L)
        n = int(rng.integers(1, 6))
        k, v, table, refs, granted, errors = pool.reserve(k, v, table, L, refs, n)
        assert "bad" not in errors
        assert (refs == _counts(table, nb)).all()
        for b in range(B):
            if granted[b] < 0:
                continue
            a = int(rng.integers(0, n + 1))
            for j in range(a):
                x = rng.standard_normal((H, d))
                page, slot = table[b, (L[b] + j) // bs], (L[b] + j) % bs
                assert refs[page] == 1
                k[page, :, slot], v[page, :, slot] = x, -x
                told[b].append(x)
            L[b] += a
        src = rng.integers(-1, B, size=int(rng.integers(1, 5)))
        if (src < 0).all():
            src[0] = 0
        table, L, refs, bad = pool.fork(table, L, refs, src, bs)
        assert not bad and (refs == _counts(table, nb)).all()
        told = [list(told[s]) if s >= 0 else [] for s in src]
        if step % 3 == 0:
            table, refs, remap, live, bad, (k, v) = pool.compact(table, refs, k, v)
            assert not bad and (refs[:live] > 0).all() and (refs[live:] == 0).all()
        for b in range(len(L)):
            if L[b] >= (width - 2) * bs:  # drop a sequence that has grown long
                keep = np.arange(len(L))
                keep[b] = -1
                table, L, refs, bad = pool.fork(table, L, refs, keep, bs)
                told[b] = []
            assert L[b] == len(told[b])
            if told[b]:
                assert (_rows(k, table, b, L[b]) == np.stack(told[b])).all()
                assert (_rows(v, table, b, L[b]) == -np.stack(told[b])).all()


def test_the_last_holder_keeps_a_shared_page():
    k = np.arange(5 * 4.0).reshape(5, 1, 4, 1)
    table = np.array([[3, -1], [3, -1], [3, -1]])
    k2, v2, t2, refs, granted, errors = pool.reserve(k, k, table, [2, 2, 2], [0, 0, 0, 3, 0], 1)
    assert t2[:, 0].tolist() == [0, 1, 3] and granted.tolist() == [1, 1, 0] and not errors
    assert refs.tolist() == [1, 1, 0, 1, 0]
    assert (k2[0, 0, :2] == k[3, 0, :2]).all() and (k2[0, 0, 2:] == k[0, 0, 2:]).all()


def test_a_short_pool_leaves_the_later_sequences():
    k = np.zeros((4, 1, 2, 1))
    table = np.array([[0, -1, -1], [1, -1, -1], [1, -1, -1]])
    _, _, t2, refs, granted, errors = pool.reserve(k, k, table, [2, 1, 1], [1, 2, 0, 0], 4)
    assert granted.tolist() == [2, -1, -1] and errors == {"short"}
    assert t2.tolist() == [[0, 2, 3], [1, -1, -1], [1, -1, -1]] and refs.tolist() == [1, 2, 1, 1]


def test_freed_pages_come_back_first():
    k = np.zeros((3, 1, 2, 1))
    _, _, t2, refs, granted, errors = pool.reserve(k, k, np.array([[-1]]), [0], [1, 1, 2], 2, freed=[[1, -1], [2, 2]])
    assert t2.tolist() == [[1]] and refs.tolist() == [1, 1, 0] and not errors
    assert pool.reserve(k, k, np.array([[-1]]), [0], [1, 1, 2], 2, freed=[1, 1])[5] == {"bad"}


def test_fork_drops_what_nobody_continues():
    table = np.array([[0, 1, 5], [2, 3, -1]])
    t2, L2, refs, bad = pool.fork(table, [3, 4], [1, 1, 1, 1, 0, 1], [0, 0, -1], 2)
    assert t2.tolist() == [[0, 1, -1], [0, 1, -1], [-1, -1, -1]] and L2.tolist() == [3, 3, 0]
    assert refs.tolist() == [2, 2, 0, 0, 0, 0] and not bad
