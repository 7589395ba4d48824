"""Pins of oracle/page_select.py: the score is an upper bound, the choice is the brute-force one, and
keeping every page is dense tree attention."""
import itertools

import numpy as np

import oracle
from oracle.page_select import grid_exponent


def _table(rng, B, width):
    return rng.permutation(B * width).reshape(B, width)


def test_bounds_enclose_the_keys_and_fit_eight_bits():
    rng = np.random.default_rng(0)
    k = rng.standard_normal((6, 2, 4, 5)) * np.exp(rng.standard_normal((6, 2, 1, 1)) * 6)
    k[1, 0, :, 2] = 0
    out = oracle.page_bounds(k, np.arange(6).reshape(1, 6), [24], [0], np.zeros((6, 2, 2, 5)))
    hi, lo = out[:, :, 0], out[:, :, 1]
    assert (hi >= k.max(2)).all() and (lo <= k.min(2)).all()
    amax = np.abs(k).max((2, 3))
    slack = np.maximum(2.0 ** np.ceil(np.log2(amax / 255)), 2.0 ** -40)
    assert (hi - k.max(2) < slack[..., None]).all() and (k.min(2) - lo < slack[..., None]).all()
    for page, h in np.ndindex(6, 2):
        units = out[page, h] / slack[page, h]
        assert (units == np.rint(units)).all() and np.abs(units).max() <= 255


def test_bounds_of_other_pages_and_odd_values():
    k = np.ones((3, 1, 2, 4))
    k[0, 0] = [[np.nan, 1, np.inf, 0], [np.nan, np.nan, 2, 0]]
    out = oracle.page_bounds(k, np.array([[0, 1, 2]]), [4], [1], np.full((3, 1, 2, 4), 7.0))
    limit = 255 * 2.0 ** 40
    assert out[0, 0, 0].tolist() == [0, 2.0 ** 40, limit, 0] and out[0, 0, 1].tolist() == [0, 0, 0, 0]
    assert (out[1] == 1).all() and (out[2] == 7).all()  # page 1 became complete, page 2 is not


def test_scores_bound_every_product_from_above():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((5, 2, 3, 8))
    b = oracle.page_bounds(k, np.arange(5).reshape(1, 5), [15], [0], np.zeros((5, 2, 2, 8)))
    q = rng.standard_normal((4, 6, 8))
    s = oracle.page_scores(q, b, np.arange(5), 5)
    qg = oracle.grid_query(q)
    for h, i, p in np.ndindex(2, 4, 5):
        dots = qg[i, 3 * h:3 * h + 3] @ k[p, h].T
        assert s[h, i, p] >= dots.max()
    assert np.abs(qg - q).max() <= np.abs(q).max() / 255


def test_choice_is_the_best_subset():
    rng = np.random.default_rng(2)
    b = np.rint(rng.standard_normal((7, 1, 2, 4)) * 3)
    b = np.stack([b.max(2), b.min(2)], 2)
    q = np.rint(rng.standard_normal((1, 2, 1, 4)) * 2)
    pages, count, words, kept = oracle.page_select(q, b, np.arange(7).reshape(1, 7), [7 * 2 + 1], 4, 1, 1, 2, 7)
    s = oracle.page_scores(q[0], b, np.arange(7), 7)[0]
    for i in range(2):
        chosen = np.nonzero(kept[0, 0, i])[0]
        assert len(chosen) == 4 and 0 in chosen and 6 in chosen
        best = max(itertools.combinations(range(1, 6), 2), key=lambda c: (s[i, list(c)].sum(), [-x for x in c]))
        assert s[i, chosen].sum() == s[i, [0, 6, *best]].sum()
    union = np.nonzero(kept[0, 0].any(0))[0]
    assert count[0, 0] == len(union) and pages[0, 0, :len(union)].tolist() == union.tolist()
    assert (pages[0, 0, len(union):] == -1).all()
    for u, p in enumerate(union):
        assert int(words[0, 0, u, 0]) == sum(1 << i for i in range(2) if kept[0, 0, i, p])


def test_all_pages_kept_is_dense_attention():
    rng = np.random.default_rng(3)
    B, m, Hq, Hkv, d, bs = 2, 3, 4, 2, 6, 4
    table = _table(rng, B, 6)
    k, v = rng.standard_normal((2, B * 6, Hkv, bs, d))
    q = rng.standard_normal((B, m, Hq, d))
    L = [13, 8]
    mask = np.tril(np.ones((B, m, m), dtype=bool))
    kept = np.ones((B, Hkv, m, 3), dtype=bool)
    kept[1, :, :, 2] = False  # the second sequence completes two pages only
    out, lse, _ = oracle.tree_attention_sparse(q, k, v, table, L, mask, kept, 0.4)
    ref, ref_lse = oracle.tree_attention(q, k, v, table, L, mask, 0.4)
    np.testing.assert_allclose(out, ref, atol=1e-13)
    np.testing.assert_allclose(lse, ref_lse, atol=1e-13)


def test_a_node_without_keys():
    k = np.ones((1, 1, 4, 2))
    out, lse, _ = oracle.tree_attention_sparse(np.ones((1, 2, 1, 2)), k, k, np.array([[0]]), [0],
                                               np.array([[[True, False], [False, False]]]), np.zeros((1, 1, 2, 1), bool), 1.0)
    assert (out[0, 1] == 0).all() and lse[0, 1, 0] == -np.inf and (out[0, 0] == 1).all()


def test_the_query_itself_exceeds_the_score_by_half_a_step_at_most():
    """The query is rounded to the nearest multiple of its step 2^e, so a channel is off by half of one at most: the
    score of the query as it is differs by at most 2^(e-1) sum_c max(|hi_c|, |lo_c|), and a page is chosen in place of
    another only where such scores are that close.  Queries with a few large channels among them."""
    rng = np.random.default_rng(3)
    nf, d, n = 24, 32, 8
    above = 0
    for big in (1.0, 30.0, 300.0):
        k = rng.standard_normal((nf, 1, 2, d)) * np.exp(rng.standard_normal((nf, 1, 1, d)))
        b = oracle.page_bounds(k, np.arange(nf).reshape(1, nf), [2 * nf], [0], np.zeros((nf, 1, 2, d)))[:, 0]
        for _ in range(20):
            q = rng.standard_normal(d)
            q[:2] *= big
            s = oracle.page_scores(q.reshape(1, 1, d), b[:, None], np.arange(nf), nf)[0, 0]
            own = np.maximum(q * b[:, 0], q * b[:, 1]).sum(-1)
            step = 2.0 ** grid_exponent(np.abs(q).max())
            room = step / 2 * np.abs(b).max(1).sum(-1) * (1 + 1e-12)
            assert (np.abs(s - own) <= room).all()
            dots = (k[:, 0] @ q).max(1)
            assert (dots <= s + room).all()
            above += int((np.abs(s - own) > 0).any())
            order = np.lexsort((np.arange(nf), -s))
            best = np.lexsort((np.arange(nf), -own))[:n]
            for p in order[:n]:
                for other in best:
                    if other not in order[:n]:
                        assert own[other] - own[p] <= room[other] + room[p]
    assert above > 50
