"""Pins of the oracle of the 8-bit cache."""
import numpy as np
import pytest
import torch

import oracle
from oracle import kv_fp8 as o8


def test_table_hand_values_and_torch():
    for c, v in ((0x00, 0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6), (0x38, 1.0), (0x3C, 1.5), (0x7E, 448.0),
                 (0xB8, -1.0)):
        assert o8.E4M3[c] == v
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, o8.E4M3, equal_nan=True)


def test_encode_is_the_nearest_code_ties_to_even():
    every = np.concatenate([o8.E4M3[:127], -o8.E4M3[:127]])
    assert np.array_equal(o8.E4M3[o8.encode(every)], every)
    for c in range(126):
        lo, hi = o8.E4M3[c], o8.E4M3[c + 1]
        mid = (lo + hi) / 2
        assert o8.encode(mid) == (c if c % 2 == 0 else c + 1)
        assert o8.encode(np.nextafter(mid, 0)) == c and o8.encode(np.nextafter(mid, 1e9)) == c + 1
    assert list(o8.encode([448.0, 1e9, np.inf, -np.inf])) == [0x7E, 0x7E, 0x7E, 0xFE]
    assert np.isnan(o8.E4M3[o8.encode(np.nan)])
    x = np.random.default_rng(0).standard_normal(4000) * 40
    assert np.array_equal(o8.E4M3[o8.encode(x)], torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())


def test_exponent_by_definition():
    for big, e in ((0.0, -40), (448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (448 * 2.0 ** 40, 40), (np.inf, 40), (1e-30, -40)):
        assert o8.exponent([0.0, -big, np.nan]) == e
    assert o8.exponent([np.nan]) == -40


def _cache(rng, nb, hkv, bs, d, sb):
    return (rng.integers(0, 120, (nb, hkv, bs, d)).astype(np.uint8) | (rng.integers(0, 2, (nb, hkv, bs, d)) * 128).astype(np.uint8),
            2.0 ** rng.integers(-6, 3, (nb, hkv, bs // sb)))


@pytest.mark.parametrize("sb", [1, 4, 8])
def test_write_keeps_what_lies_before_and_meets_the_grid(sb):
    rng = np.random.default_rng(sb)
    cache, scale = _cache(rng, 4, 2, 8, 4, sb)
    before_c, before_s = cache.copy(), scale.copy()
    table = [2, 0, 3]
    start, rows = 5, rng.standard_normal((9, 2, 4)) * 7          # positions 5 .. 13
    o8.write_one(cache, scale, rows, table, start)
    got, old = o8.values(cache, scale), o8.values(before_c, before_s)
    for t in range(9):
        pos = start + t
        page, row = table[pos // 8], pos % 8
        s = scale[page, :, row // sb][:, None]
        # half a step of three fraction bits, or half the subnormal step
        assert (np.abs(got[page, :, row] - rows[t]) <= np.maximum(np.abs(rows[t]) * 2.0 ** -4, 2.0 ** -10 * s)).all()
    for pos in range(start):
        page, row = table[pos // 8], pos % 8
        if pos // sb < start // sb:
            assert np.array_equal(cache[page, :, row], before_c[page, :, row])
        s = scale[page, :, row // sb][:, None]
        assert (np.abs(got[page, :, row] - old[page, :, row]) <= 2.0 ** -10 * s).all()   # subnormals at most
    assert np.array_equal(cache[1], before_c[1]) and np.array_equal(scale[3], before_s[3])
    assert np.array_equal(cache[0, :, 6:], before_c[0, :, 6:])                           # rows behind the write
    # every touched block is filled to its scale
    for first in range(start // sb * sb, 14, sb):
        page, row = table[first // 8], first % 8
        live = [p for p in range(first, first + sb) if p < 14]
        for h in range(2):
            vals = [old[table[p // 8], h, p % 8] if p < start else rows[p - start, h] for p in live]
            assert scale[page, h, row // sb] == 2.0 ** o8.exponent(vals)


def test_a_second_write_forgets_the_first():
    rng = np.random.default_rng(3)
    cache, scale = _cache(rng, 2, 1, 8, 4, 8)
    ref_c, ref_s = cache.copy(), scale.copy()
    small, large = rng.standard_normal((4, 1, 4)), rng.standard_normal((4, 1, 4)) * 500
    kept = o8.values(cache, scale)[0, 0, :3]
    o8.write_one(cache, scale, large, [0, 1], 3)
    o8.write_one(cache, scale, small, [0, 1], 3)
    o8.write_one(ref_c, ref_s, small, [0, 1], 3)
    assert np.array_equal(scale, ref_s)
    assert np.array_equal(cache[0, 0, 3:7], ref_c[0, 0, 3:7])
    assert (np.abs(o8.values(cache, scale)[0, 0, :3] - kept) <= 2.0 ** -9 * 16).all()


def test_commit_is_a_write_of_the_accepted_values():
    rng = np.random.default_rng(5)
    cache, scale = _cache(rng, 6, 2, 4, 4, 4)
    table, L, m, path = np.array([[5, 0, 2, 4]]), 6, 7, np.array([[0, 2, 5, -1, -1, -1, -1]])
    v = o8.values(cache, scale)
    rows = np.stack([v[table[0][(L + p) // 4], :, (L + p) % 4] for p in (0, 2, 5)])
    ref_c, ref_s = cache.copy(), scale.copy()
    o8.write_one(ref_c, ref_s, rows, table[0], L)
    t, prefix, freed, count = o8.commit((cache,), (scale,), table, [L], path, [3], m)
    assert np.array_equal(cache, ref_c) and np.array_equal(scale, ref_s)
    assert list(t[0]) == [5, 0, 2, -1] and list(freed[0]) == [4, -1, -1, -1] and list(count) == [1] and list(prefix) == [9]


def test_read_and_attention_are_those_of_the_values():
    rng = np.random.default_rng(6)
    cache, scale = _cache(rng, 5, 2, 8, 4, 4)
    cache2, scale2 = _cache(rng, 5, 2, 8, 4, 2)
    table, prefix, m = np.array([[3, 1], [0, 4]]), np.array([9, 4]), 3
    k, v = o8.values(cache, scale), o8.values(cache2, scale2)
    mask = np.stack([oracle.ancestor_mask([-1, 0, 0])] * 2)
    q = rng.standard_normal((2, m, 4, 4))
    out, lse = o8.tree_attention_fp8(q, k, v, table, prefix, mask, 0.5)
    ref, ref_lse = oracle.tree_attention(q, k, v, table, prefix, mask, 0.5)
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-12) and np.allclose(lse, ref_lse, rtol=1e-12)
    got = o8.read(cache, scale, table, prefix, [7, 0], 4)
    assert np.array_equal(got[0, 1], k[1, :, 0]) and (got[0, 2:] == 0).all() and np.array_equal(got[1, 3], k[0, :, 3])


def test_a_row_without_keys():
    out, lse = o8.tree_attention_fp8(np.ones((1, 1, 1, 2)), np.ones((1, 1, 4, 2)), np.ones((1, 1, 4, 2)), [[0]], [0],
                                     np.zeros((1, 1, 1), dtype=bool), 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()
