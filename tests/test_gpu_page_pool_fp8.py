"""GPU kv_reserve and kv_compact of an 8-bit cache vs the oracle: codes and scales move together, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import Cache, ints
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
pool = oracle.page_pool


@pytest.fixture(autouse=True)
def _built():
    lib()


def _cache(rng, nb, Hkv, d, bs, sb):
    """Every byte and any scale: what moves is not looked at."""
    c = Cache(rng, [1], 0, Hkv, d, bs, sb, spare=nb - 1)
    for i in (0, 1):
        c.codes[i] = rng.integers(0, 256, c.codes[i].shape).astype(np.uint8)
        c.scales[i] = rng.standard_normal(c.scales[i].shape).astype(np.float32)
    return c


def _assert_bits(dev, codes, scales):
    for t, ref in zip(dev[:2], codes):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), ref)
    for t, ref in zip(dev[2:], scales):
        assert np.array_equal(t.cpu().numpy(), ref)


def _state(rng, B, ways, nb, width, bs):
    """Rows in groups that share all their pages."""
    L = np.repeat(rng.integers(0, (width - 1) * bs, size=-(-B // ways)), ways)[:B]
    perm, at = rng.permutation(nb), 0
    table, refs = np.full((B, width), -1, dtype=np.int64), np.zeros(nb, dtype=np.int64)
    for b in range(B):
        if b % ways:
            table[b] = table[b - 1]
        else:
            p = -(-int(L[b]) // bs)
            table[b, :p] = perm[at:at + p]
            at += p
    for p in table[table >= 0]:
        refs[p] += 1
    return table, L, refs


@pytest.mark.parametrize("B,ways,nb,width,bs,sb,Hkv,d", [(5, 1, 60, 9, 16, 16, 2, 128), (12, 3, 80, 7, 16, 4, 2, 64), (9, 4, 20, 6, 8, 1, 1, 20),
                                                         (6, 6, 40, 5, 32, 8, 3, 4), (8, 2, 60, 5, 128, 64, 2, 128), (4, 4, 30, 3, 300, 1, 1, 4)])
def test_reserve(B, ways, nb, width, bs, sb, Hkv, d):
    for seed in range(3):
        rng = np.random.default_rng(seed + nb)
        table, L, refs = _state(rng, B, ways, nb, width, bs)
        c = _cache(rng, nb, Hkv, d, bs, sb)
        dev, status = c.device(), ts.new_status()
        got = ts.kv_reserve(*dev[:2], ints(table), ints(L), ints(refs), 5, k_scale=dev[2], v_scale=dev[3], status=status)
        rk, rv, rt, rr, rg, errors = pool.reserve(*c.codes, table, L, refs, 5, [])
        assert int(status.item()) == (0 if not errors else -7)
        # a scale is that of its block's first row
        rows = [np.repeat(s, sb, axis=2)[..., None] for s in c.scales]
        sk, sv = [x[:, :, ::sb, 0] for x in pool.reserve(*rows, table, L, refs, 5, [])[:2]]
        _assert_bits(dev, (rk, rv), (sk, sv))
        for name, ref in (("block_table", rt), ("refs", rr), ("granted", rg)):
            assert np.array_equal(got[name].cpu().numpy(), ref), name


@pytest.mark.parametrize("nb,width,bs,sb,Hkv,d", [(60, 9, 16, 16, 2, 128), (80, 7, 16, 4, 2, 36), (500, 60, 8, 1, 1, 4), (40, 12, 128, 64, 2, 128)])
def test_compact(nb, width, bs, sb, Hkv, d):
    rng = np.random.default_rng(nb)
    table, _, refs = _state(rng, 6, 2, nb, width, bs)
    c = _cache(rng, nb, Hkv, d, bs, sb)
    dev, status = c.device(), ts.new_status()
    got = ts.kv_compact(*dev[:2], ints(table), ints(refs), k_scale=dev[2], v_scale=dev[3], status=status)
    ts.check_status(status)
    rt, rr, remap, live, bad, (rk, rv, sk, sv) = pool.compact(table, refs, *c.codes, *c.scales)
    _assert_bits(dev, (rk, rv), (sk, sv))
    for name, ref in (("block_table", rt), ("refs", rr), ("remap", remap), ("live", [live])):
        assert np.array_equal(got[name].cpu().numpy(), ref), name


def test_off_aligned_caches_move_by_words():
    rng = np.random.default_rng(3)
    table, L, refs = _state(rng, 6, 3, 40, 5, 16)
    c = _cache(rng, 40, 2, 128, 16, 8)
    dev = c.device()
    for i in range(4):
        x = dev[i].view(torch.uint8).flatten()
        buf = torch.empty(x.numel() + 4, dtype=torch.uint8, device="cuda")[4:]
        buf.copy_(x)
        dev[i] = buf.view(dev[i].dtype).view(dev[i].shape)
    r = ts.kv_reserve(*dev[:2], ints(table), ints(L), ints(refs), 5, k_scale=dev[2], v_scale=dev[3])
    ts.kv_compact(*dev[:2], r["block_table"], r["refs"], k_scale=dev[2], v_scale=dev[3])
    rk, rv, rt, rr, _, _ = pool.reserve(*c.codes, table, L, refs, 5, [])
    rows = [np.repeat(s, 8, axis=2)[..., None] for s in c.scales]
    sk, sv = [x[:, :, ::8, 0] for x in pool.reserve(*rows, table, L, refs, 5, [])[:2]]
    moved = pool.compact(rt, rr, rk, rv, sk, sv)[5]
    _assert_bits(dev, moved[:2], moved[2:])


def test_refusals():
    c = _cache(np.random.default_rng(0), 6, 2, 128, 16, 8)
    dev = c.device()
    table, L, refs = ints([[0, -1]]), ints([3]), ints([1, 0, 0, 0, 0, 0])
    scales = dict(k_scale=dev[2], v_scale=dev[3])
    for kw, why in ((dict(k_scale=dev[2]), "k_scale and v_scale"), (dict(), "unsupported dtype"),
                    (dict(scales, v_scale=dev[3][:5]), "shape"), (dict(scales, k_scale=dev[2].double()), "float32")):
        with pytest.raises(ValueError, match=why):
            ts.kv_reserve(*dev[:2], table, L, refs, 4, **kw)
        with pytest.raises(ValueError, match=why):
            ts.kv_compact(*dev[:2], table, refs, **kw)
    with pytest.raises(ValueError, match="bounds"):
        ts.kv_compact(*dev[:2], table, refs, bounds=torch.zeros(6, 2, 2, 128, dtype=torch.bfloat16, device="cuda"), **scales)
    with pytest.raises(ValueError, match="float8"):
        ts.kv_reserve(*[x.float() for x in dev[:2]], table, L, refs, 4, **scales)
    out = dict(block_table=table, refs=dev[2].view(torch.int32).flatten()[:6], granted=ints([0]))
    with pytest.raises(ValueError, match="shares memory with k_scale"):
        ts.kv_reserve(*dev[:2], table, L, refs, 4, out=out, **scales)
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        ts.kv_compact(dev[0], dev[0], table, refs, **scales)
    _assert_bits(dev, c.codes, c.scales)
