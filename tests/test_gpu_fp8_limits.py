"""The 8-bit cache's calls at the ends of their ranges: scores and queries of every size, bounds and positions near 2^31."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import Cache, F8, assert_within, attention_bounds, ints, tree_mask, words
from gpu_helpers import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    lib()


class Far:
    """Four pages in one cache, named by the first table cells of a row and by those from ``at`` on of a far longer one."""

    def __init__(self, bs, sb, Hkv, d, at, cells):
        g = torch.Generator(device="cuda").manual_seed(bs + sb)
        shape = (4, Hkv, bs, d)
        self.start = [(torch.randn(shape, generator=g, device="cuda") * 50).to(F8) for _ in "kv"]
        self.start += [torch.exp2(torch.randint(-6, 7, (4, Hkv, bs // sb), generator=g, device="cuda").float()) for _ in "kv"]
        self.near = ints([[2, 0, 3]])
        self.table = torch.full((1, cells), -1, dtype=torch.int32, device="cuda")
        self.table[0, at:at + 3] = self.near[0, :cells - at]

    def cache(self):
        return [t.clone() for t in self.start]


def _same(a, b):
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bs,sb,m,a", [(1024, 1024, 20, 7), (1024, 1, 256, 256), (1024, 64, 256, 3), (128, 128, 256, 3), (128, 16, 256, 256)])
def test_commit_near_2_to_31(bs, sb, m, a, in_place):
    """As at the beginning of a cache: the same rows, blocks and pages."""
    cells = (1 << 31) // bs
    L = (1 << 31) - 257                                        # (the longest prefix that a tree may follow)
    near = L % bs
    p0 = (L - near) // bs
    c = Far(bs, sb, 2, 8, p0, cells)
    c.near = c.near[:, :cells - p0].contiguous()
    path = torch.full((1, m), -1, dtype=torch.int32, device="cuda")
    path[0, :a] = ints([0] + sorted(np.random.default_rng(m).choice(np.arange(1, m), a - 1, replace=False)))
    results = []
    for table, prefix in ((c.near, near), (c.table, L)):
        dev, status, lens = c.cache(), ts.new_status(), ints([prefix])
        out = None
        if in_place:
            table = table.clone()
            out = dict(block_table=table, prefix_len=lens, freed_blocks=torch.empty_like(table), freed_count=torch.empty_like(lens))
        r = ts.kv_commit_fp8(*dev, table, lens, path, ints([a]), out=out, status=status)
        ts.check_status(status)
        results.append((dev, r))
    (dev, r), (far, f) = results
    _same(dev, far)
    assert f["prefix_len"].item() == L + a and torch.equal(f["freed_count"], r["freed_count"])
    assert torch.equal(f["block_table"][0, p0:], r["block_table"][0]) and (f["block_table"][0, :p0] == -1).all()
    n = r["freed_count"].item()
    assert torch.equal(f["freed_blocks"][0, :n], r["freed_blocks"][0, :n]) and (f["freed_blocks"][0, n:] == -1).all()


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64), (torch.bfloat16, 20)])
@pytest.mark.parametrize("bs,sb,n,length", [(1024, 1, 300, 5), (1024, 1, 300, 100), (1024, 1024, 300, 255), (256, 8, 500, 400), (16, 16, 600, 30),
                                            (1024, 1, 20000, 100)])
def test_write_and_read_near_2_to_31(dtype, d, bs, sb, n, length):
    """As at the beginning of a cache, and nothing behind the last row, however many there might have been."""
    cells = (1 << 31) // bs
    L = (1 << 31) - 1 - length - (3 if bs > 16 else 0)
    p0 = L // bs
    p0 -= max(0, 3 - (cells - p0))                             # (three pages of the row are there)
    near = L - p0 * bs
    c = Far(bs, sb, 2, d, p0, cells)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = [torch.randn(1, n, 2, d, generator=g, device="cuda").to(dtype) for _ in "kv"]
    results = []
    for table, start in ((c.near, near), (c.table, L)):
        dev, status = c.cache(), ts.new_status()
        ts.kv_write_fp8(k, v, *dev, table, ints([start]), length=ints([length]), status=status)
        kv = ts.kv_read_fp8(*dev, table, ints([start + length]), n, start_len=ints([start]), dtype=torch.float32, status=status)
        ts.check_status(status)
        results.append((dev, kv))
    _same(*(dev for dev, _ in results))
    _same(*(kv for _, kv in results))
    for old, new in zip(c.start[:2], results[0][0]):           # (a block's kept rows may keep its scale)
        assert not torch.equal(old.view(torch.uint8), new.view(torch.uint8))


def test_commit_of_a_row_of_2_to_31_pages():
    """Pages of one token: cells of the table are counted beyond 2^31 too."""
    m, a, L = 40, 5, (1 << 31) - 257
    cells = L + m
    c = [torch.zeros(64, 1, 1, 4, dtype=F8, device="cuda") for _ in "kv"] + [torch.ones(64, 1, 1, device="cuda") for _ in "kv"]
    table = torch.full((1, cells), -1, dtype=torch.int32, device="cuda")
    table[0, L:L + m] = torch.arange(m, dtype=torch.int32, device="cuda")
    out = dict(block_table=table, prefix_len=ints([L]), freed_blocks=torch.empty_like(table), freed_count=ints([-1]))
    path = torch.full((1, m), -1, dtype=torch.int32, device="cuda")
    path[0, :a] = ints([0, 3, 7, 20, 39])
    for i in (0, 1):
        c[i].copy_(torch.arange(64.0, device="cuda").view(64, 1, 1, 1).expand(64, 1, 1, 4).to(F8))
    old, status = c[0].float().flatten(1)[:, 0], ts.new_status()
    ts.kv_commit_fp8(*c, table, out["prefix_len"], path, ints([a]), out=out, status=status)
    ts.check_status(status)
    assert out["prefix_len"].item() == L + a and out["freed_count"].item() == m - a
    assert torch.equal(table[0, L:L + a], torch.arange(a, dtype=torch.int32, device="cuda")) and (table[0, L + a:] == -1).all()
    assert torch.equal(out["freed_blocks"][0, :m - a], torch.arange(a, m, dtype=torch.int32, device="cuda"))
    assert (out["freed_blocks"][0, m - a:1 << 20] == -1).all() and (out["freed_blocks"][0, -(1 << 20):] == -1).all()
    for i in (0, 1):
        value = c[i].float().flatten(1)[:, 0] * c[2 + i].flatten()
        assert torch.equal(value[:a], old[[0, 3, 7, 20, 39]]) and torch.equal(value[a:], old[a:])


@pytest.mark.parametrize("nsb", [1, 2])
def test_reserve_with_scales_of_millions_of_tokens(nsb):
    """Scale blocks of 2^23 tokens and more: the copied page gets the scales that its rows reach, and nothing else changes."""
    bs, rows = nsb << 23, 10
    c = [torch.zeros(5, 1, bs, 4, dtype=F8, device="cuda") for _ in "kv"] + [torch.zeros(5, 1, nsb, device="cuda") for _ in "kv"]
    for i in range(2):
        c[i][1, 0, :rows] = torch.randn(rows, 4, device="cuda").to(F8)
        c[2 + i][:] = torch.arange(1, 5 * nsb + 1, device="cuda").view(5, 1, nsb) * (i + 2)
    before, status = [t.clone() for t in c[2:]], ts.new_status()
    r = ts.kv_reserve(*c[:2], ints([[0, 1, -1], [0, 1, -1]]), ints([bs + rows] * 2), ints([2, 2, 0, 0, 0]), 1, k_scale=c[2], v_scale=c[3],
                      status=status)
    ts.check_status(status)
    pages = set(r["block_table"][:, 1].tolist())
    assert r["granted"].sum().item() == 1 and 1 in pages and len(pages) == 2
    new = (pages - {1}).pop()
    for codes, scale, old in zip(c[:2], c[2:], before):
        assert torch.equal(codes[new, 0, :rows].float(), codes[1, 0, :rows].float()) and not codes[new, 0, rows:].view(torch.uint8).any()
        old[new, 0, 0] = old[1, 0, 0]
        assert torch.equal(scale, old)


# the tensor cores' forms: (m, Hq, Hkv, bs, sb); up to 16, 32 and any number of rows per KV head, scales for 16, 4 and 1 keys
TC = dict(rows16=(4, 4, 2, 16, 16), rows32=(8, 8, 2, 32, 8), wide=(33, 8, 2, 16, 16), wide4=(40, 4, 1, 64, 4), wide1=(33, 8, 2, 16, 1))
tc_forms = pytest.mark.parametrize("form", TC.values(), ids=TC.keys())


def _query(rng, shape, dtype=torch.bfloat16):
    return torch.from_numpy(rng.standard_normal(shape) * np.exp2(rng.integers(-2, 2, shape[:-1] + (1,)))).to(dtype)


def _attend(c, q, mask, dev=None, **kw):
    status = ts.new_status()
    kw.setdefault("max_prefix", int(c.lens.max()))
    r = ts.tree_attention_fp8(q.cuda(), *(dev or c.device()), ints(c.table), ints(c.lens), words(mask), status=status, **kw)
    ts.check_status(status)
    return r


def _reference(c, q, mask, scale=None):
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    return attention_bounds(q.double().numpy(), *c.values(), c.table, c.lens, mask, scale, q.dtype == torch.bfloat16)


@tc_forms
def test_small_queries_under_a_large_scale(form):
    """Rows near and below the least normal number; the call's scale makes ordinary scores of them."""
    m, Hq, Hkv, bs, sb = form
    rng = np.random.default_rng(m + 1)
    lens = (0, 140, 500)
    c = Cache(rng, lens, m, Hkv, 128, bs, sb)
    mask = tree_mask(rng, len(lens), m)
    size = np.exp2(-rng.integers(112, 131, (len(lens), m, Hq, 1)).astype(np.float64))
    q = torch.from_numpy(rng.standard_normal((len(lens), m, Hq, 128)) * size).to(torch.bfloat16)
    scale = 2.0 ** 112
    out, lse = _attend(c, q, mask, scale=scale)
    ref, ref_lse, bo, bl = _reference(c, q, mask, scale)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@tc_forms
@pytest.mark.parametrize("e,ks", [(40, 1.0), (70, 2.0 ** 40), (95, 1.0), (110, 1.0), (120, 2.0 ** 40)])
def test_low_scores_do_not_pass_for_none(form, e, ks):
    """Rows all of whose scores are far below zero, down to where fp32 ends: NaN, as any beyond 2^22, and not the zeros of a
    row without keys.  The other rows stay as they are."""
    m, Hq, Hkv, bs, sb = form
    rng = np.random.default_rng(e + m)
    lens, g = (0, 140, 500, 128), Hq // Hkv
    c = Cache(rng, lens, m, Hkv, 128, bs, sb)
    mask = tree_mask(rng, len(lens), m)
    mask[0, m - 1] = False                                     # (no key at all)
    c.codes[0][:, 0] = (c.codes[0][:, 0] & 0x1F) | 0x20        # the first KV head's keys lie between 1/8 and 2
    c.scales[0][:, 0] *= ks
    q = _query(rng, (len(lens), m, Hq, 128))
    low = np.zeros(q.shape[:3], dtype=bool)
    low[:, ::2, :g] = True
    if ks != 1.0:
        q[:, :, :g] /= ks                                      # (the first head's other rows: ordinary scores)
    q[torch.from_numpy(low)] = -(2.0 ** e) * (1 + torch.rand(int(low.sum()), 128, generator=torch.Generator().manual_seed(m)).bfloat16())
    low &= ~((~mask.any(2)) & (c.lens == 0)[:, None])[:, :, None]
    out, lse = _attend(c, q, mask)
    with np.errstate(all="ignore"):
        ref, ref_lse, bo, bl = _reference(c, q, mask)
    ref[low] = ref_lse[low] = np.nan
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@pytest.mark.parametrize("m,Hq,Hkv,d,lens", [(5, 4, 2, 64, (0, 70, 300)), (1, 2, 1, 128, (4000, 65, 0)), (40, 8, 2, 128, (500, 20, 0))])
def test_low_scores_in_fp32(m, Hq, Hkv, d, lens):
    """Scores below fp32's range, -inf there: keys without weight beside others, NaN where a row has no others."""
    rng = np.random.default_rng(m + d)
    g = Hq // Hkv
    c = Cache(rng, lens, m, Hkv, d, 16, 16)
    mask = tree_mask(rng, len(lens), m)
    c.codes[0][:, 0] = 0x7E                                    # the first KV head's keys are 448 * 8
    c.scales[0][:, 0] = 8.0
    for b, L in enumerate(lens):
        if L > 0:                                              # but for one of the prefix, of zeros
            c.codes[0][c.table[b, (L - 1) // 16], 0, (L - 1) % 16] = 0
    q = _query(rng, (len(lens), m, Hq, d), torch.float32)
    q[:, :, :g] = -1e37 * (1 + torch.rand(len(lens), m, g, d, generator=torch.Generator().manual_seed(d)))
    out, lse = _attend(c, q, mask)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    for b, L in enumerate(lens):
        if L > 0:
            v = c.values()[1][c.table[b, (L - 1) // 16], 0, (L - 1) % 16]
            ref[b, :, :g], bo[b, :, :g] = v, 0.0
            ref_lse[b, :, :g], bl[b, :, :g] = 0.0, 0.0
        else:
            ref[b, :, :g] = ref_lse[b, :, :g] = np.nan
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@tc_forms
def test_any_bound_of_the_lengths(form):
    """max_prefix 2^30, the most there is, over 256 KV heads: what a sequence can hold is bounded by its table."""
    m, Hq, Hkv, bs, sb = form
    rng = np.random.default_rng(m + 2)
    lens = tuple(int(x) for x in rng.integers(0, 200, 256 // Hkv))
    c = Cache(rng, lens, m, Hkv, 128, bs, sb)
    mask, q = tree_mask(rng, len(lens), m), _query(rng, (len(lens), m, Hq, 128))
    out, lse = _attend(c, q, mask, max_prefix=1 << 30)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@tc_forms
@pytest.mark.parametrize("above", [12, 14, 16, 18])
def test_one_large_channel_that_meets_zeros(form, above):
    """Queries with one channel 2^above times the others, whose keys are zero there: the scores are made of what the split of
    the queries into two 8-bit parts leaves of the others.  It is off by at most 2^-21 of a row's largest in each channel, so a score by
    dE = scale 2^-21 max|q| sum|k| beside what attention_bounds counts; the weights by twice that, relatively."""
    m, Hq, Hkv, bs, sb = form
    rng = np.random.default_rng(m + above)
    lens, scale = (3, 140, 500), 1 / math.sqrt(128)
    c = Cache(rng, lens, m, Hkv, 128, bs, sb, spread=1)
    c.codes[0] &= 0x7F                                         # (of one sign, so that errors add up)
    c.codes[0][..., 77] = 0
    mask = tree_mask(rng, len(lens), m)
    q = rng.uniform(0.5, 2.0, (len(lens), m, Hq, 128)) / 4
    y = torch.arange(0x3E00, 0x3F00, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()   # 1/8 .. 1/2
    x = y * 2.0 ** (9 - above)                                 # (the large channel at 128)
    lost = x - x.to(torch.float8_e4m3fn).float()
    lost -= lost.to(torch.float8_e5m2).float()
    q[:, 1::2] = y[lost.argmax()].item()                       # every other node: the value that loses most, in all channels
    q[..., 77] = 2.0 ** above / 4
    q = torch.from_numpy(q).to(torch.bfloat16)
    out, lse = _attend(c, q, mask)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    k, v = c.values()
    size = attention_bounds(q.double().numpy(), k, np.abs(v), c.table, c.lens, mask, scale, True)[0]
    dE = np.zeros(ref_lse.shape)
    for b, L in enumerate(lens):
        pos = np.arange(L + m)
        most = np.abs(k[c.table[b, pos // bs], :, pos % bs]).sum(2).max(0)                       # [Hkv]
        dE[b] = scale * 2.0 ** -21 * np.abs(q[b].double().numpy()).max(2) * np.repeat(most, Hq // Hkv)
    assert dE.max() < 1 / 4                                    # (first order in dE)
    assert_within(lse, ref_lse, bl + 1.5 * dE, "lse")
    assert_within(out, ref, bo + 3 * dE[..., None] * size, "out")
