"""Tree attention over the 8-bit cache at its edges: what must not be read, what must not be written, and what is refused."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import Cache, F8, assert_within, attention_bounds, ints, tree_mask, words
from gpu_helpers import lib
from oracle import kv_fp8 as o8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    lib()


# the forms of the kernel: (dtype, m, Hq, Hkv, d, bs, sb); up to 16, 32 and any number of rows per KV head, and fp32
FORMS = dict(rows16=(torch.bfloat16, 4, 4, 2, 128, 16, 16), rows32=(torch.bfloat16, 8, 8, 2, 128, 32, 8),
             wide=(torch.bfloat16, 33, 8, 2, 128, 16, 16), wide_fine=(torch.bfloat16, 40, 4, 1, 128, 64, 4),
             fp32=(torch.float32, 5, 4, 2, 64, 16, 8))
forms = pytest.mark.parametrize("form", FORMS.values(), ids=FORMS.keys())


def _query(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape) * np.exp2(rng.integers(-2, 2, shape[:-1] + (1,)))).to(dtype)


def _attend(dev, c, q, mask, top=None, ok=True, **kw):
    status = ts.new_status()
    r = ts.tree_attention_fp8(q.cuda(), *dev, ints(c.table), ints(c.lens), words(mask),
                              max_prefix=int(c.lens.max()) if top is None else top, status=status, **kw)
    if ok:
        ts.check_status(status)
    else:
        with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
            ts.check_status(status)
    return r


def _reference(c, q, mask):
    return attention_bounds(q.double().numpy(), *c.values(), c.table, c.lens, mask, 1 / math.sqrt(q.shape[-1]), q.dtype == torch.bfloat16)


def _row(c, b, pos):
    return c.table[b, pos // c.bs], slice(None), pos % c.bs


@forms
def test_nothing_unattended_is_read(form):
    """NaN codes behind the sequences, in free pages and in tree rows that no node attends to; scales of every kind there."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m)
    lens = (0, 3, 300, 2 * bs, 129)
    c = Cache(rng, lens, m, Hkv, d, bs, sb, spare=5)
    mask = tree_mask(rng, len(lens), m)
    mask[:, :, m // 2] = False
    bad = [x.copy() for x in c.codes]
    scales = [x.copy() for x in c.scales]
    for x, byte in zip(bad, (0x7F, 0xFF)):
        x[c.spare] = byte
        for b, L in enumerate(lens):
            x[_row(c, b, L + m // 2)] = byte
            last = L + m - 1
            x[c.table[b, last // bs], :, last % bs + 1:] = byte
    for s, value in zip(scales, (float("nan"), float("inf"))):
        s[c.spare] = value
        for b, L in enumerate(lens):
            s[c.table[b, (L + m - 1) // bs], :, (L + m - 1) % bs // sb + 1:] = value
    q = _query(rng, (len(lens), m, Hq, d), dtype)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    c.codes, c.scales = bad, scales
    out, lse = _attend(c.device(), c, q, mask)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")
    first = [b for b, L in enumerate(lens) if L == 0]
    for b in first:                                            # nothing at all to attend to: zero, and no sum
        empty = ~mask[b].any(1)
        assert (out[b].cpu()[empty] == 0).all() and (lse[b].cpu()[empty] == -math.inf).all()


@forms
def test_attended_nan_reaches_its_rows_alone(form):
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 1)
    lens, g = (140, 0, 37, 500), Hq // Hkv
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    mask = tree_mask(rng, 4, m)
    q = _query(rng, (4, m, Hq, d), dtype)
    q *= 1 / 16                                                # (so that no weight vanishes)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    j = m - 2
    head = Hkv - 1
    heads = slice(head * g, (head + 1) * g)
    c.codes[1][c.table[0, (140 + j) // bs], head, (140 + j) % bs, [3, 60]] = 0x7F       # V of a node: those columns
    ref[0, mask[0][:, j], heads, 3] = ref[0, mask[0][:, j], heads, 60] = np.nan
    c.codes[0][c.table[1, j // bs], head, j % bs, 9] = 0xFF                             # K of a node: the rows that see it
    ref[1, mask[1][:, j], heads] = np.nan
    ref_lse[1, mask[1][:, j], heads] = np.nan
    c.codes[1][c.table[2, 20 // bs], 0, 20 % bs, d - 1] = 0xFF                          # V of the prefix: a column of every row
    ref[2, :, :g, d - 1] = np.nan
    c.codes[0][c.table[3, 400 // bs], 0, 400 % bs, 0] = 0x7F                            # K of the prefix: every row
    ref[3, :, :g] = np.nan
    ref_lse[3, :, :g] = np.nan
    out, lse = _attend(c.device(), c, q, mask)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@forms
def test_queries_of_every_size_side_by_side(form):
    """Rows that are zero, subnormal, huge, infinite or NaN beside ordinary ones, which stay as they are."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 2)
    lens = (100, 1, 260)
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    mask = tree_mask(rng, 3, m)
    q = _query(rng, (3, m, Hq, d), dtype)
    q[0, 0, 0] = 0.0
    q[0, 1, 0] *= 2.0 ** -120
    q[0, 2, 1] *= 2.0 ** -133                                  # (subnormal)
    q[1, 0, 1] *= 2.0 ** 20
    q[1, 2, 0, 1:] = 0.0                                       # one element alone, and one far above the others
    q[1, 3, 0, 0] = 2.0 ** 12
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    q[2, 0, 0, 5], q[2, 1, 0, 6], q[2, 2, 0] = float("nan"), float("inf"), -float("inf")
    for i in range(3):
        ref[2, i, 0] = ref_lse[2, i, 0] = np.nan
    out, lse = _attend(c.device(), c, q, mask)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@forms
def test_scales_of_any_kind_are_read_clamped(form):
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 3)
    lens = (200, 64)
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    for s, odd in zip(c.scales, ((0.013, 1e-30, 0.0, -3.0, float("nan")), (0.3, 7.7, 1e-45, 100.0, -float("inf")))):
        at = rng.random(s.shape) < 0.4
        s[at] = rng.choice(np.array(odd, dtype=np.float32), at.sum())
    mask = tree_mask(rng, 2, m)
    q = _query(rng, (2, m, Hq, d), dtype)
    out, lse = _attend(c.device(), c, q, mask)
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")


@forms
def test_device_checks(form):
    """Pages out of range: their keys are left out.  Lengths out of range: the sequence's rows are left as they were."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 4)
    lens = (5 * bs + 3, 300, 40, 200)
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    mask = tree_mask(rng, 4, m)
    q = _query(rng, (4, m, Hq, d), dtype)
    whole, table, top = c.lens.copy(), c.table.copy(), int(c.lens.max())
    # the reference: without the page (the order of keys does not matter)
    c.table[0, 2:-1] = table[0, 3:]
    c.lens[0] -= bs
    ref, ref_lse, bo, bl = _reference(c, q, mask)
    for wrong in (-1, c.codes[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table, c.lens = table.copy(), whole.copy()
        c.table[0, 2] = wrong
        c.lens[1], c.lens[2] = -1, top + 1
        out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        _attend(c.device(), c, q, mask, top=top, ok=False, out=out, lse=lse)
        for b in (0, 3):
            assert_within(lse[b], ref_lse[b], bl[b], "lse")
            assert_within(out[b], ref[b], bo[b], "out")
        assert (out[1:3] == 7).all() and (lse[1:3] == 7).all()
    c.table, c.lens = table.copy(), whole.copy()
    c.lens[3] = table.shape[1] * bs - m + 1                    # no room for the tree
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    _attend(c.device(), c, q, mask, top=table.shape[1] * bs, ok=False, out=out, with_lse=False)
    assert (out[3] == 7).all() and not (out[:3] == 7).all()


@pytest.mark.parametrize("form", [FORMS[n] for n in ("rows16", "rows32", "wide", "wide_fine")], ids=["rows16", "rows32", "wide", "wide_fine"])
def test_many_short_and_a_few_long_sequences(form):
    """Several sequences per CTA, several CTAs per sequence."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    for B, most in ((150, 700), (3, 60000)):
        rng = np.random.default_rng(B)
        lens = rng.integers(0, most, size=B)
        lens[0], lens[B // 2] = 0, most
        Hk, g = 1, Hq // Hkv
        c = Cache(rng, lens, m, Hk, d, bs, sb)
        mask = tree_mask(rng, B, m)
        q = _query(rng, (B, m, g, d), dtype)
        out, lse = _attend(c.device(), c, q, mask)
        ref, ref_lse, bo, bl = _reference(c, q, mask)
        assert_within(lse, ref_lse, bl, "lse")
        assert_within(out, ref, bo, "out")


@forms
def test_given_outputs_and_workspace(form):
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 5)
    c = Cache(rng, (900, 70), m, Hkv, d, bs, sb)
    mask, q, dev = tree_mask(rng, 2, m), _query(rng, (2, m, Hq, d), dtype), c.device()
    want, want_lse = _attend(dev, c, q, mask)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    got = _attend(dev, c, q, mask, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, want_lse)
    got = _attend(dev, c, q, mask, with_lse=False)
    assert got[1] is None and torch.equal(got[0], want)
    need = ts.library().ts_tree_attention_fp8_workspace(int(dtype == torch.bfloat16), 2, m, Hq, Hkv, d, 900, bs)
    assert need > 256
    short = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises((ValueError, ts.TreeSpecError), match="workspace|WORKSPACE"):
        _attend(dev, c, q, mask, workspace=short)
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        _attend(dev, c, q, mask, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:])
    # a larger bound of the lengths changes the split at most
    again, _ = _attend(dev, c, q, mask, top=(c.table.shape[1] * bs))
    ref, _, bo, _ = _reference(c, q, mask)
    assert_within(again, ref, bo, "out")


def test_refusals():
    rng = np.random.default_rng(6)
    c = Cache(rng, (90,), 4, 2, 128, 16, 16)
    q = _query(rng, (1, 4, 4, 128), torch.bfloat16).cuda()
    dev, mask = c.device(), words(tree_mask(rng, 1, 4))
    good = (q, *dev, ints(c.table), ints([90]), mask)

    def call(i=None, x=None, **kw):
        a = list(good)
        if i is not None:
            a[i] = x
        kw.setdefault("max_prefix", 90)
        return ts.tree_attention_fp8(*a, **kw)

    for i, x, why in ((0, q.half(), "dtype"), (0, q.cpu(), "CUDA"), (0, q[0], "dimensions"), (0, q.transpose(1, 2), "contiguous"),
                      (0, q[..., :64].contiguous(), "match"), (1, dev[0].view(torch.uint8), "float8"), (2, dev[1][:3], "shape"),
                      (3, dev[2].half(), "float32"), (4, dev[3][:, :1].contiguous(), "shape"), (5, ints(c.table).long(), "int32"),
                      (6, ints([90, 90]), "shape"), (7, mask[:, :3].contiguous(), "shape"), (7, mask.int(), "int64")):
        with pytest.raises(ValueError, match=why):
            call(i, x)
    for kw in (dict(max_prefix=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=q)):
        with pytest.raises(ts.TreeSpecError):
            call(**kw)
    with pytest.raises(ValueError, match="shape"):
        call(out=torch.empty(1, 4, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="float32"):
        call(lse=torch.empty(1, 4, 4, dtype=torch.bfloat16, device="cuda"))
    # the tensor-core form copies rows of 16 bytes
    buf = torch.zeros(dev[0].numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(F8).view(dev[0].shape)
    for i in (1, 2):
        with pytest.raises(ts.TreeSpecError, match="INVALID"):
            call(i, buf)
    c.assert_equal(dev)


@pytest.mark.parametrize("d,dtype", [(64, torch.float32), (128, torch.float32), (64, torch.bfloat16)])
def test_cuda_cores_take_any_alignment(d, dtype):
    rng = np.random.default_rng(7)
    c = Cache(rng, (333, 20), 5, 2, d, 16, 8)
    mask, q = tree_mask(rng, 2, 5), _query(rng, (2, 5, 4, d), dtype)
    dev = c.device()
    want = _attend(dev, c, q, mask)
    for off in (1, 4, 8):
        moved = list(dev)
        for i in (0, 1):
            buf = torch.empty(dev[i].numel() + off, dtype=torch.uint8, device="cuda")[off:]
            buf.copy_(dev[i].view(torch.uint8).flatten())
            moved[i] = buf.view(F8).view(dev[i].shape)
        for i in (2, 3):
            moved[i] = torch.cat([dev[i].flatten()[:1], dev[i].flatten()])[1:].view(dev[i].shape)
        got = _attend(moved, c, q, mask)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,m", [(torch.bfloat16, 3), (torch.bfloat16, 70), (torch.float32, 3)])
def test_pages_beyond_32_bits(dtype, m):
    """The last pages of a cache of more than 2^32 bytes: all four calls give what they give on a small one."""
    rng = np.random.default_rng(m)
    Hkv, d, bs, sb, far = 8, 128, 128, 16, 33000
    c = Cache(rng, (300, 20, 129), m, Hkv, d, bs, sb)
    small, nb = c.device(), c.codes[0].shape[0]
    large = [torch.empty((far, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in small]
    first = far - nb
    for s, t in zip(small, large):
        t[first:].view(torch.uint8).copy_(s.view(torch.uint8))
    assert first * Hkv * bs * d > 2 ** 32
    prefix, mask = ints(c.lens), words(tree_mask(rng, 3, m))
    k, v = [_query(rng, (3, m, Hkv, d), dtype).cuda() for _ in "kv"]
    q = _query(rng, (3, m, 16, d), dtype).cuda()
    path = np.full((3, m), -1, dtype=np.int32)
    path[:, :2] = [0, m - 1]
    results = []
    for dev, shift in ((small, 0), (large, first)):
        table, status = ints(np.where(c.table >= 0, c.table + shift, -1)), ts.new_status()
        ts.kv_write_fp8(k, v, *dev, table, prefix, status=status)
        out, lse = ts.tree_attention_fp8(q, *dev, table, prefix, mask, max_prefix=300, status=status)
        r = ts.kv_commit_fp8(*dev, table, prefix, ints(path), ints([2, 1, 2]), status=status)
        kr, vr = ts.kv_read_fp8(*dev, r["block_table"], r["prefix_len"], 302, dtype=torch.float32, status=status)
        ts.check_status(status)
        results.append((out, lse, kr, vr, *(t[shift:].view(torch.uint8) for t in dev)))
    for a, b in zip(*results):
        assert torch.equal(a, b)


@forms
def test_scores_that_fp32_cannot_tell_apart(form):
    """Beyond 2^22 (base 2) the tensor cores' rows become NaN; below, and in fp32, they are as exact as their scores."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 6)
    c = Cache(rng, (300, 40), m, Hkv, d, bs, sb)
    mask = tree_mask(rng, 2, m)
    seen = set()
    for e in (17, 20, 22, 30, 60):
        q = _query(rng, (2, m, Hq, d), dtype) * 2.0 ** e
        out, lse = _attend(c.device(), c, q, mask)
        ref, ref_lse, bo, bl = _reference(c, q, mask)
        high = np.abs(ref_lse) * math.log2(math.e)
        far = (high > 1.01 * 2 ** 22) & (dtype == torch.bfloat16)
        near = (high < 0.99 * 2 ** 22) | (dtype == torch.float32)
        seen |= {bool(x) for x in far.flatten()}
        assert torch.isnan(lse.cpu()[torch.from_numpy(far)]).all() and torch.isnan(out.cpu()[torch.from_numpy(far)]).all()
        nan = np.where(near, 0.0, np.nan)                      # (rows in between are not looked at)
        keep = torch.from_numpy(nan).to(out.device)
        assert_within(lse + keep, ref_lse + nan, bl, "lse")
        assert_within(out + keep[..., None], ref + nan[..., None], bo, "out")
    assert seen == ({True, False} if dtype == torch.bfloat16 else {False})


@forms
def test_no_sequence_can_be_read(form):
    dtype, m, Hq, Hkv, d, bs, sb = form
    rng = np.random.default_rng(m + 7)
    c = Cache(rng, (90, 5), m, Hkv, d, bs, sb)
    mask, q, dev = tree_mask(rng, 2, m), _query(rng, (2, m, Hq, d), dtype), c.device()
    c.lens[:] = -1, 2 ** 31 - 1
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    _attend(dev, c, q, mask, top=4000, ok=False, out=out)
    assert (out == 7).all()


@forms
def test_few_and_many_tiles_of_every_length(form):
    """Shares of a fraction of a tile to several units for a CTA, sequences of one tile between longer ones."""
    dtype, m, Hq, Hkv, d, bs, sb = form
    for lens in ((0,), (700,), (3000,), (0, 0, 900), (1, 130, 0, 2000, 5), tuple(range(0, 40)), (0, 500) * 20):
        rng = np.random.default_rng(len(lens))
        c = Cache(rng, lens, m, Hkv, d, bs, sb)
        mask, q = tree_mask(rng, len(lens), m), _query(rng, (len(lens), m, Hq, d), dtype)
        out, lse = _attend(c.device(), c, q, mask)
        ref, ref_lse, bo, bl = _reference(c, q, mask)
        assert_within(lse, ref_lse, bl, "lse")
        assert_within(out, ref, bo, "out")
