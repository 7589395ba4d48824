"""GPU tree_attention_sparse vs the fp64 oracle, on both paths.

Tolerances, per output element, with S = sum_j p_j |v_j| (from the oracle):
  bf16: the weights are rounded to bf16 once (half a step, 2^-8) before they meet V, the result once
    more: 2^-8 (S + |out|).  The fp32 steps (scores of d products, the exponentials, sums) are three orders
    finer: 2^-12 S.
  fp32: N keys are added in sequence (N 2^-24), each weight carries the error of its score (d / 32 products per
    lane and five shuffle sums: 13 roundings of at most 2^-24 X, X = max_j scale |q||k|, twice: numerator
    and sum) and of two exponentials (2 ulp each): (2 N + 40 X + 16) 2^-24 S.
  lse: the scores' error with the tensor cores' sums taken as 128 roundings, and the logarithm's:
    (128 X + 4 (|lse| + N)) 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu


def _case(seed, L, m, Hq, Hkv, d, bs, dtype, n=None, spread=1.0, empty_rows=()):
    """q, caches, table, mask and kept pages; n pages per node (None: every complete page)."""
    rng = np.random.default_rng(seed)
    B = len(L)
    need = [-(-(x + m) // bs) for x in L]
    nb, width = sum(need) + 2, max(need) + 1
    perm, table, at = rng.permutation(nb), np.full((B, width), -1, dtype=np.int32), 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, m, Hq, d, generator=g) * spread).to(dtype)
    k, v = [torch.randn(nb, Hkv, bs, d, generator=g).to(dtype) for _ in range(2)]
    mask = np.zeros((B, m, m), dtype=bool)
    for b in range(B):
        parent = [-1] + [int(rng.integers(0, i)) for i in range(1, m)]
        for i in range(m):
            j = i
            while j >= 0:
                mask[b, i, j] = True
                j = parent[j]
        for i in empty_rows:
            mask[b, i] = False
    C = max(1, max(x // bs for x in L)) + 2
    kept = np.zeros((B, Hkv, m, C), dtype=bool)
    for b in range(B):
        nf = L[b] // bs
        for h in range(Hkv):
            for i in range(m):
                if i in empty_rows:
                    continue
                kept[b, h, i, rng.permutation(nf)[:nf if n is None else n]] = True
    return q, k, v, table, mask, kept


def _run(q, k, v, table, L, mask, kept, **kw):
    from oracle.page_select import pack
    m = q.shape[1]
    pages, count, words = pack(kept, (m + 63) // 64)
    mw = np.stack([oracle.mask_to_words(x) for x in mask])
    sel = dict(pages=torch.from_numpy(pages).to(dev()), count=torch.from_numpy(count).to(dev()),
               node_mask=torch.from_numpy(words.view(np.int64)).to(dev()))
    args = [x.to(dev()) for x in (q, k, v, torch.from_numpy(table))]
    return ts.tree_attention_sparse(*args, torch.tensor(L, dtype=torch.int32, device=dev()),
                                    torch.from_numpy(mw.view(np.int64)).to(dev()), sel, **kw)


def _check(q, k, v, table, L, mask, kept, out, lse, scale=None):
    d = q.shape[-1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    ref, rl, spread = oracle.tree_attention_sparse(q, k, v, table, L, mask, kept, scale)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    N = max(L) + q.shape[1]
    X = scale * float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max())
    if q.dtype == torch.bfloat16 and d == 128:
        tol = 2.0 ** -8 * (spread + np.abs(ref)) + 2.0 ** -12 * spread
    else:
        tol = (2 * N + 40 * X + 16) * 2.0 ** -24 * spread
        if q.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} out of tolerance, worst by {over.max()}"
    none = np.isneginf(rl)
    assert (np.isneginf(gl) == none).all() and (got[none] == 0).all()
    ltol = (128 * X + 4 * (np.abs(np.where(none, 0, rl)) + N)) * 2.0 ** -24
    assert (np.abs(np.where(none, 0, gl) - np.where(none, 0, rl)) <= ltol).all()


BF, F32 = torch.bfloat16, torch.float32
CASES = [dict(L=[300], m=7, Hq=4, Hkv=1, d=128, bs=16, dtype=BF, n=5),
         dict(L=[1, 0, 15, 16, 17], m=1, Hq=8, Hkv=2, d=128, bs=16, dtype=BF, n=1),
         dict(L=[700, 33], m=60, Hq=16, Hkv=2, d=128, bs=16, dtype=BF, n=9),               # four row groups
         dict(L=[520, 0], m=40, Hq=6, Hkv=2, d=128, bs=32, dtype=BF, n=3),                 # groups of three heads
         dict(L=[900], m=130, Hq=2, Hkv=2, d=128, bs=64, dtype=BF, n=4),                   # more than two mask words
         dict(L=[1000, 250], m=9, Hq=7, Hkv=1, d=128, bs=128, dtype=BF, n=2),
         dict(L=[640], m=256, Hq=1, Hkv=1, d=128, bs=16, dtype=BF, n=4),
         dict(L=[2000], m=3, Hq=4, Hkv=2, d=128, bs=16, dtype=BF, n=None),
         dict(L=[129], m=4, Hq=2, Hkv=1, d=128, bs=16, dtype=BF, n=0),
         dict(L=[100, 7], m=5, Hq=4, Hkv=2, d=64, bs=16, dtype=BF, n=3),                   # CUDA-core path
         dict(L=[100, 0, 41], m=6, Hq=6, Hkv=2, d=128, bs=16, dtype=F32, n=3),
         dict(L=[75], m=70, Hq=2, Hkv=1, d=37, bs=5, dtype=F32, n=6),
         dict(L=[64], m=2, Hq=3, Hkv=3, d=256, bs=8, dtype=F32, n=None),
         dict(L=[333], m=1, Hq=14, Hkv=2, d=64, bs=16, dtype=F32, n=7)]
_id = lambda c: f"L{c['L'][0]}_m{c['m']}_{c['Hq']}x{c['Hkv']}_d{c['d']}_bs{c['bs']}_{str(c['dtype'])[6:]}"


@pytest.mark.parametrize("c", CASES, ids=_id)
def test_matches_the_oracle(c):
    lib()
    x = _case(1, **c)
    status = ts.new_status(dev())
    out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5], status=status)
    ts.check_status(status)
    _check(*x[:4], c["L"], *x[4:], out, lse)


@pytest.mark.parametrize("split", ["direct", "cluster:2", "cluster:4", "cluster:8", "global:2", "global:3", "global:7"])
def test_every_split(split, monkeypatch):
    lib()
    monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    for c in (CASES[2], CASES[7], dict(L=[3000, 200], m=33, Hq=8, Hkv=2, d=128, bs=16, dtype=BF, n=20)):
        x = _case(2, **c)
        status = ts.new_status(dev())
        out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5], status=status)
        ts.check_status(status)
        _check(*x[:4], c["L"], *x[4:], out, lse)


@pytest.mark.parametrize("c", [CASES[2], CASES[10]], ids=_id)
def test_rows_without_keys(c):
    """Padding nodes: no page, no ancestor; with an empty incomplete page they have no key at all."""
    lib()
    c = dict(c, L=[x // c["bs"] * c["bs"] for x in c["L"]])
    x = _case(3, empty_rows=(0, c["m"] - 1), **c)
    out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5])
    _check(*x[:4], c["L"], *x[4:], out, lse)
    assert torch.isneginf(lse[:, 0]).all() and (out[:, -1] == 0).all()


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_flat_and_sharp_scores(spread):
    lib()
    c = CASES[2]
    x = _case(4, spread=spread, **c)
    out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5])
    if spread == 0.0:
        _check(*x[:4], c["L"], *x[4:], out, lse)
    else:
        # a score's own fp32 error grows with it: |q||k| scale reaches 30 * 128 / sqrt(128) = 340, so the weights
        # carry up to 2 * 128 * 340 * 2^-24 = 2^-7.6 on top
        ref, _, s = oracle.tree_attention_sparse(x[0], x[1], x[2], x[3], c["L"], x[4], x[5], 1 / math.sqrt(128))
        assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -8 * (s + np.abs(ref)) + 2.0 ** -7 * s).all()


@pytest.mark.parametrize("split", ["direct", "cluster:4", "global:3"])
@pytest.mark.parametrize("c", [CASES[2], dict(CASES[10], L=[100, 48, 41])], ids=_id)
def test_non_finite_values_in_places_not_attended_to(c, split, monkeypatch):
    """NaN and infinities in pages that a node does not keep, in other branches of the tree, and behind the
    last node reach nobody who does not attend to them; who does sees them."""
    lib()
    monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    L, m, bs = c["L"], c["m"], c["bs"]
    q, k, v, table, mask, kept = _case(5, **c)
    clean = (q, k.clone(), v.clone())
    page = int(np.nonzero(kept[0, 0, 1])[0][0])
    hit = np.zeros((len(L), m, q.shape[2]), dtype=bool)
    g = q.shape[2] // k.shape[1]
    for cache, value in ((k, float("nan")), (v, float("inf")), (v, float("nan"))):
        k2, v2 = clean[1].clone(), clean[2].clone()
        dst = k2 if cache is k else v2
        dst[table[0, page], 0, 3, 5] = value                              # a page that some nodes keep
        node = m - 2
        pos = L[1] + node
        dst[table[1, pos // bs], :, pos % bs, 7] = value                  # a tree node of the second sequence
        hit[:] = False
        for i in range(m):
            hit[0, i, :g] = kept[0, 0, i, page]
            hit[1, i] = mask[1, i, node]
        for b in range(len(L)):                                           # behind the last node, and unused pages
            for pos in range(L[b] + m, -(-(L[b] + m) // bs) * bs):
                k2[table[b, pos // bs], :, pos % bs] = float("nan")
                v2[table[b, pos // bs], :, pos % bs] = float("nan")
        free = np.setdiff1d(np.arange(k.shape[0]), table)
        k2[free], v2[free] = float("nan"), float("nan")
        out, lse = _run(q, k2, v2, table, L, mask, kept)
        good, glse = _run(*clean, table, L, mask, kept)
        assert hit.any() and not hit.all()
        assert not torch.isfinite(out.cpu()[torch.from_numpy(hit)]).all(-1).any()
        # the rows that were computed again one key at a time differ from the tensor cores' by both roundings
        ref, rl, s = oracle.tree_attention_sparse(*clean, table, L, mask, kept, 1 / math.sqrt(q.shape[-1]))
        got = out.double().cpu().numpy()[~hit]
        assert np.isfinite(got).all()
        assert (np.abs(got - ref[~hit]) <= (2.0 ** -8 * (s + np.abs(ref)) + 2.0 ** -12 * s)[~hit]).all()
        assert torch.isfinite(lse.cpu()[torch.from_numpy(~hit)]).all()


def test_every_page_kept_agrees_with_dense_attention():
    lib()
    c = dict(L=[1500, 700], m=30, Hq=8, Hkv=2, d=128, bs=16, dtype=BF)
    x = _case(6, **c)
    out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5])
    mw = np.stack([oracle.mask_to_words(y) for y in x[4]])
    dense, dl = ts.tree_attention(*[t.to(dev()) for t in (x[0], x[1], x[2], torch.from_numpy(x[3]))],
                                  torch.tensor(c["L"], dtype=torch.int32, device=dev()),
                                  torch.from_numpy(mw.view(np.int64)).to(dev()), max_prefix=1500)
    _, _, s = oracle.tree_attention_sparse(*x[:4], c["L"], *x[4:], 1 / math.sqrt(128))
    # both carry the same kinds of roundings, in different places
    diff = (out.double() - dense.double()).abs().cpu().numpy()
    assert (diff <= 2 * (2.0 ** -8 * (s + dense.double().abs().cpu().numpy()) + 2.0 ** -12 * s)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", ["count", "count_low", "page", "page_low", "prefix", "prefix_low", "entry"])
def test_bad_state_is_reported(case, dtype):
    lib()
    c = dict(L=[100, 70], m=4, Hq=4, Hkv=2, d=128, bs=16, dtype=dtype, n=3)
    q, k, v, table, mask, kept = _case(7, **c)
    from oracle.page_select import pack
    pages, count, words = pack(kept, 1)
    L = list(c["L"])
    if case == "count":
        count[0, 0] = pages.shape[-1] + 1
    elif case == "count_low":
        count[0, 0] = -1
    elif case == "page":
        pages[0, 0, 0] = 6
    elif case == "page_low":
        pages[0, 0, 0] = -1
    elif case == "prefix":
        L[0] = table.shape[1] * 16 - 3
    elif case == "prefix_low":
        L[0] = -1
    else:
        table[0, pages[0, 0, 0]] = k.shape[0]
    mw = np.stack([oracle.mask_to_words(x) for x in mask])
    status = ts.new_status(dev())
    t = lambda x: torch.from_numpy(x).to(dev())
    out, _ = ts.tree_attention_sparse(q.to(dev()), k.to(dev()), v.to(dev()), t(table),
                                      torch.tensor(L, dtype=torch.int32, device=dev()), t(mw.view(np.int64)),
                                      dict(pages=t(pages), count=t(count), node_mask=t(words.view(np.int64))), status=status)
    assert int(status.item()) == -6
    ref, _, s = oracle.tree_attention_sparse(q, k, v, np.maximum(np.minimum(table, k.shape[0] - 1), 0), c["L"], mask, kept,
                                             1 / math.sqrt(128))
    got = out.double().cpu().numpy()
    assert (np.abs(got[1] - ref[1]) <= 2.0 ** -8 * (s[1] + np.abs(ref[1])) + 2.0 ** -12 * s[1]).all()  # the other sequence


def test_refusals():
    lib()
    c = CASES[0]
    q, k, v, table, mask, kept = _case(8, **c)
    run = lambda **kw: _run(*[kw.get(n, x) for n, x in (("q", q), ("k", k), ("v", v), ("table", table))], c["L"],
                            kw.get("mask", mask), kw.get("kept", kept))
    run()
    for kw in (dict(k=k.float()), dict(v=v[:-1]), dict(q=q[..., :64].contiguous()), dict(mask=mask[:, :-1, :-1]),
               dict(kept=kept[:, :, :, :].repeat(2, 1))):
        with pytest.raises(ValueError):
            run(**kw)
    with pytest.raises(ValueError):
        run(table=table.astype(np.int64))


def test_fp32_tensors_off_the_allocations_alignment():
    lib()
    c = dict(L=[100, 48], m=6, Hq=6, Hkv=2, d=128, bs=16, dtype=F32, n=3)
    x = _case(12, **c)

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:].copy_(t.reshape(-1).to(dev()))
        return flat[1:].view(t.shape)

    from oracle.page_select import pack
    pages, count, words = pack(x[5], 1)
    t = lambda a: torch.from_numpy(a).to(dev())
    sel = dict(pages=t(pages), count=t(count), node_mask=t(words.view(np.int64)))
    mw = np.stack([oracle.mask_to_words(y) for y in x[4]])
    out, lse = ts.tree_attention_sparse(off(x[0]), off(x[1]), off(x[2]), t(x[3]),
                                        torch.tensor(c["L"], dtype=torch.int32, device=dev()), t(mw.view(np.int64)), sel)
    _check(*x[:4], c["L"], *x[4:], out, lse)


def _tolerance(q, k, L, ref, spread):
    """The tolerance of the outputs (see the top) for finite q and k."""
    if q.dtype == torch.bfloat16 and q.shape[-1] == 128:
        return 2.0 ** -8 * (spread + np.abs(ref)) + 2.0 ** -12 * spread
    X = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) / math.sqrt(q.shape[-1])
    tol = (2 * (max(L) + q.shape[1]) + 40 * X + 16) * 2.0 ** -24 * spread
    return tol + 2.0 ** -8 * np.abs(ref) if q.dtype == torch.bfloat16 else tol


def _check_attended_nan(c, where):
    """A NaN among the scores of the keys that a row attends to makes its output and sum NaN, wherever it stands; the
    other rows are as without it."""
    q, k, v, table, mask, kept = _case(13, **c)
    q2, k2 = q.clone(), k.clone()
    B, m, Hq, d = q.shape
    g = Hq // k.shape[1]
    hit = np.zeros((B, m, Hq), dtype=bool)
    if where == "query":                                   # every score of one row
        q2[0, m // 2, 1, 3] = float("nan")
        hit[0, m // 2, 1] = True
    else:                                                  # one page that nodes of the first sequence keep
        pages = np.nonzero(kept[0, 0].any(0))[0]
        page = pages[0] if where == "first_key" else pages[len(pages) // 2]
        rows = slice(0, 1) if where == "first_key" else slice(None)
        k2[table[0, page], 0, rows] = float("nan")
        hit[0, :, :g] = kept[0, 0, :, page, None]
    out, lse = _run(q2, k2, v, table, c["L"], mask, kept)
    ref, rl, spread = oracle.tree_attention_sparse(q, k, v, table, c["L"], mask, kept, 1 / math.sqrt(d))
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert hit.any()
    assert np.isnan(got[hit]).all() and np.isnan(gl[hit]).all()
    assert (np.abs(got - ref) <= _tolerance(q, k, c["L"], ref, spread))[~hit].all()
    assert np.isfinite(gl[~hit]).all()


@pytest.mark.parametrize("where", ["query", "page", "first_key"])
@pytest.mark.parametrize("split", ["direct", "cluster:4", "global:3"])
@pytest.mark.parametrize("c", [CASES[0], CASES[2], CASES[7], dict(CASES[7], m=1)], ids=_id)
def test_nan_scores_on_the_tensor_cores(c, split, where, monkeypatch):
    lib()
    monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    _check_attended_nan(c, where)


@pytest.mark.parametrize("where", ["query", "page", "first_key"])
@pytest.mark.parametrize("c", [CASES[9], CASES[10], CASES[11], CASES[12], CASES[13], dict(CASES[13], Hq=2)], ids=_id)
def test_nan_scores_on_the_cuda_cores(c, where):
    """Few nodes are spread over clusters of up to eight CTAs, whose warps may then have no other key than NaN ones."""
    lib()
    _check_attended_nan(c, where)


@pytest.mark.parametrize("split", ["direct", "cluster:4", "global:3"])
@pytest.mark.parametrize("case", ["page", "page_low", "entry", "tail", "tree"])
@pytest.mark.parametrize("dtype,bs", [(BF, 16), (BF, 32), (BF, 128), (F32, 16)])
def test_keys_of_a_page_without_an_id_are_left_out(dtype, bs, case, split, monkeypatch):
    """A chosen page that the prefix does not complete, or a table entry out of range, is reported, and the rows of
    the same sequence attend to their other keys."""
    lib()
    monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    L, m = [6 * bs + 5, 4 * bs], 5 if case != "tree" else bs + 3
    q, k, v, table, mask, kept = _case(14, L=L, m=m, Hq=4, Hkv=2, d=128, bs=bs, dtype=dtype, n=3)
    from oracle.page_select import pack
    pages, count, words = pack(kept, (m + 63) // 64)
    B, Hkv, nb = 2, 2, k.shape[0]
    # the same state as pages of one token: kept1 over the prefix, the mask over the tree
    longest = max(L)
    flat = [x.permute(0, 2, 1, 3).reshape(nb * bs, Hkv, 1, 128) for x in (k, v)]
    ids = (np.maximum(table, 0)[:, :, None] * bs + np.arange(bs)).reshape(B, -1)
    kept1 = np.zeros((B, Hkv, m, longest), dtype=bool)
    for b in range(B):
        nf = L[b] // bs
        kept1[b, :, :, :nf * bs] = np.repeat(kept[b, :, :, :nf], bs, 2)
        kept1[b, :, :, nf * bs:L[b]] = True
    mask1 = mask.copy()
    page = int(pages[0, 0, 1])
    if case in ("page", "page_low"):
        pages[0, 0, 1] = 6 if case == "page" else -1
        kept1[0, 0, :, page * bs:(page + 1) * bs] = False
    else:
        at = page if case == "entry" else 6 if case == "tail" else 7
        table[0, at] = nb if case != "tree" else -1
        kept1[0, :, :, at * bs:(at + 1) * bs] = False
        lost = np.arange(at * bs, (at + 1) * bs) - L[0]
        mask1[0][:, lost[(lost >= 0) & (lost < m)]] = False
    mw = np.stack([oracle.mask_to_words(x) for x in mask])
    t = lambda x: torch.from_numpy(x).to(dev())
    status = ts.new_status(dev())
    out, lse = ts.tree_attention_sparse(q.to(dev()), k.to(dev()), v.to(dev()), t(table),
                                        torch.tensor(L, dtype=torch.int32, device=dev()), t(mw.view(np.int64)),
                                        dict(pages=t(pages), count=t(count), node_mask=t(words.view(np.int64))), status=status)
    assert int(status.item()) == -6
    ref, rl, spread = oracle.tree_attention_sparse(q, *flat, ids, L, mask1, kept1, 1 / math.sqrt(128))
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(got - ref) <= _tolerance(q, k, L, ref, spread)).all()
    X = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) / math.sqrt(128)
    assert (np.abs(gl - rl) <= (128 * X + 4 * (np.abs(rl) + longest + m)) * 2.0 ** -24).all()


@pytest.mark.parametrize("split,B", [("", 80), ("direct", 2), ("cluster:2", 2), ("global:5", 2)])
def test_unions_longer_than_a_cta_stages(split, B, monkeypatch):
    """130 nodes of one head: a CTA stages the ids and bits of some 190 tiles, the capacity and the first sequence's
    union are of 205.  With 80 sequences the GPU is full without splitting, so only this limit splits."""
    lib()
    if split:
        monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    c = dict(L=[26000] + [40, 0, 3000, 16][:B - 1] + [25] * max(0, B - 5), m=130, Hq=1, Hkv=1, d=128, bs=16, dtype=BF, n=60)
    x = _case(15, **c)
    assert x[5][0, 0].any(0).sum() > 1550
    status = ts.new_status(dev())
    out, lse = _run(x[0], x[1], x[2], x[3], c["L"], x[4], x[5], status=status)
    ts.check_status(status)
    _check(*x[:4], c["L"], *x[4:], out, lse)


@pytest.mark.parametrize("split", ["direct", "cluster:2", "global:3"])
@pytest.mark.parametrize("c", [CASES[2], CASES[3], CASES[4], CASES[5], dict(CASES[7], m=1), CASES[10]], ids=_id)
def test_a_nan_value_reaches_its_channel_of_the_rows_that_attend_to_it(c, split, monkeypatch):
    """NaN in one channel of V, at a key of a page and at a tree node: that channel of the rows that attend to it, and
    nothing else."""
    lib()
    monkeypatch.setenv("TREESPEC_ATTN_SPLIT", split)
    q, k, v, table, mask, kept = _case(16, **c)
    L, (B, m, Hq, d), bs = c["L"], q.shape, c["bs"]
    g = Hq // k.shape[1]
    page, node, b1 = int(np.nonzero(kept[0, 0].any(0))[0][-1]), m // 2, len(L) - 1
    v2 = v.clone()
    v2[table[0, page], 0, bs - 2, 9] = float("nan")
    pos = L[b1] + node
    v2[table[b1, pos // bs], -1, pos % bs, 70] = float("nan")
    hit = np.zeros((B, m, Hq, d), dtype=bool)
    hit[0, :, :g, 9] = kept[0, 0, :, page, None]
    hit[b1, :, -g:, 70] |= mask[b1, :, node, None]
    status = ts.new_status(dev())
    out, lse = _run(q, k, v2, table, L, mask, kept, status=status)
    ts.check_status(status)
    ref, rl, spread = oracle.tree_attention_sparse(q, k, v, table, L, mask, kept, 1 / math.sqrt(d))
    got = out.double().cpu().numpy()
    assert np.isnan(got[hit]).all()
    assert (np.abs(got - ref) <= _tolerance(q, k, L, ref, spread))[~hit].all()
    X = float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) / math.sqrt(d)
    assert (np.abs(lse.double().cpu().numpy() - rl) <= (128 * X + 4 * (np.abs(rl) + max(L) + m)) * 2.0 ** -24).all()
