"""The page calls together, as a serving loop uses them: room is reserved, the tree's K/V are written, bounds kept,
pages chosen, attention computed, a path committed, sequences forked, reordered and dropped, and the pool
compacted, for many steps, against a plain record of what every sequence holds; and the same calls captured
into graphs, replayed, and run on two streams at once."""
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())


def _tree(rng, B, m):
    parents = np.full((B, m), -1, dtype=np.int64)
    mask = np.zeros((B, m, m), dtype=bool)
    for b in range(B):
        for i in range(m):
            parents[b, i] = -1 if i == 0 else rng.integers(max(0, i - 5), i)
            if i:
                mask[b, i] = mask[b, parents[b, i]]
            mask[b, i, i] = True
    words = np.stack([oracle.mask_to_words(x) for x in mask])
    return parents, mask, torch.from_numpy(words.view(np.int64)).to(dev())


def _counts(table, nb):
    return np.bincount(table[table >= 0], minlength=nb)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_serving_loop(dtype):
    lib()
    rng = np.random.default_rng(11)
    g = torch.Generator().manual_seed(11)
    Hq, Hkv, d, bs, nb, width, m = 4, 2, 128 if dtype == torch.bfloat16 else 64, 16, 120, 24, 9
    k = torch.zeros(nb, Hkv, bs, d, dtype=dtype, device=dev())
    v = torch.zeros_like(k)
    bounds = torch.zeros(nb, Hkv, 2, d, dtype=torch.bfloat16, device=dev())
    table, L, refs = _i32(np.full((3, width), -1)), _i32([0, 0, 0]), _i32([0] * nb)
    freed, told = None, [torch.zeros(0, 2, Hkv, d, dtype=dtype) for _ in range(3)]
    compacted = copied = 0
    for step in range(24):
        status = ts.new_status(dev())
        prompt = step == 0
        n = 150 if prompt else m
        r = ts.kv_reserve(k, v, table, L, refs, n, freed=freed, out=dict(block_table=table, refs=refs, granted=_i32([0] * len(told))),
                          status=status)
        ts.check_status(status)
        copied += int((r["granted"] > 0).sum())
        tb, ll = table.cpu().numpy(), L.cpu().numpy()
        rc = refs.cpu().numpy()
        np.testing.assert_array_equal(rc, _counts(tb, nb))
        B = len(told)
        # the model writes the K/V of the tokens in flight
        fresh = torch.randn(B, n, 2, Hkv, d, generator=g).to(dtype)
        pos = ll[:, None] + np.arange(n)
        pages = np.take_along_axis(tb, pos // bs, 1)
        assert (pages >= 0).all() and (rc[pages] == 1).all()     # nobody else holds what is written to
        at = torch.from_numpy(pages).to(dev()).long(), torch.from_numpy(pos % bs).to(dev()).long()
        k[at[0], :, at[1]] = fresh[:, :, 0].to(dev())
        v[at[0], :, at[1]] = fresh[:, :, 1].to(dev())
        before = L.clone()
        if prompt:
            L += n
            told = [torch.cat([t, f]) for t, f in zip(told, fresh)]
            freed = None
        else:
            parents, mask, words = _tree(rng, B, m)
            q = torch.randn(B, m, Hq, d, generator=g).to(dtype).to(dev())
            sel = ts.page_select(q, bounds, table, L, 4, block_size=bs, max_prefix=width * bs, first=1, recent=1, status=status)
            out, lse = ts.tree_attention_sparse(q, k, v, table, L, words, sel, status=status)
            ts.check_status(status)
            C = sel["pages"].shape[-1]
            pg, ct, wd, kept = oracle.page_select(q.cpu(), bounds.cpu(), tb, ll, 4, 1, 1, bs, C)
            np.testing.assert_array_equal(sel["pages"].cpu().numpy(), pg)
            np.testing.assert_array_equal(sel["node_mask"].cpu().numpy().view(np.uint64), wd)
            # the reference reads what each sequence has been told, not the pages
            seq = [torch.cat([t, f]) for t, f in zip(told, fresh)]
            longest = max(len(s) for s in seq)
            flat = torch.zeros(B * longest, Hkv, 1, d, 2, dtype=dtype)
            for b, s in enumerate(seq):
                flat[b * longest:b * longest + len(s), :, 0] = s.permute(0, 2, 3, 1)
            kept1 = np.zeros((B, Hkv, m, longest), dtype=bool)   # as pages of one token
            for b in range(B):
                for p in range(ll[b] // bs):
                    kept1[b, :, :, p * bs:(p + 1) * bs] = kept[b, :, :, p:p + 1]
                kept1[b, :, :, ll[b] // bs * bs:ll[b]] = True
            ids = np.arange(B * longest).reshape(B, longest)
            ref, _, spread = oracle.tree_attention_sparse(q.cpu(), flat[..., 0], flat[..., 1], ids, ll, mask, kept1, 1 / math.sqrt(d))
            got = out.double().cpu().numpy()
            # bf16: two roundings of half a step; fp32: some 400 sequential sums and 40 score errors of up to |q||k| / sqrt(d) < 32
            tol = (2.0 ** -8 * (spread + np.abs(ref)) + 2.0 ** -12 * spread if dtype == torch.bfloat16
                   else (2 * 400 + 40 * 32 + 16) * 2.0 ** -24 * spread)
            assert (np.abs(got - ref) <= tol).all()
            # a path is accepted and the rest given back
            path = np.full((B, m), -1)
            alen = np.zeros(B, dtype=np.int64)
            for b in range(B):
                node, up = int(rng.integers(0, m)), []
                while node >= 0:
                    up.append(node)
                    node = int(parents[b, node])
                alen[b] = len(up)
                path[b, :len(up)] = up[::-1]
            c = ts.kv_commit(k, v, table, L, _i32(path), _i32(alen), status=status)
            freed = c["freed_blocks"]
            told = [torch.cat([t, f[path[b, :alen[b]]]]) for b, (t, f) in enumerate(zip(told, fresh))]
        ts.kv_page_bounds(k, table, L, start_len=before, bounds=bounds, status=status)
        ts.check_status(status)
        # the bounds of every complete page of every sequence are right
        tb, ll = table.cpu().numpy(), L.cpu().numpy()
        want = oracle.page_bounds(k.cpu(), tb, ll, [0] * len(told), bounds.cpu())
        np.testing.assert_array_equal(bounds.double().cpu().numpy(), want)
        if step % 4 == 2:   # samples are dropped, doubled and moved; what the commit freed goes back with the next reserve
            B2 = int(rng.integers(2, 6))
            src = rng.integers(0, len(told), size=B2)
            if B2 > 3:
                src[1] = -1
            f = ts.kv_fork(table, L, refs, _i32(src), bs, status=status)
            table, L, refs = f["block_table"], f["prefix_len"], f["refs"]
            told = [told[s] if s >= 0 else told[0][:0] for s in src]
        if step % 5 == 4:
            if freed is not None:   # (first what is still to be let go)
                ids = freed[freed >= 0].long()
                refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
                freed = None
            cc = ts.kv_compact(k, v, table, refs, bounds=bounds, out=dict(block_table=table, refs=refs, remap=_i32([0] * nb), live=_i32([0])),
                               status=status)
            live = int(cc["live"].item())
            assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
            compacted += 1
        ts.check_status(status)
        for b, t in enumerate(told):   # every sequence still reads what it was told
            n_b = int(L[b].item())
            assert n_b == len(t)
            row = table[b].cpu().long()
            p = torch.arange(n_b)
            assert torch.equal(k.cpu()[row[p // bs], :, p % bs], t[:, 0]) and torch.equal(v.cpu()[row[p // bs], :, p % bs], t[:, 1])
    assert compacted == 4 and copied > 10


def _step_state(seed, B=3, m=5, Hq=8, Hkv=2, d=128, bs=16, L=(200, 37, 129)):
    rng = np.random.default_rng(seed)
    nb, width = 80, 20
    g = torch.Generator().manual_seed(seed)
    k, v = [torch.randn(nb, Hkv, bs, d, generator=g).to(torch.bfloat16).to(dev()) for _ in range(2)]
    perm, at, table = rng.permutation(nb), 0, np.full((B, width), -1)
    for b in range(B):
        p = -(-L[b] // bs)
        table[b, :p] = perm[at:at + p]
        at += p
    q = torch.randn(B, m, Hq, d, generator=g).to(torch.bfloat16).to(dev())
    _, _, words = _tree(rng, B, m)
    return dict(k=k, v=v, table=_i32(table), L=_i32(L), refs=_i32(_counts(table, nb)), q=q, words=words, bs=bs, m=m,
                maxp=width * bs, src=_i32(rng.integers(-1, B, size=B)))


def _step(s):
    """One pass through all six calls; inputs are left as they are, but for the caches' free pages."""
    f = ts.kv_fork(s["table"], s["L"], s["refs"], s["src"], s["bs"])
    r = ts.kv_reserve(s["k"], s["v"], f["block_table"], f["prefix_len"], f["refs"], s["m"])
    b = ts.kv_page_bounds(s["k"], r["block_table"], f["prefix_len"])
    sel = ts.page_select(s["q"], b, r["block_table"], f["prefix_len"], 3, block_size=s["bs"], max_prefix=s["maxp"])
    out, lse = ts.tree_attention_sparse(s["q"], s["k"], s["v"], r["block_table"], f["prefix_len"], s["words"], sel)
    k2, v2, b2 = s["k"].clone(), s["v"].clone(), b.clone()
    c = ts.kv_compact(k2, v2, r["block_table"], r["refs"], bounds=b2)
    return [*f.values(), *r.values(), b, *sel.values(), out, lse, *c.values(), k2, v2, b2]


def _same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
               for x, y in zip(a, b))


@pytest.mark.parametrize("m", [5, 1])
def test_captured_and_replayed_with_new_inputs(m):
    """The whole step in a graph: replays on other inputs give what eager calls give on them."""
    lib()
    states = [_step_state(s, m=m) for s in (1, 2, 3)]
    want = [[x.clone() for x in _step(_copy(s))] for s in states]
    held = _copy(states[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(held)
    for i in (1, 2, 0, 1):
        for name, t in states[i].items():
            if torch.is_tensor(t):
                held[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want[i]), i


def _copy(s):
    return {n: t.clone() if torch.is_tensor(t) else t for n, t in s.items()}


@pytest.mark.parametrize("m", [5, 1])
def test_two_graphs_and_two_streams_share_nothing(m):
    lib()
    states = [_step_state(s, m=m, L=L) for s, L in ((4, (200, 37, 129)), (5, (16, 255, 90)))]
    want = [[x.clone() for x in _step(_copy(s))] for s in states]
    torch.cuda.synchronize()
    graphs, got, held = [], [], [_copy(s) for s in states]
    for h in held:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(_step(h))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert _same(got[0], want[0]) and _same(got[1], want[1])
    # eager calls on two streams at once
    again = [None, None]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                again[i] = _step(held[i])
    torch.cuda.synchronize()
    assert _same(again[0], want[0]) and _same(again[1], want[1])


def test_launches_are_counted():
    lib()
    s = _step_state(6)
    _step(_copy(s))
    before = ts.launch_count()
    ts.kv_page_bounds(s["k"], s["table"], s["L"])
    assert ts.launch_count() == before + 1
    ts.kv_fork(s["table"], s["L"], s["refs"], s["src"], 16)
    assert ts.launch_count() == before + 2


def test_tensors_of_another_place_or_layout_are_refused():
    lib()
    s = _step_state(7)
    b = ts.kv_page_bounds(s["k"], s["table"], s["L"])
    calls = [lambda: ts.kv_page_bounds(s["k"], s["table"].cpu(), s["L"]),
             lambda: ts.kv_page_bounds(s["k"], s["table"].t(), s["L"]),
             lambda: ts.kv_page_bounds(s["k"], s["table"], s["L"].long()),
             lambda: ts.kv_page_bounds(s["k"], s["table"], s["L"], status=torch.zeros(1, dtype=torch.int32)),
             lambda: ts.page_select(s["q"], b, s["table"], s["L"][:2], 3, block_size=16, max_prefix=320),
             lambda: ts.kv_reserve(s["k"], s["v"][:, :1], s["table"], s["L"], s["refs"], 4),
             lambda: ts.kv_reserve(s["k"], s["v"], s["table"], s["L"], s["refs"][1:], 4),
             lambda: ts.kv_fork(s["table"], s["L"], s["refs"], s["src"].long(), 16),
             lambda: ts.kv_compact(s["k"], s["v"], s["table"], s["refs"], bounds=b[:-1])]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ts.TreeSpecError):
        ts.kv_reserve(s["k"], s["v"], s["table"], s["L"], s["refs"], 0)


@pytest.mark.parametrize("m", [5, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_caches_whose_offsets_pass_32_bits(dtype, m):
    """A step over the last 80 of 2^19 + 80 pages of 4096 values gives what it gives over 80 pages alone."""
    lib()
    s = _step_state(8, m=m)
    s["k"], s["v"] = s["k"].to(dtype), s["v"].to(dtype)
    s["q"] = s["q"].to(dtype)
    low = 2 ** 19
    far = dict(s)
    for name in ("k", "v"):
        far[name] = torch.empty(low + 80, *s[name].shape[1:], dtype=dtype, device=dev())
        far[name][:low // 2].fill_(float("nan"))   # (the rest of the low half is never touched: whatever is there)
        far[name][low:] = s[name]
    assert far["k"].numel() > 2 ** 31
    far["table"] = torch.where(s["table"] >= 0, s["table"] + low, -1)
    far["refs"] = torch.cat([torch.ones(low, dtype=torch.int32, device=dev()), s["refs"]])   # the low pages are others'

    def step(t):
        f = ts.kv_fork(t["table"], t["L"], t["refs"], t["src"], t["bs"])
        r = ts.kv_reserve(t["k"], t["v"], f["block_table"], f["prefix_len"], f["refs"], t["m"])
        b = ts.kv_page_bounds(t["k"], r["block_table"], f["prefix_len"])
        sel = ts.page_select(t["q"], b, r["block_table"], f["prefix_len"], 3, block_size=t["bs"], max_prefix=t["maxp"])
        out, lse = ts.tree_attention_sparse(t["q"], t["k"], t["v"], r["block_table"], f["prefix_len"], t["words"], sel)
        c = ts.kv_compact(t["k"], t["v"], r["block_table"], r["refs"], bounds=b)
        return ([f["block_table"], r["block_table"], c["block_table"]], [f["refs"], r["refs"], c["refs"], c["remap"], t["k"], t["v"], b],
                [f["prefix_len"], r["granted"], *sel.values(), out, lse], c["live"])

    tables, pages, others, live = step(_copy(s))
    far_tables, far_pages, far_others, far_live = step(far)
    for x, y in zip(tables, far_tables):
        assert torch.equal(torch.where(x >= 0, x + low, -1), y)
    pages[3] = torch.where(pages[3] >= 0, pages[3] + low, -1)
    assert _same(pages, [x[low:] for x in far_pages]) and _same(others, far_others)
    assert int(far_live.item()) == int(live.item()) + low and (pages[3] >= low).any() and (s["refs"] == 0).any()
