"""The 8-bit cache's calls together, as a serving loop uses them: room is reserved, rows are quantised, attention computed, a
path committed, sequences forked and the pool compacted, for many steps, against the oracle's state; captured into
graphs and replayed, two graphs and two streams at once."""
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import F8, assert_within, attention_bounds, ints, tree_mask, words
from gpu_helpers import lib
from oracle import kv_fp8 as o8

pytestmark = pytest.mark.gpu
pool = oracle.page_pool


@pytest.fixture(autouse=True)
def _built():
    lib()


def _rows(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape) * np.exp2(rng.integers(-3, 3, shape[:-1] + (1,)))).to(dtype)


def _trees(rng, B, m):
    parents = np.full((B, m), -1)
    for b in range(B):
        for i in range(1, m):
            parents[b, i] = rng.integers(max(0, i - 5), i)
    return parents, np.stack([oracle.ancestor_mask(p.tolist()) for p in parents])


def _live(codes, scales, table, lens, sb):
    """The bytes and scales of everything that a sequence holds."""
    bs, out = codes[0].shape[2], []
    for b, n in enumerate(lens):
        pos = np.arange(int(n))
        out += [x[table[b][pos // bs], :, pos % bs] for x in codes]
        out += [x[table[b][pos // bs], :, pos % bs // sb] for x in scales]
    return out


@pytest.mark.parametrize("dtype,Hq,Hkv,d,bs,sb,m", [(torch.bfloat16, 4, 2, 128, 16, 16, 9), (torch.bfloat16, 8, 1, 128, 32, 8, 12),
                                                   (torch.float32, 4, 2, 64, 16, 4, 6)])
def test_a_serving_loop(dtype, Hq, Hkv, d, bs, sb, m):
    rng = np.random.default_rng(m)
    nb, width = 100, 20
    dev = ([torch.zeros(nb, Hkv, bs, d, dtype=torch.uint8, device="cuda").view(F8) for _ in "kv"]
           + [torch.zeros(nb, Hkv, bs // sb, device="cuda") for _ in "kv"])
    scales_of = dict(k_scale=dev[2], v_scale=dev[3])
    codes = [np.zeros((nb, Hkv, bs, d), dtype=np.uint8) for _ in "kv"]
    scales = [np.zeros((nb, Hkv, bs // sb)) for _ in "kv"]
    table, L, refs, freed = ints(np.full((3, width), -1)), ints([0, 0, 0]), ints([0] * nb), None
    ht, hl, hr, hf = np.full((3, width), -1), np.zeros(3, dtype=np.int64), np.zeros(nb, dtype=np.int64), []
    copied = compacted = 0
    for step in range(14):
        status = ts.new_status()
        n = 2 * bs + 5 if step == 0 else m
        B = len(hl)
        r = ts.kv_reserve(*dev[:2], table, L, refs, n, freed=freed, **scales_of, status=status)
        table, refs = r["block_table"], r["refs"]
        rows = [np.repeat(s, sb, axis=2)[..., None] for s in scales]
        old = ht
        ck, cv, ht, rr, _, errors = pool.reserve(*codes, ht, hl, hr, n, hf)
        assert not errors
        scales = [x[:, :, ::sb, 0].copy() for x in pool.reserve(*rows, old, hl, hr, n, hf)[:2]]
        codes, hr = [ck, cv], rr
        copied += int(((old >= 0) & (ht != old)).sum())
        assert np.array_equal(table.cpu().numpy(), ht) and np.array_equal(refs.cpu().numpy(), hr)
        x = [_rows(rng, (B, n, Hkv, d), dtype) for _ in "kv"]
        ts.kv_write_fp8(*[t.cuda() for t in x], *dev, table, L, status=status)
        for i in (0, 1):
            o8.write(codes[i], scales[i], x[i].double().numpy(), ht, hl, [n] * B)
        if step == 0:
            L, hl, freed, hf = L + n, hl + n, None, []
        else:
            parents, mask = _trees(rng, B, m)
            q = _rows(rng, (B, m, Hq, d), dtype)
            out, lse = ts.tree_attention_fp8(q.cuda(), *dev, table, L, words(mask), max_prefix=width * bs - m, status=status)
            ts.check_status(status)
            values = [o8.values(c, s) for c, s in zip(codes, scales)]
            ref, ref_lse, bo, bl = attention_bounds(q.double().numpy(), *values, ht, hl, mask, 1 / math.sqrt(d), dtype == torch.bfloat16)
            assert_within(lse, ref_lse, bl, "lse")
            assert_within(out, ref, bo, "out")
            path, alen = np.full((B, m), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
            for b in range(B):
                node, up = int(rng.integers(0, m)), []
                while node >= 0:
                    up.append(node)
                    node = int(parents[b, node])
                alen[b] = len(up)
                path[b, :len(up)] = up[::-1]
            r = ts.kv_commit_fp8(*dev, table, L, ints(path), ints(alen), status=status)
            table, L, freed = r["block_table"], r["prefix_len"], r["freed_blocks"]
            ht, hl, hf, _ = o8.commit(codes, scales, ht, hl, path, alen, m)
            hl = np.asarray(hl, dtype=np.int64)
        if step % 4 == 2:
            B2 = int(rng.integers(2, 5))
            src = rng.integers(0, B, size=B2)
            f = ts.kv_fork(table, L, refs, ints(src), bs, status=status)
            table, L, refs = f["block_table"], f["prefix_len"], f["refs"]
            ht, hl, hr, bad = pool.fork(ht, hl, hr, src, bs)
            assert not bad
        if step % 5 == 4:
            let_go = np.asarray(hf).reshape(-1)                # first what is still to be given back
            for p in let_go[let_go >= 0]:
                hr[p] -= 1
            refs, freed, hf = ints(hr), None, []
            cc = ts.kv_compact(*dev[:2], table, refs, **scales_of, status=status)
            table, refs = cc["block_table"], cc["refs"]
            ht, hr, _, _, bad, moved = pool.compact(ht, hr, *codes, *scales)
            assert not bad
            codes, scales = [x.copy() for x in moved[:2]], [x.copy() for x in moved[2:]]
            compacted += 1
        ts.check_status(status)
        assert np.array_equal(table.cpu().numpy(), ht) and np.array_equal(L.cpu().numpy(), hl)
        got = _live([t.view(torch.uint8).cpu().numpy() for t in dev[:2]], [t.cpu().numpy().astype(np.float64) for t in dev[2:]], ht, hl, sb)
        for a, b in zip(got, _live(codes, scales, ht, hl, sb)):
            assert np.array_equal(a, b), step
    assert copied >= 1 and compacted == 2


def _state(seed, dtype, m, lens=(200, 37, 129), Hq=8, Hkv=2, bs=16, sb=8):
    rng = np.random.default_rng(seed)
    d = 128 if dtype == torch.bfloat16 else 64
    nb, width, B = 80, 24, len(lens)
    perm, at, table = rng.permutation(nb), 0, np.full((B, width), -1)
    for b in range(B):
        p = -(-lens[b] // bs)
        table[b, :p] = perm[at:at + p]
        at += p
    s = dict(k=torch.from_numpy(o8.encode(rng.standard_normal((nb, Hkv, bs, d)) * 100)).cuda().view(F8),
             v=torch.from_numpy(o8.encode(rng.standard_normal((nb, Hkv, bs, d)) * 100)).cuda().view(F8),
             ks=torch.from_numpy(np.exp2(rng.integers(-9, -5, (nb, Hkv, bs // sb)))).float().cuda(),
             vs=torch.from_numpy(np.exp2(rng.integers(-9, -5, (nb, Hkv, bs // sb)))).float().cuda(),
             table=ints(table), L=ints(lens), refs=ints(np.bincount(table[table >= 0], minlength=nb)),
             src=ints(rng.integers(0, B, size=B)), q=_rows(rng, (B, m, Hq, d), dtype).cuda(), words=words(tree_mask(rng, B, m)))
    s["nk"], s["nv"] = [_rows(rng, (B, m, Hkv, d), dtype).cuda() for _ in "kv"]
    path = np.full((B, m), -1)
    path[:, 0] = 0
    path[0, 1:2] = m - 1
    s["path"], s["alen"] = ints(path), ints([min(m, 2)] + [1] * (B - 1))
    return s


def _step(s):
    """One pass through every call; the state that it starts from is left as it is."""
    dev = [s[n].view(torch.uint8).clone().view(F8) for n in ("k", "v")] + [s[n].clone() for n in ("ks", "vs")]
    scales = dict(k_scale=dev[2], v_scale=dev[3])
    m, maxp = s["q"].shape[1], 24 * 16 - s["q"].shape[1]
    f = ts.kv_fork(s["table"], s["L"], s["refs"], s["src"], 16)
    r = ts.kv_reserve(*dev[:2], f["block_table"], f["prefix_len"], f["refs"], m, **scales)
    ts.kv_write_fp8(s["nk"], s["nv"], *dev, r["block_table"], f["prefix_len"])
    out, lse = ts.tree_attention_fp8(s["q"], *dev, r["block_table"], f["prefix_len"], s["words"], max_prefix=maxp)
    c = ts.kv_commit_fp8(*dev, r["block_table"], f["prefix_len"], s["path"], s["alen"])
    k, v = ts.kv_read_fp8(*dev, c["block_table"], c["prefix_len"], 64)
    cc = ts.kv_compact(*dev[:2], c["block_table"], r["refs"], **scales)
    return [out, lse, k, v, *f.values(), *r.values(), *c.values(), *cc.values(), *dev]


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _same(a, b):
    return all(torch.equal(_bytes(x), _bytes(y)) for x, y in zip(a, b))


CASES = [(torch.bfloat16, 1), (torch.bfloat16, 8), (torch.bfloat16, 40), (torch.float32, 3)]


@pytest.mark.parametrize("dtype,m", CASES)
def test_captured_and_replayed_with_new_inputs(dtype, m):
    states = [_state(i, dtype, m) for i in (1, 2, 3)]
    want = [[x.clone() for x in _step(s)] for s in states]
    held = {n: t.clone() for n, t in states[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(held)
    for i in (1, 2, 0, 1):
        for n, t in states[i].items():
            _bytes(held[n]).copy_(_bytes(t))
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want[i]), i


@pytest.mark.parametrize("dtype,m", CASES)
def test_two_graphs_and_two_streams_share_nothing(dtype, m):
    states = [_state(i, dtype, m, lens) for i, lens in ((4, (200, 37, 129)), (5, (16, 255, 90)))]
    want = [[x.clone() for x in _step(s)] for s in states]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(_step(s))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert _same(got[0], want[0]) and _same(got[1], want[1])
    again = [None, None]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                again[i] = _step(states[i])
    torch.cuda.synchronize()
    assert _same(again[0], want[0]) and _same(again[1], want[1])


def test_launches_are_counted():
    s = _state(6, torch.bfloat16, 4)
    dev = [s[n] for n in ("k", "v", "ks", "vs")]
    before = ts.launch_count()
    ts.kv_read_fp8(*dev, s["table"], s["L"], 8)
    assert ts.launch_count() == before + 1
    ts.kv_reserve(*dev[:2], s["table"], s["L"], s["refs"], 4, k_scale=dev[2], v_scale=dev[3])
    assert ts.launch_count() == before + 3
