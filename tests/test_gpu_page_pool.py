"""GPU kv_reserve, kv_fork and kv_compact vs the oracle: tables, counts and cache bits exactly equal."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu
pool = oracle.page_pool


def _g(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())


def _bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


def _state(rng, B, ways, nb, width, bs, Lmax, pinned=0.05):
    """Rows in groups that share all their pages; some pages held by others too."""
    L = np.repeat(rng.integers(0, Lmax + 1, size=-(-B // ways)), ways)[:B]
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
    refs += rng.random(nb) < pinned
    return table, L, refs


def _caches(rng, nb, H, bs, d, dtype):
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    return [torch.randn(nb, H, bs, d, generator=g).to(dtype) for _ in range(2)]


RESERVE = [dict(B=5, ways=1, nb=200, width=12, bs=16, Lmax=120, n=60, H=2, d=128, dtype=torch.bfloat16),
           dict(B=12, ways=3, nb=300, width=9, bs=16, Lmax=100, n=8, H=2, d=64, dtype=torch.bfloat16),
           dict(B=9, ways=4, nb=40, width=6, bs=8, Lmax=30, n=12, H=1, d=3, dtype=torch.float32),      # runs short
           dict(B=1, ways=1, nb=3, width=1, bs=4, Lmax=3, n=1, H=3, d=2, dtype=torch.bfloat16),
           dict(B=7, ways=7, nb=20000, width=80, bs=1, Lmax=20, n=50, H=1, d=8, dtype=torch.float32),
           dict(B=300, ways=2, nb=9000, width=20, bs=16, Lmax=200, n=33, H=1, d=8, dtype=torch.bfloat16),
           dict(B=1500, ways=5, nb=4000, width=3, bs=64, Lmax=120, n=1, H=1, d=8, dtype=torch.bfloat16),
           dict(B=2, ways=2, nb=3000, width=2100, bs=16, Lmax=5, n=32768, H=1, d=8, dtype=torch.bfloat16)]


@pytest.mark.parametrize("place", ["apart", "in_place"])
@pytest.mark.parametrize("c", RESERVE, ids=lambda c: f"B{c['B']}x{c['ways']}_nb{c['nb']}_bs{c['bs']}_n{c['n']}")
def test_reserve_matches_the_oracle(c, place):
    lib()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        table, L, refs = _state(rng, c["B"], c["ways"], c["nb"], c["width"], c["bs"], c["Lmax"])
        k, v = _caches(rng, c["nb"], c["H"], c["bs"], c["d"], c["dtype"])
        idle = np.nonzero(refs == 0)[0]
        freed = idle[:len(idle) // 3]
        refs[freed] = 2
        freed = np.concatenate([freed, freed[::2], [-1, -1]])  # some listed twice: those come free
        rng.shuffle(freed)
        gk, gv, gt, gr = k.to(dev()), v.to(dev()), _g(table), _g(refs)
        out = dict(block_table=gt, refs=gr, granted=_g(np.zeros(c["B"]))) if place == "in_place" else None
        status = ts.new_status(dev())
        got = ts.kv_reserve(gk, gv, gt, _g(L), gr, c["n"], freed=_g(freed), out=out, status=status)
        torch.cuda.synchronize()
        rk, rv, rt, rr, rg, errors = pool.reserve(_bits(k), _bits(v), table, L, refs, c["n"], freed)
        assert int(status.item()) == (0 if not errors else -7 if errors == {"short"} else -6)
        np.testing.assert_array_equal(got["granted"].cpu().numpy(), rg)
        np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
        np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)
        np.testing.assert_array_equal(_bits(gk), rk)
        np.testing.assert_array_equal(_bits(gv), rv)
        if place == "apart":
            np.testing.assert_array_equal(gt.cpu().numpy(), table)
            np.testing.assert_array_equal(gr.cpu().numpy(), refs)


def test_a_short_pool_with_shared_pages():
    """The sequence that was to keep a shared page, because those before it would have left it, is refused too."""
    lib()
    k = torch.randn(6, 1, 4, 4)
    for free in range(4):
        refs = np.array([3, 2, 9, 9, 9, 9])
        refs[2:2 + free] = 0
        table, L = np.array([[0, -1], [0, -1], [1, -1], [1, -1], [0, -1]]), [2, 2, 1, 1, 2]
        gk, gv = k.to(dev()), (-k).to(dev())
        status = ts.new_status(dev())
        got = ts.kv_reserve(gk, gv, _g(table), _g(L), _g(refs), 2, status=status)
        rk, rv, rt, rr, rg, errors = pool.reserve(_bits(k), _bits(-k), table, L, refs, 2)
        assert int(status.item()) == (-7 if errors else 0)
        np.testing.assert_array_equal(got["granted"].cpu().numpy(), rg)
        np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
        np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)
        np.testing.assert_array_equal(_bits(gk), rk)


@pytest.mark.parametrize("case", ["negative", "too_long", "entry", "below", "freed_id", "freed_free"])
def test_reserve_reports_bad_state(case):
    lib()
    rng = np.random.default_rng(5)
    table, L, refs = _state(rng, 4, 1, 60, 6, 8, 30, pinned=0)
    L[1], table[1, :2] = 9, np.nonzero(refs == 0)[0][:2]
    refs[table[1, :2]] = 1
    freed = []
    if case == "negative":
        L[1] = -3
    elif case == "too_long":
        L[1] = 45
    elif case == "entry":
        table[1, 1] = 60
    elif case == "below":
        table[1, 1] = -2
    elif case == "freed_id":
        freed = [60]
    else:
        freed = [int(np.nonzero(refs == 0)[0][0])]
    k, v = _caches(rng, 60, 1, 8, 4, torch.float32)
    gk, gv = k.to(dev()), v.to(dev())
    status = ts.new_status(dev())
    got = ts.kv_reserve(gk, gv, _g(table), _g(L), _g(refs), 4, freed=_g(freed), status=status)
    rk, rv, rt, rr, rg, errors = pool.reserve(_bits(k), _bits(v), table, L, refs, 4, freed)
    assert errors == {"bad"} and int(status.item()) == -6
    np.testing.assert_array_equal(got["granted"].cpu().numpy(), rg)
    np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
    np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)
    np.testing.assert_array_equal(_bits(gk), rk)


FORK = [dict(B=1, R=8, nb=40, width=8, bs=16, Lmax=100), dict(B=6, R=6, nb=100, width=9, bs=4, Lmax=30),
        dict(B=500, R=700, nb=30000, width=70, bs=16, Lmax=900), dict(B=3, R=1, nb=5000, width=2000, bs=1, Lmax=1500)]


@pytest.mark.parametrize("place", ["apart", "in_place"])
@pytest.mark.parametrize("c", FORK, ids=lambda c: f"B{c['B']}_R{c['R']}_nb{c['nb']}")
def test_fork_matches_the_oracle(c, place):
    lib()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        table, L, refs = _state(rng, c["B"], 1 + seed, c["nb"], c["width"], c["bs"], c["Lmax"])
        idle = np.nonzero(refs == 0)[0]
        for b in range(min(c["B"], len(idle) // 2)):  # pages reserved beyond the length
            p = -(-int(L[b]) // c["bs"])
            if p < c["width"]:
                table[b, p] = idle[b]
                refs[idle[b]] += 1
        src = rng.integers(-1, c["B"], size=c["R"])
        status = ts.new_status(dev())
        gt, gl, gr = _g(table), _g(L), _g(refs)
        out = None
        if place == "in_place":
            out = dict(block_table=torch.empty(c["R"], c["width"], dtype=torch.int32, device=dev()),
                       prefix_len=torch.empty(c["R"], dtype=torch.int32, device=dev()), refs=gr)
        got = ts.kv_fork(gt, gl, gr, _g(src), c["bs"], out=out, status=status)
        ts.check_status(status)
        rt, rl, rr, bad = pool.fork(table, L, refs, src, c["bs"])
        assert not bad
        np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
        np.testing.assert_array_equal(got["prefix_len"].cpu().numpy(), rl)
        np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)


@pytest.mark.parametrize("case", ["src", "src_low", "length", "entry", "missing", "count"])
def test_fork_reports_bad_state(case):
    lib()
    table, L, refs, src = np.array([[0, 1], [2, -1]]), [4, 2], np.array([1, 1, 1, 0]), [0, 1]
    if case == "src":
        src = [0, 2]
    elif case == "src_low":
        src = [-2, 1]
    elif case == "length":
        L = [5, 2]
    elif case == "entry":
        table[0, 1] = 4
    elif case == "missing":
        L = [4, 3]
    else:
        refs[0], src = 0, [1, 1]
    status = ts.new_status(dev())
    got = ts.kv_fork(_g(table), _g(L), _g(refs), _g(src), 2, status=status)
    rt, rl, rr, bad = pool.fork(table, L, refs, src, 2)
    assert bad and int(status.item()) == -6
    np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
    np.testing.assert_array_equal(got["prefix_len"].cpu().numpy(), rl)
    np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)


COMPACT = [dict(B=4, nb=100, width=9, bs=16, Lmax=100, H=2, d=128, dtype=torch.bfloat16, bounds=True),
           dict(B=3, nb=7, width=2, bs=4, Lmax=8, H=1, d=3, dtype=torch.float32, bounds=True),
           dict(B=40, nb=20001, width=30, bs=1, Lmax=20, H=1, d=8, dtype=torch.bfloat16, bounds=False),
           dict(B=2, nb=1, width=1, bs=4, Lmax=0, H=1, d=2, dtype=torch.bfloat16, bounds=False),
           dict(B=64, nb=900, width=12, bs=32, Lmax=350, H=2, d=64, dtype=torch.float32, bounds=True)]


@pytest.mark.parametrize("place", ["apart", "in_place"])
@pytest.mark.parametrize("c", COMPACT, ids=lambda c: f"B{c['B']}_nb{c['nb']}_d{c['d']}")
def test_compact_matches_the_oracle(c, place):
    lib()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        table, L, refs = _state(rng, c["B"], 1 + seed, c["nb"], c["width"], c["bs"], c["Lmax"], pinned=0.1 * seed)
        bufs = _caches(rng, c["nb"], c["H"], c["bs"], c["d"], c["dtype"])
        if c["bounds"]:
            bufs.append(torch.randn(c["nb"], c["H"], 2, c["d"]).to(torch.bfloat16))
        g = [x.to(dev()) for x in bufs]
        gt, gr = _g(table), _g(refs)
        out = None
        if place == "in_place":
            out = dict(block_table=gt, refs=gr, remap=_g(np.zeros(c["nb"])), live=_g([0]))
        status = ts.new_status(dev())
        got = ts.kv_compact(g[0], g[1], gt, gr, bounds=g[2] if c["bounds"] else None, out=out, status=status)
        ts.check_status(status)
        rt, rr, remap, live, bad, moved = pool.compact(table, refs, *[_bits(x) for x in bufs])
        assert not bad and int(got["live"].item()) == live
        np.testing.assert_array_equal(got["block_table"].cpu().numpy(), rt)
        np.testing.assert_array_equal(got["refs"].cpu().numpy(), rr)
        np.testing.assert_array_equal(got["remap"].cpu().numpy(), remap)
        for x, y in zip(g, moved):
            np.testing.assert_array_equal(_bits(x), y)


def test_compact_reports_entries_without_a_page():
    lib()
    k = torch.randn(4, 1, 2, 2, device=dev())
    for table in ([[0, 3]], [[0, 4]], [[0, -2]]):
        status = ts.new_status(dev())
        got = ts.kv_compact(k.clone(), k.clone(), _g(table), _g([0, 1, 1, 0]), status=status)
        assert int(status.item()) == -6
        assert got["block_table"].cpu().tolist() == [[-1, -1]]
        assert got["remap"].cpu().tolist() == [-1, 1, 0, -1]


def test_overlapping_outputs_are_refused():
    lib()
    k = torch.zeros(4, 1, 2, 2, device=dev())
    both = torch.zeros(3, 2, dtype=torch.int32, device=dev())
    L, refs = _g([0, 0]), _g([0, 0, 0, 0])
    out = dict(block_table=both[1:], refs=_g([0] * 4), granted=_g([0, 0]))
    with pytest.raises(ValueError):
        ts.kv_reserve(k, k.clone(), both[:2], L, refs, 1, out=out)
    with pytest.raises(ValueError):
        ts.kv_compact(k, k.clone(), both[:2], refs, out=dict(out, remap=_g([0] * 4), live=_g([0])))
    with pytest.raises(ValueError):
        ts.kv_fork(both[:2], L, refs, _g([0, 1]), 2, out=dict(block_table=both[:2], prefix_len=_g([0, 0]), refs=_g([0] * 4)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_caches_off_the_allocations_alignment(dtype):
    """fp32 caches at any element move in 4-byte pieces; bf16 ones two bytes off are refused."""
    lib()
    rng = np.random.default_rng(4)
    table, L, refs = _state(rng, 6, 2, 60, 6, 8, 30, pinned=0.1)
    k, v = _caches(rng, 60, 2, 8, 4, dtype)

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
        flat[1:].copy_(t.reshape(-1).to(dev()))
        return flat[1:].view(t.shape)

    gk, gv = off(k), off(v)
    if dtype == torch.bfloat16:
        with pytest.raises(ts.TreeSpecError):
            ts.kv_reserve(gk, gv, _g(table), _g(L), _g(refs), 4)
        with pytest.raises(ts.TreeSpecError):
            ts.kv_compact(gk, gv, _g(table), _g(refs))
        return
    got = ts.kv_reserve(gk, gv, _g(table), _g(L), _g(refs), 4)
    rk, rv, rt, rr, rg, errors = pool.reserve(_bits(k), _bits(v), table, L, refs, 4)
    assert not errors
    np.testing.assert_array_equal(_bits(gk), rk)
    ts.kv_compact(gk, gv, got["block_table"], got["refs"])
    *_, (rk, rv) = pool.compact(rt, rr, rk, rv)
    np.testing.assert_array_equal(_bits(gk), rk)
    np.testing.assert_array_equal(_bits(gv), rv)


@pytest.mark.parametrize("op,name,other", [
    ("reserve", "granted", "L"), ("reserve", "granted", "freed"), ("reserve", "granted", "refs"), ("reserve", "refs", "refs_out"),
    ("fork", "refs", "src"), ("fork", "prefix_len", "L"), ("fork", "prefix_len", "refs"), ("compact", "remap", "refs"),
    ("compact", "live", "table"), ("compact", "live", "remap")])
def test_outputs_that_are_other_inputs_or_outputs_are_refused(op, name, other):
    lib()
    k = torch.zeros(4, 1, 2, 2, device=dev())
    t = dict(table=_g(np.full((4, 2), -1)), L=_g([0] * 4), refs=_g([0] * 4), freed=_g([-1] * 4), src=_g([0] * 4))
    outs = dict(reserve=dict(block_table=_g(np.zeros((4, 2))), refs=_g([0] * 4), granted=_g([0] * 4)),
                fork=dict(block_table=_g(np.zeros((4, 2))), refs=_g([0] * 4), prefix_len=_g([0] * 4)),
                compact=dict(block_table=_g(np.zeros((4, 2))), refs=_g([0] * 4), remap=_g([0] * 4), live=_g([0])))
    call = dict(reserve=lambda out: ts.kv_reserve(k, k.clone(), t["table"], t["L"], t["refs"], 1, freed=t["freed"], out=out),
                fork=lambda out: ts.kv_fork(t["table"], t["L"], t["refs"], t["src"], 2, out=out),
                compact=lambda out: ts.kv_compact(k, k.clone(), t["table"], t["refs"], out=out))[op]
    call(outs[op])
    out = dict(outs[op])
    out[name] = (out["granted"] if other == "refs_out" else t.get(other, out.get(other))).view(-1)[:out[name].numel()].view(out[name].shape)
    with pytest.raises(ValueError):
        call(out)
