"""GPU kv_page_bounds and page_select vs the oracle: every value and every chosen page exactly equal
(both are exact by construction: eight-bit whole numbers on power-of-two grids)."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_eagle_gb300 as ts
from gpu_helpers import dev, lib

pytestmark = pytest.mark.gpu


def _table(rng, need, spare=2):
    """Shuffled block tables whose row b holds need[b] pages."""
    nb = sum(need) + spare
    perm, table, at = rng.permutation(nb), np.full((len(need), max(max(need), 1)), -1, dtype=np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, nb


def _keys(rng, nb, Hkv, bs, d, dtype):
    k = torch.from_numpy(rng.standard_normal((nb, Hkv, bs, d)) * np.exp(rng.standard_normal((nb, Hkv, 1, 1)) * 3)).to(dtype)
    return k


BOUNDS = [dict(L=[64, 17, 0], start=None, Hkv=2, bs=16, d=128, dtype=torch.bfloat16),
          dict(L=[150, 31, 128], start=[100, 31, 0], Hkv=3, bs=32, d=64, dtype=torch.bfloat16),
          dict(L=[7, 1], start=None, Hkv=1, bs=1, d=256, dtype=torch.bfloat16),
          dict(L=[60, 9], start=[3, 8], Hkv=2, bs=3, d=80, dtype=torch.bfloat16),
          dict(L=[40], start=None, Hkv=2, bs=8, d=37, dtype=torch.bfloat16),
          dict(L=[33, 50], start=None, Hkv=2, bs=16, d=128, dtype=torch.float32),
          dict(L=[33], start=[16], Hkv=1, bs=16, d=200, dtype=torch.float32),
          dict(L=[256], start=None, Hkv=2, bs=128, d=6, dtype=torch.float32)]


@pytest.mark.parametrize("c", BOUNDS, ids=lambda c: f"bs{c['bs']}_d{c['d']}_{str(c['dtype'])[6:]}")
def test_bounds_match_the_oracle(c):
    lib()
    rng = np.random.default_rng(c["d"])
    table, nb = _table(rng, [-(-n // c["bs"]) for n in c["L"]])
    k = _keys(rng, nb, c["Hkv"], c["bs"], c["d"], c["dtype"])
    before = torch.from_numpy(rng.standard_normal((nb, c["Hkv"], 2, c["d"]))).to(torch.bfloat16)
    start = c["start"] or [0] * len(c["L"])
    status = ts.new_status(dev())
    got = ts.kv_page_bounds(k.to(dev()), torch.from_numpy(table).to(dev()), torch.tensor(c["L"], dtype=torch.int32, device=dev()),
                            start_len=None if c["start"] is None else torch.tensor(start, dtype=torch.int32, device=dev()),
                            bounds=before.to(dev()), status=status)
    ts.check_status(status)
    np.testing.assert_array_equal(got.double().cpu().numpy(), oracle.page_bounds(k, table, c["L"], start, before))


def test_bounds_of_odd_values():
    """NaN, infinities, zeros, subnormals and the largest values of the type."""
    lib()
    inf, nan, big = float("inf"), float("nan"), 3.38e38
    for dtype in (torch.bfloat16, torch.float32):
        k = torch.zeros(2, 2, 16, 128, dtype=torch.float32)
        k[0, 0, :, 0] = nan
        k[0, 0, 3, 1:6] = torch.tensor([nan, inf, -inf, big, -big])
        k[0, 1] = 1e-39
        k[1, 0, 5] = -1e-20
        k[1, 1, :, :] = 255.0
        k[1, 1, 0, 7] = -256.0
        k = k.to(dtype)
        table = np.array([[1, 0]], dtype=np.int32)
        status = ts.new_status(dev())
        got = ts.kv_page_bounds(k.to(dev()), torch.from_numpy(table).to(dev()), torch.tensor([32], dtype=torch.int32, device=dev()),
                                status=status)
        ts.check_status(status)
        np.testing.assert_array_equal(got.double().cpu().numpy(),
                                      oracle.page_bounds(k, table, [32], [0], np.zeros((2, 2, 2, 128))))


def test_bounds_report_bad_state_and_skip_it():
    lib()
    k = torch.ones(3, 1, 4, 8, device=dev())
    before = torch.full((3, 1, 2, 8), 5.0, dtype=torch.bfloat16, device=dev())
    for table, L in (([[0, 3], [1, 2]], [8, 8]), ([[0, -1], [1, 2]], [8, 8]), ([[0, 0], [1, 2]], [-1, 8]),
                     ([[0, 0], [1, 2]], [9, 8])):
        status = ts.new_status(dev())
        got = ts.kv_page_bounds(k, torch.tensor(table, dtype=torch.int32, device=dev()),
                                torch.tensor(L, dtype=torch.int32, device=dev()), bounds=before.clone(), status=status)
        assert int(status.item()) == -6
        assert (got[1:] == 1).all()                               # the sound sequence is done
        assert (got[0] == (1 if L[0] == 8 else 5)).all()


SELECT = [dict(L=[300, 16, 7], m=5, Hq=8, Hkv=2, d=128, bs=16, n=4, first=1, recent=2, dtype=torch.bfloat16),
          dict(L=[2100], m=1, Hq=8, Hkv=8, d=128, bs=16, n=9, first=0, recent=0, dtype=torch.bfloat16),
          dict(L=[2300, 640], m=70, Hq=6, Hkv=2, d=64, bs=16, n=5, first=1, recent=1, dtype=torch.bfloat16),
          dict(L=[700, 0, 1000], m=3, Hq=14, Hkv=2, d=128, bs=16, n=20, first=2, recent=3, dtype=torch.float32),
          dict(L=[90], m=256, Hq=2, Hkv=1, d=256, bs=2, n=7, first=0, recent=1, dtype=torch.bfloat16),
          dict(L=[1000], m=2, Hq=5, Hkv=1, d=200, bs=8, n=3, first=1, recent=0, dtype=torch.float32),
          dict(L=[500], m=4, Hq=4, Hkv=4, d=37, bs=5, n=11, first=1, recent=1, dtype=torch.bfloat16),
          dict(L=[160], m=2, Hq=256, Hkv=2, d=16, bs=4, n=1, first=0, recent=1, dtype=torch.bfloat16),
          dict(L=[2600], m=2, Hq=2, Hkv=1, d=16, bs=1, n=300, first=5, recent=5, dtype=torch.bfloat16),
          dict(L=[9000], m=1, Hq=2, Hkv=1, d=8, bs=1, n=1000, first=5, recent=5, dtype=torch.bfloat16)]


# one node per sequence: head groups of 1 to 9 (8 is the last that a cluster takes), head dims of 8 to 256 and one not a
# multiple of 8, rows of up to 8192 pages and one more, empty and short sequences, all pages wanted, 16
# clusters and 25
ONE = [dict(L=[2100, 0, 5], m=1, Hq=4, Hkv=4, d=128, bs=1, n=40, first=1, recent=1, dtype=torch.bfloat16),
       dict(L=[8192, 8191], m=1, Hq=4, Hkv=2, d=8, bs=1, n=1000, first=5, recent=5, dtype=torch.bfloat16),
       dict(L=[8193], m=1, Hq=4, Hkv=2, d=8, bs=1, n=1000, first=5, recent=5, dtype=torch.bfloat16),
       dict(L=[513, 1024, 1], m=1, Hq=6, Hkv=2, d=64, bs=1, n=100, first=0, recent=0, dtype=torch.bfloat16),
       dict(L=[700, 300], m=1, Hq=8, Hkv=2, d=72, bs=2, n=1, first=0, recent=0, dtype=torch.float32),
       dict(L=[900], m=1, Hq=5, Hkv=1, d=256, bs=3, n=299, first=1, recent=1, dtype=torch.bfloat16),
       dict(L=[900], m=1, Hq=16, Hkv=2, d=200, bs=3, n=300, first=1, recent=1, dtype=torch.float32),
       dict(L=[640, 77], m=1, Hq=14, Hkv=2, d=128, bs=16, n=30, first=2, recent=3, dtype=torch.bfloat16),
       dict(L=[640], m=1, Hq=9, Hkv=1, d=128, bs=16, n=12, first=2, recent=3, dtype=torch.bfloat16),
       dict(L=[640], m=1, Hq=4, Hkv=2, d=36, bs=4, n=12, first=12, recent=0, dtype=torch.float32),
       dict(L=[40, 33, 16, 15] * 4, m=1, Hq=2, Hkv=1, d=16, bs=4, n=4, first=0, recent=4, dtype=torch.bfloat16),
       dict(L=[40, 33, 16, 15, 3] * 5, m=1, Hq=8, Hkv=1, d=16, bs=4, n=4, first=2, recent=1, dtype=torch.bfloat16)]


def _select_case(c, seed=0, ties=False):
    rng = np.random.default_rng(seed + c["d"])
    B = len(c["L"])
    table, nb = _table(rng, [-(-n // c["bs"]) for n in c["L"]])
    Hkv, d = c["Hkv"], c["d"]
    if ties:
        rows = rng.integers(-2, 3, size=(nb, Hkv, 2, d)) * (rng.random((nb, Hkv, 2, d)) < 0.05)
    else:
        rows = rng.integers(-255, 256, size=(nb, Hkv, 2, d)) * 2.0 ** rng.integers(-9, -7, size=(nb, Hkv, 1, 1))
    bounds = torch.from_numpy(np.sort(rows, axis=2)[:, :, ::-1].copy().astype(np.float64)).to(torch.bfloat16)
    q = torch.from_numpy(rng.standard_normal((B, c["m"], c["Hq"], d)) * np.exp(rng.standard_normal((B, c["m"], c["Hq"], 1)))).to(
        c["dtype"])
    return table, bounds, q


def _run_select(c, table, bounds, q, status=None, max_prefix=None, **kw):
    return ts.page_select(q.to(dev()), bounds.to(dev()), torch.from_numpy(table).to(dev()),
                          torch.tensor(c["L"], dtype=torch.int32, device=dev()), c["n"], block_size=c["bs"],
                          max_prefix=max(c["L"]) if max_prefix is None else max_prefix, first=c["first"], recent=c["recent"],
                          status=status, **kw)


def _check_select(c, table, bounds, q, got):
    C = got["pages"].shape[-1]
    pages, count, words, _ = oracle.page_select(q, bounds, table, c["L"], c["n"], c["first"], c["recent"], c["bs"], C)
    np.testing.assert_array_equal(got["count"].cpu().numpy(), count)
    np.testing.assert_array_equal(got["pages"].cpu().numpy(), pages)
    np.testing.assert_array_equal(got["node_mask"].cpu().numpy().view(np.uint64), words)


@pytest.mark.parametrize("ties", [False, True], ids=["spread", "ties"])
@pytest.mark.parametrize("c", SELECT, ids=lambda c: f"L{c['L'][0]}_m{c['m']}_{c['Hq']}x{c['Hkv']}_d{c['d']}_{str(c['dtype'])[6:]}")
def test_choice_matches_the_oracle(c, ties):
    lib()
    table, bounds, q = _select_case(c, ties=ties)
    status = ts.new_status(dev())
    got = _run_select(c, table, bounds, q, status)
    ts.check_status(status)
    _check_select(c, table, bounds, q, got)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("c", ONE, ids=lambda c: f"L{c['L'][0]}_{c['Hq']}x{c['Hkv']}_d{c['d']}_{str(c['dtype'])[6:]}")
def test_choice_of_one_node_matches_the_oracle(c, ties):
    lib()
    table, bounds, q = _select_case(c, ties=ties)
    status = ts.new_status(dev())
    got = _run_select(c, table, bounds, q, status)
    ts.check_status(status)
    _check_select(c, table, bounds, q, got)
    _check_select(c, table, bounds, q, _run_select(c, table, bounds, _offset(q), status))  # queries off 16 bytes


@pytest.mark.parametrize("g", [4, 8])
@pytest.mark.parametrize("d", [128, 256])
def test_scores_of_one_node_are_exact_at_their_largest(d, g):
    """As test_scores_are_exact_at_their_largest, one query per sequence and sign, the group's last head the best."""
    lib()
    c = dict(L=[200, 200], m=1, Hq=g, Hkv=1, d=d, bs=1, n=60, first=0, recent=0)
    rng = np.random.default_rng(4)
    bounds = np.full((200, 1, 2, d), 255.0)
    less = rng.permutation(200)
    for p in range(200):
        np.subtract.at(bounds[p, 0, 0], rng.integers(0, d, size=less[p]), 1.0)
    bounds[:, :, 1] = -255.0
    q = torch.zeros((2, 1, g, d), dtype=torch.bfloat16)
    q[0, 0, g - 1], q[1, 0, g - 1] = 255.0, -255.0
    table = np.stack([np.arange(200), rng.permutation(200)]).astype(np.int32)
    b = torch.from_numpy(bounds).to(torch.bfloat16)
    status = ts.new_status(dev())
    got = _run_select(c, table, b, q, status)
    ts.check_status(status)
    _check_select(c, table, b, q, got)


@pytest.mark.parametrize("L,entry", [(640, 40), (640, -1), (-1, 0), (641, 0)])
def test_bad_state_of_one_node_is_reported(L, entry):
    """A table entry out of range (its page scores 0) or a length that is not in 0 .. max_prefix (no pages)."""
    lib()
    c = dict(L=[L], m=1, Hq=4, Hkv=2, d=64, bs=16, n=5, first=1, recent=1)
    rng = np.random.default_rng(5)
    table = np.arange(40, dtype=np.int32)[None].copy()
    bounds = torch.from_numpy(rng.integers(1, 200, size=(40, 2, 2, 64)).astype(np.float64)).to(torch.bfloat16)
    bounds[:, :, 1] = -bounds[:, :, 0]
    q = torch.from_numpy(rng.standard_normal((1, 1, 4, 64))).to(torch.bfloat16)
    table[0, 7] = entry if entry else table[0, 7]
    status = ts.new_status(dev())
    got = _run_select(c, table, bounds, q, status, max_prefix=640)
    assert int(status.item()) == -6
    if L != 640:
        assert (got["count"] == 0).all() and (got["pages"] == -1).all() and (got["node_mask"] == 0).all()
    else:
        table[0, 7], rest = 0, torch.cat([bounds, torch.zeros_like(bounds[:1])])
        table[0, 7] = 40  # a page of zeros
        _check_select(c, table, rest, q, got)


@pytest.mark.parametrize("d", [128, 256])
def test_scores_are_exact_at_their_largest(d):
    """Pages whose scores differ by one unit in up to 255 * 255 * d: the sums must not round."""
    lib()
    c = dict(L=[200], m=2, Hq=2, Hkv=1, d=d, bs=1, n=60, first=0, recent=0)
    rng = np.random.default_rng(3)
    bounds = np.full((202, 1, 2, d), 255.0)
    less = rng.permutation(200)
    for p in range(200):  # page p's upper bounds sum to less[p] below the most
        at = rng.integers(0, d, size=less[p])
        np.subtract.at(bounds[p, 0, 0], at, 1.0)
    bounds[:, :, 1] = -255.0
    q = torch.full((1, 2, 2, d), 255.0, dtype=torch.bfloat16)
    q[0, 1] *= -1  # every page ties at the lower bounds
    table = rng.permutation(202)[:200].reshape(1, 200).astype(np.int32)
    full = np.empty_like(bounds)
    full[table[0]] = bounds[:200]
    full[np.setdiff1d(np.arange(202), table[0])] = 0
    b = torch.from_numpy(full).to(torch.bfloat16)
    status = ts.new_status(dev())
    got = _run_select(c, table, b, q, status)
    ts.check_status(status)
    _check_select(c, table, b, q, got)


def test_odd_queries():
    """NaN, infinite, zero and tiny queries."""
    lib()
    c = dict(L=[320], m=5, Hq=2, Hkv=1, d=64, bs=16, n=5, first=1, recent=1)
    table, bounds, q = _select_case(dict(c, dtype=torch.float32))
    q[0, 0] = 0
    q[0, 1, 0, 3], q[0, 1, 1, 5] = float("nan"), float("inf")
    q[0, 2] = float("nan")
    q[0, 3] *= 1e-30
    q[0, 4, :, 1] = -3.4e38
    for dtype in (torch.float32, torch.bfloat16):
        qd = q.to(dtype)
        status = ts.new_status(dev())
        got = _run_select(c, table, bounds, qd, status)
        ts.check_status(status)
        _check_select(c, table, bounds, qd, got)


def test_a_larger_host_bound_and_reused_outputs():
    """The outputs' capacity follows max_prefix; what lies behind the last page is written too, and a
    workspace and outputs of the caller's may hold anything."""
    lib()
    c = SELECT[0]
    table, bounds, q = _select_case(c)
    wide = np.full((3, 40), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    out = dict(pages=torch.full((3, 2, 37), 99, dtype=torch.int32, device=dev()),
               count=torch.full((3, 2), 99, dtype=torch.int32, device=dev()),
               node_mask=torch.full((3, 2, 37, 1), 99, dtype=torch.int64, device=dev()))
    ws = torch.full((1 << 18,), 255, dtype=torch.uint8, device=dev())
    got = _run_select(c, wide, bounds, q, max_prefix=600, out=out, workspace=ws)
    _check_select(c, wide, bounds, q, got)


def test_bad_state_is_reported():
    lib()
    c = SELECT[0]
    table, bounds, q = _select_case(c)
    for L in ([301, 16, 7], [-1, 16, 7]):
        status = ts.new_status(dev())
        got = _run_select(dict(c, L=L), table, bounds, q, status, max_prefix=300)
        assert int(status.item()) == -6
        assert (got["count"][0] == 0).all() and (got["pages"][0] == -1).all() and (got["node_mask"][0] == 0).all()
        assert (got["count"][1] > 0).all()
    table[0, 5] = 1000
    status = ts.new_status(dev())
    got = _run_select(c, table, bounds, q, status)
    assert int(status.item()) == -6
    _check_select(c, table, bounds, q, got)  # its score is 0


def test_one_page_and_no_page():
    lib()
    c = dict(L=[15, 16, 0], m=2, Hq=2, Hkv=2, d=128, bs=16, n=3, first=1, recent=1, dtype=torch.bfloat16)
    table, bounds, q = _select_case(c)
    for maxp in (16, 40):
        wide = np.full((3, 3), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        got = _run_select(c, wide, bounds, q, max_prefix=maxp)
        _check_select(c, wide, bounds, q, got)
    c = dict(c, L=[5, 9, 0])
    got = _run_select(c, wide, bounds, q)
    assert (got["count"] == 0).all() and (got["pages"] == -1).all()


def test_refusals():
    lib()
    c = SELECT[0]
    table, bounds, q = _select_case(c)
    with pytest.raises(ts.TreeSpecError):
        _run_select(dict(c, n=2), table, bounds, q)                    # first + recent > n
    with pytest.raises(ts.TreeSpecError):
        _run_select(c, table, bounds, q, max_prefix=4000)              # more than the table holds
    with pytest.raises(ValueError):
        _run_select(c, table, bounds[..., :64].contiguous(), q)
    with pytest.raises(ValueError):
        _run_select(c, table, bounds.float(), q)
    with pytest.raises(ValueError):
        _run_select(c, table, bounds, q, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError):
        _run_select(c, table, bounds, q, out=dict(pages=torch.empty(3, 2, 4, dtype=torch.int32, device=dev())))


def _offset(t):
    """The same contiguous tensor one element off the allocation's alignment."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev())
    flat[1:].copy_(t.reshape(-1).to(dev()))
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_off_the_allocations_alignment(dtype):
    lib()
    rng = np.random.default_rng(9)
    table, nb = _table(rng, [5, 3])
    k = _keys(rng, nb, 2, 16, 128, dtype)
    want = oracle.page_bounds(k, table, [80, 41], [0, 0], np.zeros((nb, 2, 2, 128)))
    L = torch.tensor([80, 41], dtype=torch.int32, device=dev())
    out = _offset(torch.zeros(nb, 2, 2, 128, dtype=torch.bfloat16))
    got = ts.kv_page_bounds(_offset(k), torch.from_numpy(table).to(dev()), L, bounds=out)
    np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    c = dict(SELECT[0], dtype=dtype)
    table, bounds, q = _select_case(c)
    got = ts.page_select(_offset(q), bounds.to(dev()), torch.from_numpy(table).to(dev()),
                         torch.tensor(c["L"], dtype=torch.int32, device=dev()), c["n"], block_size=16, max_prefix=300, first=1,
                         recent=2)
    _check_select(c, table, bounds, q, got)
    with pytest.raises(ts.TreeSpecError):   # bounds are copied 16 bytes at a time
        ts.page_select(q.to(dev()), _offset(bounds), torch.from_numpy(table).to(dev()),
                       torch.tensor(c["L"], dtype=torch.int32, device=dev()), c["n"], block_size=16, max_prefix=300)
