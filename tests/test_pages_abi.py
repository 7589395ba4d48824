"""Host-side validation of the page calls (CPU only: every call here is refused before any launch)."""
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from speculative_decoding_tree_eagle_gb300 import build as tsbuild

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    tsbuild.build()
    return ts.library()


def test_status_string_of_a_short_pool():
    assert ts.status_string(-7).startswith("TS_ERR_NO_PAGES")


def _bounds(lib, dt=1, nb=4, bs=16, hkv=2, d=128, width=4, B=1, ptr=16):
    P = ptr
    return lib.ts_kv_page_bounds(P, dt, nb, bs, hkv, d, P, width, P, None, B, P, None, None)


def test_page_bounds_validation(lib):
    for kw in (dict(dt=2), dict(nb=0), dict(bs=0), dict(hkv=0), dict(d=0), dict(width=0), dict(B=0), dict(ptr=None)):
        assert _bounds(lib, **kw) == INVALID, kw
    for kw in (dict(d=257), dict(B=65536)):
        assert _bounds(lib, **kw) == UNSUPPORTED, kw


def _select(lib, dt=1, nb=4, bs=16, width=8, maxp=100, B=1, m=4, Hq=4, Hkv=2, d=128, n=4, first=1, recent=1, ptr=16, ws=16,
            wsb=1 << 30):
    P = ptr
    return lib.ts_page_select(P, dt, P, nb, bs, P, width, P, maxp, B, m, Hq, Hkv, d, n, first, recent, P, P, P, ws, wsb, None,
                              None)


def test_page_select_validation(lib):
    for kw in (dict(dt=5), dict(nb=0), dict(bs=0), dict(width=0), dict(maxp=-1), dict(B=0), dict(m=0), dict(Hq=5), dict(Hkv=0),
               dict(d=0), dict(n=0), dict(first=-1), dict(recent=-1), dict(n=1), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1),
               dict(width=2), dict(ptr=None), dict(ws=None), dict(ptr=8), dict(ws=8)):
        assert _select(lib, **kw) == INVALID, kw
    for kw in (dict(m=257), dict(d=257), dict(Hq=258, Hkv=2), dict(B=65536), dict(maxp=2 ** 31 - 1, width=2 ** 28)):
        assert _select(lib, **kw) == UNSUPPORTED, kw
    assert _select(lib, wsb=64) == WORKSPACE
    assert lib.ts_page_select_workspace(2, 60, 32, 8, 128, 4096, 16) >= 2 * 8 * 60 * 256 * 4 + 2 * 8 * 256 * 8
    assert lib.ts_page_select_workspace(2, 60, 30, 8, 128, 4096, 16) == 0


def _sparse(lib, dt=1, nb=4, bs=16, width=8, C=4, B=1, m=4, Hq=4, Hkv=2, d=128, scale=0.1, ptr=16, ws=16, wsb=1 << 30):
    P = ptr
    return lib.ts_tree_attention_sparse(P, P, P, dt, nb, bs, P, width, P, P, P, P, P, C, B, m, Hq, Hkv, d, scale, P, None, ws,
                                        wsb, None, None)


def test_tree_attention_sparse_validation(lib):
    for kw in (dict(dt=5), dict(nb=0), dict(bs=0), dict(width=0), dict(C=0), dict(B=0), dict(m=0), dict(Hq=5), dict(d=0),
               dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(ptr=None), dict(ptr=8)):
        assert _sparse(lib, **kw) == INVALID, kw
    for kw in (dict(m=257), dict(d=257), dict(B=65536), dict(C=2 ** 27)):
        assert _sparse(lib, **kw) == UNSUPPORTED, kw
    assert lib.ts_tree_attention_sparse_workspace(1, 1, 4, 5, 2, 128, 4, 16) == 0
    assert lib.ts_tree_attention_sparse_workspace(0, 1, 4, 4, 2, 64, 4, 16) > 0


def _reserve(lib, dt=1, nb=4, bs=16, hkv=2, d=128, width=8, B=2, n=8, freed=None, nfreed=0, ptr=16, ws=16, wsb=1 << 20):
    P = ptr
    return lib.ts_kv_reserve(P, P, dt, nb, bs, hkv, d, P, width, P, P, B, n, freed, nfreed, P, P, P, ws, wsb, None, None)


def test_kv_reserve_validation(lib):
    for kw in (dict(dt=5), dict(nb=0), dict(bs=0), dict(hkv=0), dict(d=0), dict(d=3), dict(width=0), dict(B=0), dict(n=0),
               dict(nfreed=-1), dict(nfreed=1), dict(ptr=None), dict(ws=None), dict(ptr=18), dict(ws=8)):
        assert _reserve(lib, **kw) == INVALID, kw
    for kw in (dict(B=4097), dict(nb=(1 << 28) + 1), dict(B=4096, width=1 << 20)):
        assert _reserve(lib, **kw) == UNSUPPORTED, kw
    assert _reserve(lib, wsb=16) == WORKSPACE
    assert lib.ts_kv_reserve_workspace(4, 16, 4097, 8) == 0


def _fork(lib, nb=4, bs=16, width=8, B=2, R=3, src=(16, 32, 48, 64, 80, 96, 112)):
    t, lens, refs, s, t2, l2, r2 = src
    return lib.ts_kv_fork(t, width, lens, refs, nb, bs, B, s, R, t2, l2, r2, None, None)


def test_kv_fork_validation(lib):
    for kw in (dict(nb=0), dict(bs=0), dict(width=0), dict(B=0), dict(R=0), dict(src=(16, 32, 48, None, 80, 96, 112)),
               dict(src=(16, 32, 48, 64, 16, 96, 112)), dict(src=(16, 32, 48, 64, 80, 32, 112)), dict(src=(16, 32, 48, 64, 80, 64, 112))):
        assert _fork(lib, **kw) == INVALID, kw
    assert _fork(lib, B=65536) == UNSUPPORTED and _fork(lib, R=65536) == UNSUPPORTED


def _compact(lib, dt=1, nb=4, bs=16, hkv=2, d=128, width=8, B=2, bounds=None, ptr=16, ws=16, wsb=1 << 20):
    P = ptr
    return lib.ts_kv_compact(P, P, dt, bounds, nb, bs, hkv, d, P, width, P, B, P, P, P, P, ws, wsb, None, None)


def test_kv_compact_validation(lib):
    for kw in (dict(dt=5), dict(nb=0), dict(bs=0), dict(hkv=0), dict(d=0), dict(d=3), dict(width=0), dict(B=0), dict(ptr=None),
               dict(ws=None), dict(bounds=8), dict(ptr=18), dict(ws=8)):
        assert _compact(lib, **kw) == INVALID, kw
    assert _compact(lib, nb=(1 << 28) + 1) == UNSUPPORTED
    assert _compact(lib, wsb=8) == WORKSPACE


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(2, 4, dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(4, 2, 16, 8)
    sel = dict(pages=torch.zeros(2, 2, 1, dtype=torch.int32), count=torch.zeros(2, 2, dtype=torch.int32),
               node_mask=torch.zeros(2, 2, 1, 1, dtype=torch.int64))
    calls = [lambda: ts.kv_page_bounds(cache, i, v),
             lambda: ts.page_select(torch.zeros(2, 1, 2, 8), torch.zeros(4, 2, 2, 8, dtype=torch.bfloat16), i, v, 2, block_size=16,
                                    max_prefix=32),
             lambda: ts.tree_attention_sparse(torch.zeros(2, 1, 2, 8), cache, cache, i, v, torch.zeros(2, 1, 1, dtype=torch.int64),
                                              sel),
             lambda: ts.kv_reserve(cache, cache, i, v, torch.zeros(4, dtype=torch.int32), 4),
             lambda: ts.kv_fork(i, v, torch.zeros(4, dtype=torch.int32), v, 16),
             lambda: ts.kv_compact(cache, cache, i, torch.zeros(4, dtype=torch.int32))]
    for call in calls:
        with pytest.raises(ValueError):
            call()


# Addresses a MiB apart; the calls below are refused, so nothing is ever read there.
_AT = {n: (i + 1) << 20 for i, n in enumerate(("k", "v", "bounds", "table", "lens", "refs", "src", "freed", "table_out", "lens_out",
                                               "refs_out", "granted", "remap", "live", "ws"))}


def _pool_call(lib, op, **at):
    p = {**_AT, **at}
    if op == "reserve":   # 300 rows of 8 pages
        return lib.ts_kv_reserve(p["k"], p["v"], 1, 500, 16, 2, 8, p["table"], 8, p["lens"], p["refs"], 300, 8, p["freed"], 70,
                                 p["table_out"], p["refs_out"], p["granted"], p["ws"], 1 << 20, None, None)
    if op == "fork":      # 300 rows become 200
        return lib.ts_kv_fork(p["table"], 8, p["lens"], p["refs"], 500, 16, 300, p["src"], 200, p["table_out"], p["lens_out"],
                              p["refs_out"], None, None)
    return lib.ts_kv_compact(p["k"], p["v"], 1, p["bounds"], 500, 16, 2, 8, p["table"], 8, p["refs"], 300, p["table_out"],
                             p["refs_out"], p["remap"], p["live"], p["ws"], 1 << 20, None, None)


@pytest.mark.parametrize("op,out,others", [
    ("reserve", "granted", ("lens", "refs", "table", "freed", "k", "v", "refs_out", "table_out", "ws")),
    ("reserve", "refs_out", ("lens", "table", "freed", "table_out", "k")),
    ("reserve", "table_out", ("lens", "refs", "freed", "v")),
    ("fork", "table_out", ("table", "lens", "refs", "src", "lens_out", "refs_out")),
    ("fork", "lens_out", ("table", "lens", "refs", "src", "refs_out")),
    ("fork", "refs_out", ("table", "lens", "src")),
    ("compact", "remap", ("table", "refs", "k", "v", "bounds", "table_out", "refs_out", "live", "ws")),
    ("compact", "live", ("table", "refs", "bounds", "table_out", "refs_out", "ws")),
    ("compact", "refs_out", ("table", "table_out", "k")),
    ("compact", "table_out", ("refs", "v"))])
def test_pool_outputs_that_overlap_are_refused(lib, op, out, others):
    for other in others:
        assert _pool_call(lib, op, **{out: _AT[other]}) == INVALID, other           # the very buffer
        if other != "live":
            assert _pool_call(lib, op, **{out: _AT[other] + 64}) == INVALID, other  # a part of it


def test_pool_updates_in_place_are_of_the_whole_buffer(lib):
    for op in ("reserve", "compact"):
        assert _pool_call(lib, op, table_out=_AT["table"] + 32) == INVALID
        assert _pool_call(lib, op, refs_out=_AT["refs"] - 4) == INVALID
    assert _pool_call(lib, "fork", refs_out=_AT["refs"] + 4) == INVALID


def _choice_call(lib, op, **at):
    p = {**{n: (i + 1) << 24 for i, n in enumerate(("q", "k", "v", "bounds", "table", "lens", "start", "mask", "pages", "count", "bits",
                                                    "out", "lse", "ws"))}, **at}
    if op == "bounds":
        return lib.ts_kv_page_bounds(p["k"], 1, 500, 16, 2, 128, p["table"], 40, p["lens"], p["start"], 6, p["bounds"], None, None)
    if op == "select":
        return lib.ts_page_select(p["q"], 1, p["bounds"], 500, 16, p["table"], 40, p["lens"], 600, 6, 9, 4, 2, 128, 4, 1, 1,
                                  p["pages"], p["count"], p["bits"], p["ws"], 1 << 22, None, None)
    return lib.ts_tree_attention_sparse(p["q"], p["k"], p["v"], 1, 500, 16, p["table"], 40, p["lens"], p["mask"], p["pages"],
                                        p["count"], p["bits"], 37, 6, 9, 4, 2, 128, 0.1, p["out"], p["lse"], p["ws"], 1 << 22,
                                        None, None)


@pytest.mark.parametrize("op,out,others", [
    ("bounds", "bounds", ("k", "table", "lens", "start")),
    ("select", "pages", ("q", "bounds", "table", "lens", "count", "bits", "ws")),
    ("select", "count", ("q", "bounds", "table", "lens", "bits", "ws")),
    ("select", "bits", ("q", "bounds", "table", "lens", "ws")),
    ("attend", "out", ("q", "k", "v", "table", "lens", "mask", "pages", "count", "bits", "lse")),
    ("attend", "lse", ("q", "k", "v", "table", "lens", "mask", "pages", "count", "bits"))])
def test_outputs_that_overlap_are_refused(lib, op, out, others):
    """(also where the other is given the output's address: 16 bytes into it)"""
    base = {n: (i + 1) << 24 for i, n in enumerate(("q", "k", "v", "bounds", "table", "lens", "start", "mask", "pages", "count", "bits",
                                                    "out", "lse", "ws"))}
    for other in others:
        assert _choice_call(lib, op, **{out: base[other]}) == INVALID, other
        assert _choice_call(lib, op, **{other: base[out] + 16}) == INVALID, other
