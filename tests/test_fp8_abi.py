"""Host-side validation of the 8-bit cache's calls (CPU only: every call here is refused before any launch)."""
import ctypes

import pytest

import speculative_decoding_tree_eagle_gb300 as ts
from speculative_decoding_tree_eagle_gb300 import build as tsbuild

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    tsbuild.build()
    return ts.library()


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def _places(n, **given):
    """n addresses a GiB apart, some of them replaced by position."""
    at = [(i + 1) * GB for i in range(n)]
    for name, x in given.items():
        at[int(name[1:])] = x
    return at


def _write(lib, dt=1, nb=4, bs=16, sb=8, hkv=2, d=128, width=4, B=2, n=8, ks=(2048, 256, 128), vs=(2048, 256, 128), **at):
    k, v, kc, vc, sk, sv, t, start, length = _places(9, **at)
    return lib.ts_kv_write_fp8(k, v, dt, _strides(*ks), _strides(*vs), kc, vc, sk, sv, nb, bs, sb, hkv, d, t, width, start, length, B,
                               n, None, None)


def test_write_validation(lib):
    for kw in (dict(dt=2), dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=5), dict(sb=32), dict(hkv=0), dict(d=0), dict(width=0), dict(B=0),
               dict(n=0), dict(ks=(-1, 256, 128)), dict(vs=(2048, 1 << 41, 128)), dict(p0=GB + 1), dict(dt=0, p1=2 * GB + 2),
               dict(p4=5 * GB + 2), dict(p5=6 * GB + 1), *({f"p{i}": None} for i in range(8))):
        assert _write(lib, **kw) == INVALID, kw
    for kw in (dict(d=257), dict(B=65536), dict(hkv=32768)):
        assert _write(lib, **kw) == UNSUPPORTED, kw
    # an output on an input or on another output, by a byte
    for kw in (dict(p3=3 * GB + 4 * 2 * 16 * 128 - 1), dict(p0=3 * GB + 4), dict(p6=5 * GB), dict(p7=6 * GB), dict(p8=4 * GB), dict(p5=5 * GB + 60)):
        assert _write(lib, **kw) == INVALID, kw


def _read(lib, dt=1, nb=4, bs=16, sb=8, hkv=2, d=128, width=4, B=2, n=8, **at):
    kc, vc, sk, sv, t, prefix, start, k, v = _places(9, **at)
    return lib.ts_kv_read_fp8(kc, vc, sk, sv, nb, bs, sb, hkv, d, t, width, prefix, start, B, n, k, v, dt, None, None)


def test_read_validation(lib):
    for kw in (dict(dt=2), dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=5), dict(hkv=0), dict(d=0), dict(width=0), dict(B=0), dict(n=0),
               dict(p7=8 * GB + 1), dict(dt=0, p8=9 * GB + 2), dict(p2=3 * GB + 2),
               *({f"p{i}": None} for i in (0, 1, 2, 3, 4, 5, 7, 8))):
        assert _read(lib, **kw) == INVALID, kw
    for kw in (dict(d=257), dict(B=65536)):
        assert _read(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(p8=8 * GB + 2), dict(p7=GB), dict(p8=3 * GB), dict(p7=5 * GB), dict(p7=6 * GB), dict(p8=7 * GB)):
        assert _read(lib, **kw) == INVALID, kw


def _commit(lib, nb=4, bs=16, sb=8, hkv=2, d=128, width=4, B=2, m=8, **at):
    kc, vc, sk, sv, t, prefix, path, alen, t2, p2, freed, count = _places(12, **at)
    return lib.ts_kv_commit_fp8(kc, vc, sk, sv, nb, bs, sb, hkv, d, t, width, prefix, path, alen, B, m, t2, p2, freed, count, None,
                                None)


def test_commit_validation(lib):
    for kw in (dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=3), dict(hkv=0), dict(d=0), dict(width=0), dict(B=0), dict(m=0),
               dict(p3=4 * GB + 1), *({f"p{i}": None} for i in range(12))):
        assert _commit(lib, **kw) == INVALID, kw
    for kw in (dict(d=257), dict(B=65536), dict(m=257)):
        assert _commit(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(p8=5 * GB + 4), dict(p9=6 * GB + 4), dict(p10=5 * GB), dict(p11=8 * GB), dict(p1=GB), dict(p10=9 * GB), dict(p6=3 * GB)):
        assert _commit(lib, **kw) == INVALID, kw


def _attend(lib, dt=1, nb=4, bs=16, sb=8, width=40, maxp=100, B=2, m=4, Hq=4, Hkv=2, d=128, scale=0.1, wsb=1 << 29, **at):
    q, kc, vc, sk, sv, t, prefix, mask, out, lse, ws = _places(11, **at)
    return lib.ts_tree_attention_fp8(q, dt, kc, vc, sk, sv, nb, bs, sb, t, width, prefix, maxp, mask, B, m, Hq, Hkv, d, scale, out, lse,
                                     ws, wsb, None, None)


def test_attention_validation(lib):
    for kw in (dict(dt=5), dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=7), dict(width=0), dict(B=0), dict(m=0), dict(Hq=5), dict(Hkv=0),
               dict(d=0), dict(maxp=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(p3=4 * GB + 2), dict(p0=GB + 8), dict(p1=2 * GB + 8), dict(p2=3 * GB + 4), dict(p8=9 * GB + 8), dict(dt=0, p0=GB + 2),
               *({f"p{i}": None} for i in range(9))):
        assert _attend(lib, **kw) == INVALID, kw
    for kw in (dict(m=257), dict(d=257), dict(B=65536), dict(maxp=(1 << 30) + 1)):
        assert _attend(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(p8=GB), dict(p9=8 * GB), dict(p9=9 * GB + 4), dict(p8=6 * GB)):
        assert _attend(lib, **kw) == INVALID, kw


def test_attention_workspace_of_refused_sizes(lib):
    for a in ((2, 1, 4, 4, 2, 128, 100, 16), (1, 0, 4, 4, 2, 128, 100, 16), (1, 1, 257, 4, 2, 128, 100, 16), (1, 1, 4, 5, 2, 128, 100, 16),
              (1, 1, 4, 4, 2, 257, 100, 16), (1, 1, 4, 4, 2, 128, -1, 16), (1, 1, 4, 4, 2, 128, 100, 0),
              (1, 1, 4, 4, 2, 128, (1 << 30) + 1, 16)):
        assert lib.ts_tree_attention_fp8_workspace(*a) == 0, a


def _reserve(lib, nb=4, bs=16, sb=8, hkv=2, d=128, width=8, B=2, n=8, nfreed=4, wsb=1 << 20, **at):
    kc, vc, sk, sv, t, prefix, refs, freed, t2, r2, granted, ws = _places(12, **at)
    return lib.ts_kv_reserve_fp8(kc, vc, sk, sv, nb, bs, sb, hkv, d, t, width, prefix, refs, B, n, freed, nfreed, t2, r2, granted, ws, wsb,
                                 None, None)


def test_reserve_validation(lib):
    for kw in (dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=5), dict(hkv=0), dict(d=0), dict(d=6), dict(width=0), dict(B=0), dict(n=0),
               dict(nfreed=-1), dict(p0=GB + 2), dict(p2=3 * GB + 1), dict(p11=12 * GB + 8), *({f"p{i}": None} for i in range(12))):
        assert _reserve(lib, **kw) == INVALID, kw
    for kw in (dict(B=4097), dict(B=4096, width=1 << 20), dict(d=260)):
        assert _reserve(lib, **kw) == UNSUPPORTED, kw
    assert _reserve(lib, wsb=16) == WORKSPACE
    # the caches and their scales lie apart; so do the outputs from them
    for kw in (dict(p1=GB), dict(p3=3 * GB), dict(p2=GB + 64), dict(p8=3 * GB), dict(p10=4 * GB + 4), dict(p11=2 * GB), dict(p9=5 * GB)):
        assert _reserve(lib, **kw) == INVALID, kw


def _compact(lib, nb=4, bs=16, sb=8, hkv=2, d=128, width=8, B=2, wsb=1 << 20, **at):
    kc, vc, sk, sv, t, refs, t2, r2, remap, live, ws = _places(11, **at)
    return lib.ts_kv_compact_fp8(kc, vc, sk, sv, nb, bs, sb, hkv, d, t, width, refs, B, t2, r2, remap, live, ws, wsb, None, None)


def test_compact_validation(lib):
    for kw in (dict(nb=0), dict(bs=0), dict(sb=0), dict(sb=5), dict(hkv=0), dict(d=0), dict(d=6), dict(width=0), dict(B=0), dict(p1=2 * GB + 2),
               dict(p3=4 * GB + 2), dict(p10=11 * GB + 8), *({f"p{i}": None} for i in range(11))):
        assert _compact(lib, **kw) == INVALID, kw
    for kw in (dict(d=260), dict(B=65536)):
        assert _compact(lib, **kw) == UNSUPPORTED, kw
    assert _compact(lib, wsb=16) == WORKSPACE
    for kw in (dict(p1=GB), dict(p3=3 * GB), dict(p2=2 * GB), dict(p6=3 * GB), dict(p8=4 * GB + 4), dict(p9=2 * GB), dict(p7=5 * GB)):
        assert _compact(lib, **kw) == INVALID, kw
