"""kv_commit at positions and table cells just below 2^31."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from gpu_helpers import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    lib()


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _path(m, a):
    path = torch.full((1, m), -1, dtype=torch.int32, device="cuda")
    path[0, :a] = _ints([0] + sorted(np.random.default_rng(m).choice(np.arange(1, m), a - 1, replace=False)))
    return path


def _commit(*args, **kw):
    r = ts.kv_commit(*args, **kw)
    return r["freed_blocks"], r["freed_count"]


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 5)])
@pytest.mark.parametrize("bs,m,a", [(1024, 20, 7), (1024, 256, 256), (128, 256, 3)])
def test_near_2_to_31(dtype, d, bs, m, a):
    """As at the beginning of a cache: the same rows and pages; the longest prefix that the tree may follow."""
    cells = (1 << 31) // bs
    L = (1 << 31) - 1 - m
    p0 = L // bs
    g = torch.Generator(device="cuda").manual_seed(bs)
    start = [torch.randn(4, 2, bs, d, generator=g, device="cuda").to(dtype) for _ in "kv"]
    near = _ints([[2, 0, 3]])[:, :cells - p0].contiguous()
    far = torch.full((1, cells), -1, dtype=torch.int32, device="cuda")
    far[0, p0:] = near[0, :cells - p0]
    results = []
    for table, prefix in ((near, L - p0 * bs), (far, L)):
        dev, status, lens, table = [t.clone() for t in start], ts.new_status(), _ints([prefix]), table.clone()
        freed, count = _commit(*dev, table, lens, _path(m, a), _ints([a]), status=status)
        ts.check_status(status)
        assert lens.item() == prefix + a
        results.append((dev, table, freed, count.item()))
    (d0, t0, f0, n0), (d1, t1, f1, n1) = results
    assert all(torch.equal(x, y) for x, y in zip(d0, d1)) and n0 == n1
    assert torch.equal(t0[0], t1[0, p0:]) and (t1[0, :p0] == -1).all()
    assert torch.equal(f0[0, :n0], f1[0, :n0]) and (f1[0, n0:] == -1).all()


def test_a_row_of_2_to_31_pages():
    """Pages of one token; and a tree that would end behind the last position is refused."""
    m, a, L = 40, 5, (1 << 31) - 257
    cells = L + m
    k, v = [torch.arange(64.0, device="cuda").view(64, 1, 1, 1).expand(64, 1, 1, 4).contiguous() for _ in "kv"]
    table = torch.full((1, cells), -1, dtype=torch.int32, device="cuda")
    table[0, L:] = torch.arange(m, dtype=torch.int32, device="cuda")
    prefix, status = _ints([L]), ts.new_status()
    path = torch.full((1, m), -1, dtype=torch.int32, device="cuda")
    path[0, :a] = _ints([0, 3, 7, 20, 39])
    freed, count = _commit(k, v, table, prefix, path, _ints([a]), status=status)
    ts.check_status(status)
    assert prefix.item() == L + a and count.item() == m - a
    assert torch.equal(table[0, L:L + a], torch.arange(a, dtype=torch.int32, device="cuda")) and (table[0, L + a:] == -1).all()
    assert torch.equal(freed[0, :m - a], torch.arange(a, m, dtype=torch.int32, device="cuda")) and (freed[0, -(1 << 20):] == -1).all()
    for t in (k, v):
        assert t[:a, 0, 0, 0].tolist() == [0, 3, 7, 20, 39] and torch.equal(t[a:, 0, 0, 0], torch.arange(a, 64.0, device="cuda"))


def test_a_tree_behind_the_last_position_is_refused():
    table = torch.zeros((1, 1 << 27), dtype=torch.int32, device="cuda")     # room for 2^32 positions
    k, v = [torch.ones(2, 1, 32, 8, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    prefix, status = _ints([(1 << 31) - 20]), ts.new_status()
    freed, count = _commit(k, v, table, prefix, _path(40, 30), _ints([30]), status=status)
    with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
        ts.check_status(status)
    assert prefix.item() == (1 << 31) - 20 and count.item() == 0 and (freed == -1).all() and (table == 0).all()
    assert (k == 1).all() and (v == 1).all()
