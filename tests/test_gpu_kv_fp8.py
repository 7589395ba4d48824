"""The 8-bit cache on the GPU against the oracle: write, read and commit bit for bit."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import Cache, F8, ints
from gpu_helpers import lib
from oracle import kv_fp8 as o8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    lib()


def _rows(rng, shape, dtype):
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-3, 4, shape[-1:]))
    return torch.from_numpy(x).to(dtype)


def _write_both(c, k, v, start, length, status=None):
    """The write on the device, and on the host's copy; compared."""
    dev = c.device()
    ts.kv_write_fp8(k.cuda(), v.cuda(), *dev, ints(c.table), ints(start), length=None if length is None else ints(length),
                    status=status)
    n = [k.shape[1]] * k.shape[0] if length is None else length
    for i, x in enumerate((k, v)):
        o8.write(c.codes[i], c.scales[i], x.double().numpy(), c.table, start, n)
    c.assert_equal(dev)
    return dev


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,sb,Hkv", [(128, 16, 16, 2), (128, 16, 1, 2), (128, 64, 16, 1), (128, 128, 128, 2), (64, 32, 32, 3),
                                         (96, 16, 8, 2), (256, 16, 16, 1), (256, 128, 128, 1), (80, 12, 4, 2), (7, 5, 5, 2),
                                         (1, 16, 16, 1), (32, 128, 64, 2)])
def test_write(dtype, d, bs, sb, Hkv):
    rng = np.random.default_rng(d + bs + sb)
    start, length = [0, 1, bs - 1, 2 * bs + 3, 17], [2 * bs + 1, 0, 2, 1, 2 * bs + 1]
    n = max(length)
    c = Cache(rng, start, n, Hkv, d, bs, sb)
    status = ts.new_status()
    _write_both(c, _rows(rng, (5, n, Hkv, d), dtype), _rows(rng, (5, n, Hkv, d), dtype), start, length, status)
    ts.check_status(status)


@pytest.mark.parametrize("n", [1, 2, 33])
def test_write_without_lengths(n):
    rng = np.random.default_rng(n)
    start = [0, 15, 16, 31]
    c = Cache(rng, start, n, 4, 128, 16, 16)
    _write_both(c, _rows(rng, (4, n, 4, 128), torch.bfloat16), _rows(rng, (4, n, 4, 128), torch.bfloat16), start, None)


def test_write_special_values():
    rng = np.random.default_rng(1)
    c = Cache(rng, [3, 0, 9], 24, 2, 128, 16, 8)
    k, v = _rows(rng, (3, 24, 2, 128), torch.float32), _rows(rng, (3, 24, 2, 128), torch.float32)
    k[0, 2, 0, 5] = float("nan")
    k[0, 3, 1, 6] = float("inf")
    k[1, 0:8] = 0.0
    k[1, 8:16] = -0.0
    k[1, 16:24] = 1e-30
    v[0, 0:8] = float("nan")
    v[1, 3, 0, 0] = -float("inf")
    v[1, 9, 1, 100] = 3e38
    v[2, 4] = 1e-45
    v[2, 12, 0] = 448.0
    v[2, 12, 1, 0] = 448.0 * 2 ** 7
    # midpoints of codes, and their neighbours
    mids = torch.from_numpy((o8._POS[:-1] + o8._POS[1:])[:124] / 2).float()
    v[2, 13, 0, :124] = mids
    v[2, 14, 0, :124] = torch.nextafter(mids, torch.tensor(1e9))
    v[2, 15, 0, :124] = -torch.nextafter(mids, torch.tensor(0.0))
    _write_both(c, k, v, [3, 0, 9], None)


def test_write_takes_slices_of_a_projection():
    rng = np.random.default_rng(2)
    start, n = [5, 40], 19
    for dtype, pad in ((torch.bfloat16, 0), (torch.float32, 0), (torch.bfloat16, 1), (torch.float32, 1)):
        c = Cache(rng, start, n, 2, 128, 16, 16)
        qkv = _rows(rng, (2, n, 8 * 128 + pad), dtype).cuda()      # with a pad the rows are off their alignment
        k = qkv[..., 4 * 128:6 * 128].unflatten(-1, (2, 128))
        v = qkv[..., 6 * 128:8 * 128].unflatten(-1, (2, 128))
        dev = c.device()
        ts.kv_write_fp8(k, v, *dev, ints(c.table), ints(start))
        for i, x in enumerate((k, v)):
            o8.write(c.codes[i], c.scales[i], x.double().cpu().numpy(), c.table, start, [n, n])
        c.assert_equal(dev)
    # head-major storage, and one row for every sequence (stride 0)
    c = Cache(rng, start, n, 2, 128, 16, 16)
    k = _rows(rng, (2, 2, n, 128), torch.bfloat16).transpose(1, 2)
    v = _rows(rng, (1, n, 2, 128), torch.bfloat16).expand(2, n, 2, 128)
    _write_both(c, k, v, start, None)


def test_write_of_off_aligned_caches():
    rng = np.random.default_rng(4)
    c = Cache(rng, [3], 20, 2, 128, 16, 16)
    dev = c.device()
    for i in (0, 1):
        buf = torch.empty(dev[i].numel() + 1, dtype=torch.uint8, device="cuda")[1:]
        buf.copy_(dev[i].view(torch.uint8).flatten())
        dev[i] = buf.view(F8).view(dev[i].shape)
    k, v = _rows(rng, (1, 20, 2, 128), torch.bfloat16), _rows(rng, (1, 20, 2, 128), torch.bfloat16)
    ts.kv_write_fp8(k.cuda(), v.cuda(), *dev, ints(c.table), ints([3]))
    for i, x in enumerate((k, v)):
        o8.write(c.codes[i], c.scales[i], x.double().numpy(), c.table, [3], [20])
    c.assert_equal(dev)
    got = ts.kv_read_fp8(*dev, ints(c.table), ints([23]), 23)
    for i in (0, 1):
        ref = o8.read(c.codes[i], c.scales[i], c.table, [23], [0], 23)
        assert np.array_equal(got[i].double().cpu().numpy(), ref)


def test_write_reads_foreign_scales_clamped():
    """Kept rows under scales that are no powers of two, or out of range."""
    rng = np.random.default_rng(7)
    c = Cache(rng, [8, 8, 8, 8], 8, 1, 128, 16, 16)
    for i in (0, 1):
        for b, s in enumerate((0.3, 0.0, float("nan"), -1.0)):
            c.scales[i][c.table[b, 0]] = s
        c.codes[i][c.table[0, 0], :, :8] &= 0xF8           # (one significant bit: the product with 0.3 is rounded once)
    x = [_rows(rng, (4, 8, 1, 128), torch.float32) for _ in "kv"]
    _write_both(c, *x, [8] * 4, None)


def test_write_device_checks():
    rng = np.random.default_rng(8)
    start = [5, -1, 20, 30, 3]
    c = Cache(rng, [5, 5, 20, 5, 3], 10, 2, 128, 16, 16)
    c.table = np.pad(c.table, ((0, 0), (0, 1)), constant_values=-1)
    c.table[4, 0] = 10 ** 6
    k, v = _rows(rng, (5, 10, 2, 128), torch.bfloat16), _rows(rng, (5, 10, 2, 128), torch.bfloat16)
    length = [10, 10, 11, 10, 10]                                     # sequence 2: longer than n
    dev = c.device()
    status = ts.new_status()
    ts.kv_write_fp8(k.cuda(), v.cuda(), *dev, ints(c.table), ints([5, -1, 20, 47, 3]), length=ints(length), status=status)
    with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
        ts.check_status(status)
    for i, x in enumerate((k, v)):
        o8.write_one(c.codes[i], c.scales[i], x[0].double().numpy(), c.table[0], 5)
    c.assert_equal(dev)
    del start


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,sb,Hkv", [(128, 16, 16, 2), (128, 64, 1, 2), (64, 32, 8, 3), (80, 12, 4, 2), (7, 5, 5, 2), (256, 16, 2, 1)])
def test_read(dtype, d, bs, sb, Hkv):
    rng = np.random.default_rng(d + bs)
    lens, start, n = [3 * bs + 5, 0, 1, bs, 2 * bs + 1], [2, 0, 0, bs, 2 * bs], 2 * bs + 3
    c = Cache(rng, lens, 0, Hkv, d, bs, sb)
    c.codes[0].reshape(-1)[::97] = 127                                # NaN codes
    status = ts.new_status()
    k, v = ts.kv_read_fp8(*c.device(), ints(c.table), ints(lens), n, start_len=ints(start), dtype=dtype, status=status)
    ts.check_status(status)
    for i, got in enumerate((k, v)):
        ref = o8.read(c.codes[i], c.scales[i], c.table, lens, start, n)
        assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)
    out = (torch.full_like(k, 3.0), torch.full_like(v, 3.0))
    r = ts.kv_read_fp8(*c.device(), ints(c.table), ints(lens), n, start_len=ints(start), out=out)
    assert r[0] is out[0] and torch.equal(out[0].nan_to_num(5.0), k.nan_to_num(5.0)) and torch.equal(out[1], v)


def test_read_device_checks():
    rng = np.random.default_rng(9)
    c = Cache(rng, [20, 20, 20], 0, 1, 128, 16, 16)
    c.table[1, 1] = -5
    status = ts.new_status()
    k, _ = ts.kv_read_fp8(*c.device(), ints(c.table), ints([20, 20, 33]), 20, status=status)
    with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
        ts.check_status(status)
    ref = o8.read(c.codes[0], c.scales[0], np.abs(c.table) % 3, [20, 16, 0], [0, 0, 0], 20)
    ref[0] = o8.read(c.codes[0], c.scales[0], c.table[:1], [20], [0], 20)[0]
    ref[1, :16] = o8.read(c.codes[0], c.scales[0], c.table[1:2, :1], [16], [0], 16)[0]
    assert np.array_equal(k.double().cpu().numpy(), ref)


def _paths(rng, B, m, most):
    path, length = np.full((B, m), -1, dtype=np.int32), []
    for b in range(B):
        a = int(rng.integers(1, most + 1))
        path[b, :a] = [0] + sorted(rng.choice(np.arange(1, m), a - 1, replace=False).tolist())
        length.append(a)
    return path, np.array(length, dtype=np.int32)


@pytest.mark.parametrize("d,bs,sb,Hkv,m,most", [(128, 16, 16, 2, 60, 7), (128, 16, 4, 1, 9, 9), (128, 64, 64, 2, 128, 17),
                                               (64, 32, 32, 3, 8, 3), (80, 12, 4, 2, 20, 5), (7, 5, 5, 2, 11, 4), (128, 16, 1, 2, 1, 1),
                                               (256, 16, 8, 1, 256, 200), (36, 16, 16, 2, 10, 10)])
def test_commit(d, bs, sb, Hkv, m, most):
    rng = np.random.default_rng(d + m)
    lens = [0, 1, bs - 1, 3 * bs, 2 * bs + 3]
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    path, length = _paths(rng, 5, m, most)
    dev = c.device()
    table, prefix = ints(c.table), ints(lens)
    status = ts.new_status()
    r = ts.kv_commit_fp8(*dev, table, prefix, ints(path), ints(length), status=status)
    ts.check_status(status)
    t, p, freed, count = o8.commit(c.codes, c.scales, c.table, lens, path, length, m)
    c.assert_equal(dev)
    for name, ref in (("block_table", t), ("prefix_len", p), ("freed_blocks", freed), ("freed_count", count)):
        assert np.array_equal(r[name].cpu().numpy(), ref), name
    assert torch.equal(table, ints(c.table)) and torch.equal(prefix, ints(lens))       # the old state is as it was


def test_commit_in_place_and_contract():
    rng = np.random.default_rng(11)
    lens, m = [5, 16, 2, 7], 6
    c = Cache(rng, lens, m, 2, 128, 16, 8)
    path, length = np.full((4, m), -1, dtype=np.int32), np.array([2, 3, 2, 9], dtype=np.int32)
    path[0, :2], path[1, :3], path[2, :2] = [0, 4], [0, 3, 3], [1, 2]                  # 1, 2: not a path; 3: too long
    dev = c.device()
    table, prefix = ints(c.table), ints(lens)
    status = ts.new_status()
    out = dict(block_table=table, prefix_len=prefix, freed_blocks=torch.empty_like(table), freed_count=torch.empty_like(prefix))
    ts.kv_commit_fp8(*dev, table, prefix, ints(path), ints(length), out=out, status=status)
    with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
        ts.check_status(status)
    codes, scales = [x for x in c.codes], [x for x in c.scales]
    t, p, freed, count = o8.commit(codes, scales, c.table[:1], lens[:1], path[:1], length[:1], m)
    c.assert_equal(dev)
    assert np.array_equal(table.cpu().numpy(), np.concatenate([t, c.table[1:]]))
    assert prefix.tolist() == [p[0]] + lens[1:] and out["freed_count"].tolist() == [count[0], 0, 0, 0]
    assert (out["freed_blocks"][1:] == -1).all()
    with pytest.raises(ValueError, match="shares memory"):
        ts.kv_commit_fp8(*dev, table, prefix, ints(path), ints(length),
                         out=dict(out, block_table=torch.empty_like(table), freed_blocks=table))


def test_refusals():
    rng = np.random.default_rng(12)
    c = Cache(rng, [5], 4, 2, 128, 16, 8)
    dev = c.device()
    k = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    table, start = ints(c.table), ints([5])
    good = (k, k.clone(), *dev, table, start)

    def broken(i, x):
        a = list(good)
        a[i] = x
        return a

    for i, x, why in ((0, k.half(), "dtype"), (0, k.cpu(), "CUDA"), (1, k.float(), "bfloat16"), (0, k[..., :64], "shape"),
                      (0, k.transpose(2, 3), "shape"), (0, k[0], "dimensions"), (2, dev[0].view(torch.uint8), "float8"),
                      (4, dev[2][:, :, :1].expand(-1, -1, 3).contiguous(), "divisor"), (4, dev[2].double(), "float32"),
                      (5, dev[3][:1], "shape"), (6, table.long(), "int32"), (7, ints([5, 5]), "shape")):
        with pytest.raises(ValueError, match=why):
            ts.kv_write_fp8(*broken(i, x))
    strided = torch.zeros(1, 4, 2, 256, dtype=torch.bfloat16, device="cuda")[..., ::2]
    with pytest.raises(ValueError, match="contiguous head rows"):
        ts.kv_write_fp8(*broken(0, strided))
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        ts.kv_write_fp8(k[:, :0], k[:, :0], *good[2:])
    with pytest.raises(ValueError, match="shape"):
        ts.kv_write_fp8(*good, length=ints([1, 1]))
    with pytest.raises(ValueError, match="dtype"):
        ts.kv_read_fp8(*dev, table, start, 4, dtype=torch.float16)
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        ts.kv_read_fp8(*dev, table, start, 0)
    # a cache that shares memory with what is written to it
    shared = dev[0].view(torch.uint8).flatten()[:2048].view(torch.bfloat16).view(1, 4, 2, 128)
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        ts.kv_write_fp8(*broken(0, shared))
    with pytest.raises(ts.TreeSpecError, match="INVALID"):
        ts.kv_read_fp8(*dev, table, start, 4, out=(k, k))
    c.assert_equal(dev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,bs,sb,Hkv", [(128, 16, 1, 2), (128, 16, 2, 1), (128, 32, 4, 3), (128, 64, 8, 2), (64, 32, 1, 2), (64, 64, 16, 1), (64, 16, 4, 2),
                                         (256, 16, 2, 2), (256, 8, 1, 1), (32, 128, 2, 2), (32, 64, 8, 1), (16, 128, 32, 1), (8, 256, 4, 1)])
def test_write_of_small_blocks(dtype, d, bs, sb, Hkv):
    """Blocks of which a warp takes several, at every place of a page."""
    rng = np.random.default_rng(d * bs + sb)
    start = [0, 1, bs - 1, bs, bs // 2 + 3, 2 * bs + sb, 5, 2 * bs - sb]
    length = [2 * bs, 1, 2, bs + 1, 0, 3, sb, 2 * sb]
    n = max(length)
    c = Cache(rng, start, n, Hkv, d, bs, sb)
    status = ts.new_status()
    k, v = _rows(rng, (8, n, Hkv, d), dtype), _rows(rng, (8, n, Hkv, d), dtype)
    k[0, ::3], v[0, 1::5] = 0.0, float("nan")
    k[3, :, 0] *= 2.0 ** 20
    _write_both(c, k, v, start, length, status)
    ts.check_status(status)


@pytest.mark.parametrize("dtype,d,bs,sb,Hkv", [(torch.bfloat16, 128, 16, 1, 4), (torch.bfloat16, 64, 64, 2, 4), (torch.bfloat16, 256, 16, 2, 4),
                                               (torch.float32, 128, 32, 4, 2), (torch.float32, 32, 64, 1, 4)])
def test_write_of_many_small_blocks(dtype, d, bs, sb, Hkv):
    """As many blocks as a warp takes a run of: prompts behind prefixes that end anywhere."""
    rng = np.random.default_rng(d + bs + sb)
    start = [0, 1, 3 * bs - 1, bs + bs // 2 + 1]
    n = -(-32768 * sb // (8 * Hkv)) + 3
    length = [n, n - 1, n - bs - 2, n]
    c = Cache(rng, start, n, Hkv, d, bs, sb)
    status = ts.new_status()
    k, v = _rows(rng, (4, n, Hkv, d), dtype), _rows(rng, (4, n, Hkv, d), dtype)
    k[0, ::3], v[0, 1::5] = 0.0, float("nan")
    _write_both(c, k, v, start, length, status)
    ts.check_status(status)
    # one sequence too long, and one page out of range: the others are written
    c2 = Cache(rng, start, n, Hkv, d, bs, sb)
    c2.table[1, 2] = -1
    dev, before = c2.device(), [t.view(torch.uint8).clone() for t in c2.device()]
    starts = list(start)
    starts[2] = c2.table.shape[1] * bs - n + 1
    ts.kv_write_fp8(k.cuda(), v.cuda(), *dev, ints(c2.table), ints(starts), status=status)
    with pytest.raises(ts.TreeSpecError, match="DEVICE_CHECK"):
        ts.check_status(status)
    for t, old in zip(dev, before):
        pages = c2.table[2][c2.table[2] >= 0]
        assert torch.equal(t.view(torch.uint8)[pages], old[pages])              # as they were
        assert not torch.equal(t.view(torch.uint8)[c2.table[0, :2]], old[c2.table[0, :2]])
