"""Tree attention over the 8-bit cache against fp64, on both paths."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from fp8_helpers import Cache, assert_within, attention_bounds, ints, tree_mask, words
from gpu_helpers import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    lib()


def _query(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape) * np.exp2(rng.integers(-2, 2, shape[:-1] + (1,)))).to(dtype)


def _attend(c, q, mask, scale=None, max_prefix=None, **kw):
    status = ts.new_status()
    B, m, Hq, d = q.shape
    top = int(c.lens.max()) if max_prefix is None else max_prefix
    need = ts.library().ts_tree_attention_fp8_workspace(int(q.dtype == torch.bfloat16), B, m, Hq, c.codes[0].shape[1], d, top, c.bs)
    kw.setdefault("workspace", torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))      # (any contents, NaN here)
    r = ts.tree_attention_fp8(q.cuda(), *c.device(), ints(c.table), ints(c.lens), words(mask),
                              max_prefix=top, scale=scale, status=status, **kw)
    ts.check_status(status)
    return r


def _check(c, q, mask, scale=None, **kw):
    out, lse = _attend(c, q, mask, scale, **kw)
    s = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    ref, ref_lse, bo, bl = attention_bounds(q.double().numpy(), *c.values(), c.table, c.lens, mask, s, q.dtype == torch.bfloat16)
    assert_within(lse, ref_lse, bl, "lse")
    assert_within(out, ref, bo, "out")
    return out, lse


# (lens, m, Hq, Hkv, bs, sb): 1 to 16, 32, 64, 128 rows per KV head, and several groups of 128
TC = [((0,), 1, 1, 1, 16, 16), ((1, 300), 1, 4, 1, 16, 16), ((127, 128, 129), 1, 8, 2, 32, 8), ((1000, 0, 77), 3, 10, 2, 64, 64),
      ((200, 513), 4, 16, 4, 16, 1), ((90, 2000), 8, 8, 2, 128, 128), ((40, 300, 5), 17, 6, 2, 16, 16), ((255, 640), 60, 2, 2, 64, 16),
      ((250,), 64, 4, 2, 16, 16), ((33, 500), 9, 64, 2, 16, 4), ((700, 3), 60, 16, 2, 16, 16), ((100,), 130, 2, 1, 32, 32),
      ((60, 129), 256, 2, 2, 16, 16), ((1500,), 33, 40, 5, 16, 16)]


@pytest.mark.parametrize("lens,m,Hq,Hkv,bs,sb", TC)
def test_tensor_core_path(lens, m, Hq, Hkv, bs, sb):
    rng = np.random.default_rng(sum(lens) + m + Hq)
    c = Cache(rng, lens, m, Hkv, 128, bs, sb)
    _check(c, _query(rng, (len(lens), m, Hq, 128), torch.bfloat16), tree_mask(rng, len(lens), m))


@pytest.mark.parametrize("dtype,lens,m,Hq,Hkv,d,bs,sb", [
    (torch.float32, (0, 1), 1, 2, 1, 128, 16, 16), (torch.float32, (63, 64, 65), 8, 8, 2, 64, 16, 8),
    (torch.float32, (700, 20), 5, 14, 2, 128, 12, 4), (torch.float32, (3000,), 1, 4, 4, 256, 64, 64),
    (torch.float32, (100, 9), 65, 4, 2, 80, 16, 16), (torch.float32, (40,), 3, 3, 1, 7, 5, 5), (torch.float32, (300,), 2, 2, 2, 192, 16, 2),
    (torch.bfloat16, (500, 70), 9, 8, 2, 64, 16, 16), (torch.bfloat16, (129,), 4, 4, 1, 128, 8, 8), (torch.bfloat16, (70,), 2, 6, 2, 33, 16, 1)])
def test_cuda_core_path(dtype, lens, m, Hq, Hkv, d, bs, sb):
    rng = np.random.default_rng(sum(lens) + m + d)
    c = Cache(rng, lens, m, Hkv, d, bs, sb)
    _check(c, _query(rng, (len(lens), m, Hq, d), dtype), tree_mask(rng, len(lens), m))


@pytest.mark.parametrize("sb", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("m,Hq", [(2, 4), (6, 8), (40, 4)])
def test_every_scale_block(m, Hq, sb):
    rng = np.random.default_rng(sb + m)
    c = Cache(rng, (400, 63, 5), m, 2, 128, 64, sb, spread=6)
    _check(c, _query(rng, (3, m, Hq, 128), torch.bfloat16), tree_mask(rng, 3, m))
