"""Sizes at which the 8-bit cache's calls refuse, and the arithmetic of the queries' split (CPU only)."""
import ctypes

import pytest
import torch

import speculative_decoding_tree_eagle_gb300 as ts
from speculative_decoding_tree_eagle_gb300 import build as tsbuild

UNSUPPORTED = -2
TB = 1 << 40


@pytest.fixture(scope="module")
def lib():
    tsbuild.build()
    return ts.library()


@pytest.mark.parametrize("bs,sb,d", [(1 << 24, 1 << 24, 128), (1 << 23, 1 << 23, 256), (1 << 24, 1 << 24, 255), (1 << 30, 1 << 30, 2),
                                     ((1 << 31) - 1, (1 << 31) - 1, 3), ((1 << 31) - 1, (1 << 31) - 1, 1),
                                     ((1 << 31) - 256, (1 << 31) - 256, 1)])
def test_scale_blocks_of_more_elements_than_are_counted(lib, bs, sb, d):
    """A scale block of 2^31 - 256 elements of a head and more is neither written nor committed."""
    at = [(i + 1) * TB * 16 for i in range(12)]
    strides = (ctypes.c_int64 * 3)(4 * d, d, d)
    assert lib.ts_kv_write_fp8(at[0], at[1], 1, strides, strides, *at[2:6], 1, bs, sb, 1, d, at[6], 4, at[7], None, 1, 4, None,
                               None) == UNSUPPORTED
    assert lib.ts_kv_commit_fp8(*at[:4], 1, bs, sb, 1, d, at[4], 4, *at[5:8], 1, 4, *at[8:12], None, None) == UNSUPPORTED


def test_split_of_the_queries():
    """A query row's largest element lies in [128, 256) when its elements are taken apart into the nearest e4m3 and the e5m2 nearest to
    the rest.  Exact from 2^-6 on, 2^-13 of the largest at most; below, e4m3's steps are 2^-9, the rest is 2^-10 at most and e5m2's
    steps there are 2^-13: off by 2^-14 at most, 2^-21 of the largest."""
    y = torch.arange(0, 0x4380, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()   # every bf16 value of [0, 256)
    y = torch.cat([y, -y])
    hi = y.to(torch.float8_e4m3fn).float()
    off = (y - hi - (y - hi).to(torch.float8_e5m2).float()).abs()
    assert y.max() < 256 and off[y.abs() >= 2.0 ** -6].max() == 0
    assert off.max() == 2.0 ** -14
