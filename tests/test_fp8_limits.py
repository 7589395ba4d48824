"""Sizes at which the 8-bit cache's calls refuse, and the arithmetic of the queries' split (CPU only)."""
import ctypes

import pytest

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
