"""Helpers of the 8-bit cache's GPU tests: seeded caches on the host and the device, and derived error bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv_fp8 as o8

F8 = torch.float8_e4m3fn


class Cache:
    """Codes (uint8) and scales of K and V on the host, with a block table."""

    def __init__(self, rng, lens, more, Hkv, d, bs, sb, spread=3, spare=3):
        pages = [-(-(n + more) // bs) for n in lens]
        nb = sum(pages) + spare
        perm = rng.permutation(nb)
        width = max(1, max(pages))
        self.table = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = perm[at:at + p]
            at += p
        self.spare = perm[at:]
        self.lens, self.bs, self.sb = np.asarray(lens, dtype=np.int32), bs, sb
        self.codes, self.scales = [], []
        for _ in "kv":
            x = rng.standard_normal((nb, Hkv, bs, d)) * 100 * np.exp2(rng.integers(-2, 1, (1, Hkv, 1, d)))
            self.codes.append(o8.encode(x))
            self.scales.append(np.exp2(rng.integers(-9 - spread, -8 + spread, (nb, Hkv, bs // sb))).astype(np.float32))

    def values(self):
        return [o8.values(c, s) for c, s in zip(self.codes, self.scales)]

    def device(self):
        """(k_cache, v_cache, k_scale, v_scale) on the GPU."""
        return ([torch.from_numpy(c.copy()).cuda().view(F8) for c in self.codes]
                + [torch.from_numpy(s.copy()).cuda() for s in self.scales])

    def assert_equal(self, dev):
        for c, t in zip(self.codes, dev[:2]):
            got = t.view(torch.uint8).cpu().numpy()
            nan = (c & 127) == 127
            assert np.array_equal((got & 127) == 127, nan), "NaN codes differ"
            bad = (got != c) & ~nan
            assert not bad.any(), f"{bad.sum()} codes differ, first at {np.argwhere(bad)[0]}"
        for s, t in zip(self.scales, dev[2:]):
            assert np.array_equal(t.cpu().numpy(), s.astype(np.float32))


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def words(mask_bool):
    B, m, _ = mask_bool.shape
    W = (m + 63) // 64
    out = np.zeros((B, m, W), dtype=np.uint64)
    for b, i, j in np.argwhere(mask_bool):
        out[b, i, j >> 6] |= np.uint64(1) << np.uint64(j & 63)
    return torch.from_numpy(out.view(np.int64)).cuda()


def tree_mask(rng, B, m):
    import oracle
    return np.stack([oracle.ancestor_mask([-1] + [int(rng.integers(max(0, i // 2 - 3), i)) for i in range(1, m)]) for _ in range(B)])


def attention_bounds(q, k, v, table, prefix, mask, scale, bf16):
    """(out, lse, bound of out, bound of lse) in fp64, the bounds from the arithmetic of the kernels.

    Per row: a score is off by at most E = scale * (2^-24 max|q| sum|k| (bf16 queries' split: 2^-25 of the largest, twice for
    the row's power-of-two range) + (d + 8) 2^-23 sum|q k|) (fp32 products and sums) + 2^-21 (1 + |s|) (the exponent's
    multiply-add, maximum and 2^x); the weights by 2E relative, fp16 weights by 2^-11 more; sums of n terms in fp32 by
    n 2^-24.  The output's rounding is half a step: 2^-8 of bf16, 2^-24 of fp32.  Weights below fp16's range: n 2^-31 of
    the largest contribution."""
    q = np.asarray(q, dtype=np.float64)
    B, m, Hq, d = q.shape
    bs, g = k.shape[2], Hq // k.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, m, Hq), -np.inf)
    bo, bl = np.zeros(q.shape), np.zeros((B, m, Hq))
    for b in range(B):
        L = int(prefix[b])
        pos = np.arange(L + m)
        pages = np.asarray(table[b])[pos // bs]
        ks, vs = k[pages, :, pos % bs], v[pages, :, pos % bs]
        seen = np.concatenate([np.ones((m, L), dtype=bool), mask[b]], 1)
        n = L + m
        for h in range(Hq):
            K, V, x = ks[:, h // g], vs[:, h // g], q[b, :, h]
            s = np.where(seen, scale * (x @ K.T), -np.inf)
            top = s.max(1, keepdims=True)
            some = np.isfinite(top[:, 0])
            with np.errstate(all="ignore"):
                w = np.exp(s - top)
                z = w.sum(1, keepdims=True)
                p = np.where(seen, w / z, 0.0)
                out[b, :, h] = np.where(some[:, None], p @ V, 0.0)
                lse[b, :, h] = np.where(some, (top + np.log(z))[:, 0], -np.inf)
            split = 2.0 ** -24 * np.abs(x).max(1) * np.abs(K).sum(1).max() if bf16 else 0.0
            E = scale * (split + (d + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(K).T).max(1))
            E = E + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(s), s, 0.0)).max(1))
            A = p @ np.abs(V)
            rel = 2 * E + n * 2.0 ** -24 + (2.0 ** -11 if bf16 else 0.0)
            lost = n * 2.0 ** -31 * (p.max(1) * np.abs(V).max())[:, None] if bf16 else 0.0
            bo[b, :, h] = np.abs(out[b, :, h]) * (2.0 ** -8 if bf16 else 2.0 ** -23) + 1.5 * rel[:, None] * A + lost
            bl[b, :, h] = np.where(some, 1.5 * E + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(some, lse[b, :, h], 0.0)), 0.0)
    return out, lse, bo, bl


def assert_within(got, ref, bound, what):
    got = got.detach().double().cpu().numpy()
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - ref) <= bound)
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} values out of bounds, first at {at}: {got[at]} for {ref[at]}, bound "
                             f"{np.broadcast_to(bound, ok.shape)[at]}")
