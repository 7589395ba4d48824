"""Cases for measuring the paged cache's operators: the page pool, the pages' key bounds, the choice of pages for
each tree node, and tree attention over the chosen pages.

Shared notation: B sequences, m tree nodes, Hq query heads on Hkv KV heads (g = Hq / Hkv), d head dim, pages of ``bs``
tokens, a prefix of L tokens (its complete pages are the ones a choice is made from), ``refs`` the number of
block-table entries that name each page (0 = free).
"""
import math
import random

import numpy as np
import torch

own = False

GRID_LO, GRID_HI = -40, 40        # the exponents that a bound's or a query's grid may take
TOP = 255                         # magnitudes on a grid: whole numbers up to 255, which bf16 holds exactly


# --------------------------------------------------------------------------------------------------- cases
def listed():
    bf, f32 = "bf16", "f32"
    return [
        # the prompt has just been read: bounds of every page of a long-context batch
        dict(name="bounds_prompt", op="bounds", B=4, Hkv=8, d=128, bs=16, dtype=bf, lo=32768, hi=32768, new=0),
        # after a verify step: only the pages that the last committed tokens filled
        dict(name="bounds_step", op="bounds", B=8, Hkv=8, d=128, bs=16, dtype=bf, lo=1024, hi=8192, new=7),
        # one sequence, one token: the choice before a plain decode step
        dict(name="select_token", op="select", B=1, m=1, Hq=32, Hkv=8, d=128, bs=16, dtype=bf, lo=32768, hi=32768, n=64),
        # a long-context batch with 64-node trees
        dict(name="select_tree", op="select", B=4, m=64, Hq=32, Hkv=8, d=128, bs=16, dtype=bf, lo=32768, hi=32768, n=128),
        # plain decode over the chosen pages, a small batch
        dict(name="attend_token", op="attend", B=2, m=1, Hq=32, Hkv=8, d=128, bs=16, dtype=bf, lo=30000, hi=32768, n=64),
        # verifying 60-node trees of a batch of sixteen over 128 pages a node
        dict(name="attend_tree", op="attend", B=16, m=60, Hq=64, Hkv=8, d=128, bs=16, dtype=bf, lo=32768, hi=32768, n=128),
        # before a verify step: room for 64 nodes after ragged prefixes, what the last commit released given back first
        dict(name="reserve_tree", op="reserve", B=8, Hkv=8, d=128, bs=16, dtype=bf, lo=1024, hi=8192, n=64, ways=1,
             slack=2.0),
        # 64 prompts sampled four ways: the forks' half-filled last pages are copied
        dict(name="reserve_forks", op="reserve", B=256, Hkv=8, d=128, bs=64, dtype=bf, lo=600, hi=1500, n=60, ways=4,
             slack=1.5),
        # one prompt becomes eight samples
        dict(name="fork_samples", op="fork", B=1, out=8, bs=16, lo=2048, hi=2048, slack=2.0),
        # 512 beams change places: rows dropped, doubled and moved
        dict(name="fork_beams", op="fork", B=512, out=512, bs=16, lo=1024, hi=8192, slack=1.2),
        # a small pool, a few sequences gone
        dict(name="compact_small", op="compact", B=4, Hkv=8, d=128, bs=16, dtype=bf, lo=500, hi=1500, holes=0.2),
        # a large pool after a third of its pages have been freed here and there
        dict(name="compact_large", op="compact", B=64, Hkv=8, d=128, bs=16, dtype=bf, lo=1024, hi=8192, holes=0.33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "select", "attend", "attend", "reserve", "fork", "compact"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    Hq, Hkv = rng.choice([(32, 32), (32, 8), (64, 8), (8, 2), (28, 4), (4, 4)])
    d = rng.choice([128, 128, 128, 64])
    bs = rng.choice([16, 16, 32, 64, 128])
    hi = _log(rng, 40, 32768)
    lo = rng.choice([hi, max(0, hi // 2 - rng.randint(0, 9)), rng.randint(0, hi)])
    B = _log(rng, 1, 16)
    while B > 1 and B * hi * Hkv * d * (4 if dtype == "f32" else 2) > 4 * 32768 * 8 * 128 * 2:
        B -= 1
    if op == "bounds":
        while B * hi * Hkv * d * (4 if dtype == "f32" else 2) > 4 * 32768 * 8 * 128 * 2:
            hi = hi // 2 + 1
            lo = min(lo, hi)
        return dict(op=op, B=B, Hkv=Hkv, d=d, bs=bs, dtype=dtype, lo=lo, hi=hi, new=rng.choice([0, rng.randint(1, 200)]))
    if op in ("select", "attend"):
        m = rng.choice([1, rng.randint(2, 33), rng.randint(34, 128)])
        n = _log(rng, 4, 256)
        if dtype == "f32":
            # 32-bit caches are for small work
            hi, lo, m, n = min(hi, 4096), min(lo, 4096), min(m, 32), min(n, 64)
            Hq, Hkv = rng.choice([(8, 2), (4, 4), (14, 2)])
        elif op == "attend":
            d = 128
        if op == "select":
            # a choice is made where there are more pages than are wanted
            lo, hi = max(lo, 8 * bs), max(hi, 8 * bs)
            n = min(n, max(4, lo // bs * 3 // 4))
        while B > 1 and B * m * Hq * min(hi, n * bs) > 4 * 64 * 32 * 2048:
            B -= 1
        return dict(op=op, B=B, m=m, Hq=Hq, Hkv=Hkv, d=d, bs=bs, dtype=dtype, lo=lo, hi=hi, n=n)
    if op == "reserve":
        ways, heads = rng.choice([1, 2, 3, 4]), rng.choice([1, 4, 8])
        row = heads * d * (8 if dtype == "f32" else 4)
        rows = max(1, _log(rng, 1, 192) // ways)
        while rows > 1 and rows * (ways * (bs - 1) * row) > 256 * 32 * 8 * 128 * 4:
            rows -= 1
        return dict(op=op, B=ways * rows, Hkv=heads, d=d, bs=bs, dtype=dtype, lo=min(lo, 1500), hi=min(hi, 1500),
                    n=_log(rng, 1, 400), ways=ways, slack=rng.choice([0.6, 1.2, 3.0]))
    if op == "fork":
        B = _log(rng, 1, 400)
        return dict(op=op, B=B, out=rng.choice([B, _log(rng, 1, 512)]), bs=bs, lo=min(lo, 8192), hi=min(hi, 8192), slack=1.3)
    B, heads, holes = _log(rng, 1, 48), rng.choice([1, 4, 8]), rng.choice([0.0, 0.05, 0.3, 0.7])
    hi = min(hi, 4096)
    while B > 1 and B * hi * heads * d * (8 if dtype == "f32" else 4) * max(holes, 0.2) > 64 * 4608 * 8 * 128 * 4 * 0.3:
        B -= 1
    return dict(op=op, B=B, Hkv=heads, d=d, bs=bs, dtype=dtype, lo=min(lo, hi), hi=hi, holes=holes)


# -------------------------------------------------------------------------------------------------- inputs
def _lens(case, seed):
    """Lengths spread over the case's range, in another order for each seed (a pool's size goes by the case alone)."""
    B, ways = case["B"], case.get("ways", 1)
    r = random.Random(case["hi"] * 65537 + B)
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(B // ways)]
    random.Random(seed * 7919 + 13).shuffle(lens)
    return [n for n in lens for _ in range(ways)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _tables(pages, extra, seed, width=None):
    """Block tables whose rows hold ``pages[b]`` pages of a shuffled pool with ``extra`` more pages."""
    total = sum(pages) + extra
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    width = width or max(max(pages), 1)
    rows, at = [], 0
    for p in pages:
        rows.append(perm[at:at + p] + [-1] * (width - p))
        at += p
    return rows, total


def _parents(m, r):
    return [-1] + [r.randint(max(0, i // 2 - 3), i - 1) for i in range(1, m)]


def _mask_words(B, m, seed):
    r = random.Random(seed + 5)
    words = np.zeros((B, m, (m + 63) // 64), dtype=np.uint64)
    for b in range(B):
        par = _parents(m, r)
        for i in range(m):
            j = i
            while j >= 0:
                words[b, i, j >> 6] |= np.uint64(1 << (j & 63))
                j = par[j]
    return torch.from_numpy(words.view(np.int64)).cuda()


def _tree_queries(case, g, dt):
    """Nodes of one tree ask for much the same: a common part of each head and one of each node's own."""
    B, m, Hq, d = case["B"], case["m"], case["Hq"], case["d"]
    q = torch.randn(B, m, Hq, d, generator=g, device="cuda") * 0.6
    return (q + torch.randn(B, 1, Hq, d, generator=g, device="cuda") * 0.8).to(dt)


def _words_of(sel, m):
    """bool [..., m] -> int64 words [..., ceil(m / 64)]."""
    W = (m + 63) // 64
    pad = torch.zeros(*sel.shape[:-1], W * 64 - m, dtype=torch.bool, device=sel.device)
    bits = torch.cat([sel, pad], -1).unflatten(-1, (W, 64)).long()
    return (bits << torch.arange(64, device=sel.device)).sum(-1)


def prepare(case, seed):
    g = _gen(seed)
    lens = _lens(case, seed)
    op, bs, B = case["op"], case["bs"], case["B"]
    st = dict(case=case, lens=lens, prefix_len=_ints(lens))
    full = [n // bs for n in lens]
    if op == "bounds":
        rows, nb = _tables([-(-n // bs) for n in lens], 3, seed, max(1, -(-case["hi"] // bs)))
        dt = _dtype(case)
        k = torch.randn(nb, case["Hkv"], bs, case["d"], generator=g, device="cuda", dtype=dt)
        k.mul_(torch.rand(nb, case["Hkv"], 1, case["d"], generator=g, device="cuda", dtype=dt) * 3)  # channels differ in size
        start = [max(0, n - case["new"]) if case["new"] else 0 for n in lens]
        st.update(k_cache=k, block_table=_ints(rows), start=start, start_len=_ints(start),
                  bounds=torch.randn(nb, case["Hkv"], 2, case["d"], generator=g, device="cuda", dtype=torch.bfloat16))
    elif op in ("select", "attend"):
        m, Hkv, d = case["m"], case["Hkv"], case["d"]
        dt = _dtype(case)
        width = -(-(case["hi"] + m) // bs)
        rows, nb = _tables([-(-(n + m) // bs) for n in lens], 3, seed, width)
        cap = max(1, case["hi"] // bs)
        st.update(q=_tree_queries(case, g, dt), block_table=_ints(rows), full=full, cap=cap, max_prefix=case["hi"],
                  n=max(case["n"], 4), first=1, recent=2)
        if op == "select":
            mid = torch.randn(nb, Hkv, d, generator=g, device="cuda") * 30
            half = torch.rand(nb, Hkv, d, generator=g, device="cuda") * 100 + 20
            grid = torch.exp2(torch.randint(-8, -6, (nb, Hkv, 1, 1), generator=g, device="cuda").float())
            st["bounds"] = ((torch.stack([mid + half, mid - half], 2).round().clamp(-TOP, TOP)) * grid).to(torch.bfloat16)
        else:
            shape = (nb, Hkv, bs, d)
            k = torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(0.8)
            k.add_(torch.randn(nb, Hkv, 1, d, generator=g, device="cuda", dtype=dt).mul_(0.6))
            v = torch.randn(shape, generator=g, device="cuda", dtype=dt)
            # each node keeps n pages out of a pool of 2n that its tree shares, the first and the latest always
            nf = torch.tensor(full, device="cuda").view(B, 1, 1, 1)
            at = torch.arange(cap, device="cuda")
            liking = torch.rand(B, Hkv, 1, cap, generator=g, device="cuda").masked_fill(at >= nf, -1)
            liking = liking + ((at < 1) | (at >= nf - 2)) * 9.0
            pool = liking.argsort(-1, descending=True).argsort(-1) < 2 * st["n"]
            each = torch.rand(B, Hkv, m, cap, generator=g, device="cuda") + pool * 1.0 + ((at < 1) | (at >= nf - 2)) * 9.0
            each = each.masked_fill(at >= nf, -1)
            top = each.topk(min(st["n"], cap), -1).indices
            sel = torch.zeros(B, Hkv, m, cap, dtype=torch.bool, device="cuda").scatter_(-1, top, True) & (at < nf)
            st["selection"] = _pack_selection(sel, m)
            st.update(k_cache=k, v_cache=v, mask=_mask_words(B, m, seed))
    elif op == "reserve":
        # prompts of which every `ways` rows share all pages, the half-filled last one among them
        ways = case["ways"]
        n, r = case["n"], random.Random(seed)
        need = -(-n // bs) + 2
        extra = int(B * need * case["slack"]) + 2
        have = [-(-lens[b] // bs) for b in range(0, B, ways)]
        width = -(-(case["hi"] + n) // bs)
        rows, nb = _tables(have, extra, seed, width)
        rows = [list(rows[b // ways]) for b in range(B)]
        refs = [0] * nb
        for row in rows:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        idle = [p for p in range(nb) if refs[p] == 0]
        # what the last commit let go of: pages still counted, in no table any more
        freed = [r.choice([idle[i], -1]) if i < len(idle) // 4 else -1 for i in range(B * 4)]
        for p in freed:
            if p >= 0:
                refs[p] += 1
        shape = (nb, case["Hkv"], bs, case["d"])
        st.update(block_table=_ints(rows), refs=_ints(refs), freed=_ints(freed), n=n,
                  k_cache=torch.randn(shape, generator=g, device="cuda", dtype=_dtype(case)),
                  v_cache=torch.randn(shape, generator=g, device="cuda", dtype=_dtype(case)))
    elif op == "fork":
        pages = [-(-(n + 8) // bs) for n in lens]
        rows, nb = _tables(pages, int(sum(pages) * (case["slack"] - 1)) + 16, seed, -(-(case["hi"] + 8) // bs))
        r = random.Random(seed)
        refs = [r.choice([0, 0, 0, 1, 2]) for _ in range(nb)]      # some pages are also held by others
        for row in rows:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        src = [r.randrange(B) if B > 1 else 0 for _ in range(case["out"])]
        if case["out"] > 8:
            src = [-1 if r.random() < 0.05 else s for s in src]
        st.update(block_table=_ints(rows), refs=_ints(refs), src=_ints(src))
    else:
        pages = [-(-n // bs) for n in lens]
        live = sum(pages)
        extra = int(live * case["holes"] / (1 - case["holes"])) + 1
        rows, nb = _tables(pages, extra, seed, max(1, -(-case["hi"] // bs)))
        refs = [0] * nb
        for row in rows:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        shape = (nb, case["Hkv"], bs, case["d"])
        st.update(block_table=_ints(rows), refs=_ints(refs),
                  k_cache=torch.randn(shape, generator=g, device="cuda", dtype=_dtype(case)),
                  v_cache=torch.randn(shape, generator=g, device="cuda", dtype=_dtype(case)),
                  bounds=torch.randn(nb, case["Hkv"], 2, case["d"], generator=g, device="cuda", dtype=torch.bfloat16))
    return st


def _pack_selection(sel, m):
    """bool [B, Hkv, m, C] -> pages [B, Hkv, C] ascending with -1 behind, count [B, Hkv], node_mask [B, Hkv, C, W]."""
    C = sel.shape[-1]
    any_node = sel.any(2)
    at = torch.arange(C, device=sel.device).expand_as(any_node)
    order = torch.where(any_node, at, C).sort(-1).values
    there = order < C
    bits = sel.transpose(2, 3).gather(2, order.clamp(max=C - 1).unsqueeze(-1).expand(-1, -1, -1, m)) & there.unsqueeze(-1)
    return dict(pages=torch.where(there, order, -1).int(), count=any_node.sum(-1).int(), node_mask=_words_of(bits, m))


# --------------------------------------------------------------------------------------------- plain forms
def _grid(amax):
    """The smallest 2^e with amax <= 255 * 2^e, e between the two limits."""
    f, e = torch.frexp(amax)                                   # amax = f * 2^e, f in [1/2, 1)
    e = (e - 8 + (f > TOP / 256.0).int()).clamp(GRID_LO, GRID_HI)
    return torch.exp2(torch.where(amax > 0, e, GRID_LO).float())


def _plain_bounds(st):
    c, k, bounds = st["case"], st["k_cache"], st["bounds"]
    lim = TOP * 2.0 ** GRID_HI
    for b, (s, n) in enumerate(zip(st["start"], st["lens"])):
        ids = st["block_table"][b, s // c["bs"]: n // c["bs"]].long()
        if ids.numel() == 0:
            continue
        rows = k[ids].float()
        nan = rows.isnan()
        hi = rows.masked_fill(nan, -math.inf).amax(2)
        lo = rows.masked_fill(nan, math.inf).amin(2)
        none = nan.all(2)
        hi = hi.masked_fill(none, 0).clamp(-lim, lim)
        lo = lo.masked_fill(none, 0).clamp(-lim, lim)
        grid = _grid(torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True))
        bounds[ids] = torch.stack([torch.ceil(hi / grid) * grid, torch.floor(lo / grid) * grid], 2).to(torch.bfloat16)
    return bounds


def _plain_select(st):
    c = st["case"]
    B, m, Hkv, d, cap = c["B"], c["m"], c["Hkv"], c["d"], st["cap"]
    g = c["Hq"] // Hkv
    lim = TOP * 2.0 ** GRID_HI
    sel = torch.zeros(B, Hkv, m, cap, dtype=torch.bool, device="cuda")
    for b in range(B):
        nf = st["full"][b]
        if nf == 0:
            continue
        q = st["q"][b].float().nan_to_num(0.0, lim, -lim).clamp(-lim, lim).view(m, Hkv, g, d).permute(1, 0, 2, 3)
        grid = _grid(q.abs().amax(-1, keepdim=True))
        q = (q / grid).round() * grid
        bnd = st["bounds"][st["block_table"][b, :nf].long()].float().permute(1, 2, 3, 0)        # [Hkv, 2, d, nf]
        score = q.clamp(min=0).reshape(Hkv, m * g, d) @ bnd[:, 0] + q.clamp(max=0).reshape(Hkv, m * g, d) @ bnd[:, 1]
        score = score.view(Hkv, m, g, nf).amax(2)
        at = torch.arange(nf, device="cuda")
        score = score.masked_fill((at < st["first"]) | (at >= nf - st["recent"]), math.inf)
        top = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :st["n"]]
        sel[b, :, :, :nf].scatter_(-1, top, True)
    return _pack_selection(sel, m)


def _plain_attend(st):
    c, s = st["case"], st["selection"]
    B, m, Hq, Hkv, d, bs = c["B"], c["m"], c["Hq"], c["Hkv"], c["d"], c["bs"]
    g = Hq // Hkv
    out, lse = torch.empty_like(st["q"]), torch.empty(B, m, Hq, device="cuda")
    heads = torch.arange(Hkv, device="cuda").view(Hkv, 1)
    node = torch.arange(m, device="cuda")
    for b in range(B):
        n, nf = st["lens"][b], st["full"][b]
        logical = s["pages"][b].long()                                                     # [Hkv, C]
        there = logical >= 0
        phys = st["block_table"][b][logical.clamp(min=0)].long().clamp(min=0)
        tail = torch.arange(nf * bs, n + m, device="cuda")
        tphys = st["block_table"][b][tail // bs].long()
        tk = st["k_cache"][tphys, :, tail % bs].float().transpose(0, 1)                    # [Hkv, tail, d]
        tv = st["v_cache"][tphys, :, tail % bs].float().transpose(0, 1)
        kk = torch.cat([st["k_cache"][phys, heads].float().flatten(1, 2), tk], 1)
        vv = torch.cat([st["v_cache"][phys, heads].float().flatten(1, 2), tv], 1)
        bits = (s["node_mask"][b][:, :, node // 64] >> (node % 64)) & 1                     # [Hkv, C, m]
        seen = ((bits == 1) & there.unsqueeze(-1)).repeat_interleave(bs, 1).transpose(1, 2)  # [Hkv, m, C * bs]
        t = tail - n
        word = st["mask"][b][:, t.clamp(min=0) // 64]
        tseen = (t < 0) | (((word >> (t.clamp(min=0) % 64)) & 1) == 1)                      # [m, tail]
        seen = torch.cat([seen, tseen.expand(Hkv, m, -1)], 2).unsqueeze(2)                  # [Hkv, m, 1, keys]
        q = st["q"][b].float().view(m, Hkv, g, d).transpose(0, 1).reshape(Hkv, m * g, d)
        x = (q @ kk.transpose(1, 2)).view(Hkv, m, g, -1) / math.sqrt(d)
        x = x.masked_fill(~seen, -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top)
        z = e.sum(-1, keepdim=True)
        o = (e.view(Hkv, m * g, -1) @ vv).view(Hkv, m, g, d) / z
        out[b] = o.transpose(0, 1).reshape(m, Hq, d).to(out.dtype)
        lse[b] = (top + torch.log(z)).squeeze(-1).transpose(0, 1).reshape(m, Hq)
    return out, lse


def _plain_reserve(st):
    c, table, n, bs = st["case"], st["block_table"].long(), st["n"], st["case"]["bs"]
    B, width = table.shape
    L = st["prefix_len"].long()
    freed = st["freed"].long()
    refs = st["refs"].long().index_add(0, freed.clamp(min=0), -(freed >= 0).long())
    first = L // bs
    pages = -(-(L + n) // bs) - first
    j = torch.arange((n + bs - 2) // bs + 1, device="cuda")
    lp = first[:, None] + j
    active = j < pages[:, None]
    entry = table.gather(1, lp.clamp(max=width - 1))
    has = active & (entry >= 0)
    # the half-filled last page, where others hold it too: every holder but the last takes a copy
    tail = torch.where(has[:, 0] & (L % bs > 0), entry[:, 0], -1)
    before = ((tail[:, None] == tail[None, :]) & (tail >= 0)).tril(-1).sum(1)
    copy = (tail >= 0) & (refs[tail.clamp(min=0)] - before > 1)
    need = active & ~has
    need[:, 0] |= copy
    rank = need.flatten().cumsum(0).view_as(need) - 1
    free = (refs == 0).nonzero().flatten()
    short = (need & (rank >= free.numel())).any(1)
    take = need & ~short[:, None]
    fresh = free[rank[take]]
    rows, cols = take.nonzero(as_tuple=True)
    out_table = table.clone()
    out_table[rows, lp[rows, cols]] = fresh
    copy = copy & ~short
    refs = refs.index_add(0, tail.clamp(min=0), -copy.long())
    refs[fresh] = 1
    src, dst, keep = tail[copy], out_table.gather(1, lp[:, :1].clamp(max=width - 1))[copy][:, 0], (L % bs)[copy]
    below = (torch.arange(bs, device="cuda") < keep[:, None])[:, None, :, None]
    for cache in (st["k_cache"], st["v_cache"]):
        cache[dst] = torch.where(below, cache[src], cache[dst])
    granted = torch.where(short, -1, take.sum(1))
    return out_table.int(), refs.int(), granted.int(), st["k_cache"], st["v_cache"]


def _plain_fork(st):
    bs, table, src = st["case"]["bs"], st["block_table"].long(), st["src"].long()
    L = torch.where(src >= 0, st["prefix_len"].long()[src.clamp(min=0)], 0)
    kept = torch.arange(table.shape[1], device="cuda") < (-(-L // bs))[:, None]
    new = torch.where(kept, table[src.clamp(min=0)], -1)
    refs = st["refs"].long()
    for t, sign in ((table, -1), (new, 1)):
        refs = refs.index_add(0, t.clamp(min=0).flatten(), sign * (t >= 0).long().flatten())
    return new.int(), L.int(), refs.int()


def _plain_compact(st):
    refs, table = st["refs"].long(), st["block_table"].long()
    live = refs > 0
    total = live.sum()
    at = torch.arange(refs.numel(), device="cuda")
    src = (live & (at >= total)).nonzero().flatten()
    dst = (~live & (at < total)).nonzero().flatten()
    remap = torch.where(live, at, -1)
    remap[src] = dst
    for buf in (st["k_cache"], st["v_cache"], st["bounds"]):
        buf[dst] = buf[src]
    new = refs.clone()
    new[dst] = refs[src]
    new[src] = 0
    table = torch.where(table >= 0, remap[table.clamp(min=0)], -1)
    return (table.int(), new.int(), remap.int(), total.view(1).int(), st["k_cache"], st["v_cache"], st["bounds"])


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "select":
            s = _plain_select(st)
            return s["pages"], s["count"], s["node_mask"]
        return dict(bounds=_plain_bounds, attend=_plain_attend, reserve=_plain_reserve, fork=_plain_fork,
                    compact=_plain_compact)[op](st)
    import speculative_decoding_tree_eagle_gb300 as ts
    if op == "bounds":
        return ts.kv_page_bounds(st["k_cache"], st["block_table"], st["prefix_len"], start_len=st["start_len"],
                                 bounds=st["bounds"])
    if op == "select":
        s = ts.page_select(st["q"], st["bounds"], st["block_table"], st["prefix_len"], st["n"], block_size=c["bs"],
                           max_prefix=st["max_prefix"], first=st["first"], recent=st["recent"])
        return s["pages"], s["count"], s["node_mask"]
    if op == "attend":
        return ts.tree_attention_sparse(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["prefix_len"],
                                        st["mask"], st["selection"])
    if op == "reserve":
        r = ts.kv_reserve(st["k_cache"], st["v_cache"], st["block_table"], st["prefix_len"], st["refs"], st["n"],
                          freed=st["freed"])
        return r["block_table"], r["refs"], r["granted"], st["k_cache"], st["v_cache"]
    if op == "fork":
        r = ts.kv_fork(st["block_table"], st["prefix_len"], st["refs"], st["src"], c["bs"])
        return r["block_table"], r["prefix_len"], r["refs"]
    r = ts.kv_compact(st["k_cache"], st["v_cache"], st["block_table"], st["refs"], bounds=st["bounds"])
    return (r["block_table"], r["refs"], r["remap"], r["live"], st["k_cache"], st["v_cache"], st["bounds"])


# --------------------------------------------------------------------------------------------------- costs
def work(case):
    op, bs, B = case["op"], case["bs"], case["B"]
    mean = (case["lo"] + case["hi"]) / 2
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "bounds":
        toks = mean // bs * bs if not case["new"] else min(case["new"], mean)
        elems = B * toks * case["Hkv"] * case["d"]
        return dict(bytes=elems * size + elems / bs * 4 + B * toks / bs * 4, flops=2 * elems)
    if op in ("select", "attend"):
        m, Hq, Hkv, d = case["m"], case["Hq"], case["Hkv"], case["d"]
        n, full, W = max(case["n"], 4), mean // bs, -(-case["m"] // 64)
        union = min(full, n if m == 1 else 2 * n)
        q = B * m * Hq * d * size
        if op == "select":
            cap = max(1, case["hi"] // bs)
            return dict(bytes=q + B * full * Hkv * 4 * d + B * Hkv * (cap * (4 + 8 * W) + 4) + B * full * 4,
                        flops=2.0 * B * m * Hq * 2 * d * full)
        keys = min(full, n) * bs + bs / 2 + m / 2
        kv = B * Hkv * (union * bs + bs / 2 + m) * d * size * 2
        return dict(bytes=2 * q + 4 * B * m * Hq + kv + B * Hkv * union * (4 + 8 * W), flops=4.0 * B * m * Hq * d * keys)
    width = -(-(case["hi"] + case.get("n", 8)) // bs)
    tables = B * width * 4
    if op == "fork":
        pool = B * mean / bs * case["slack"]
        return dict(bytes=tables + case["out"] * width * 4 + 8 * pool, flops=0)
    row = case["Hkv"] * case["d"] * size * 2
    if op == "reserve":
        pool = B / case["ways"] * mean / bs + B * (case["n"] / bs + 2) * case["slack"]
        copies = B * (case["ways"] - 1) / case["ways"] * (bs - 1) / 2
        return dict(bytes=2 * tables + 8 * pool + 2 * copies * row, flops=0)
    live = B * mean / bs
    moved = live * case["holes"]
    return dict(bytes=2 * tables + 12 * live / (1 - case["holes"]) + 2 * moved * (bs * row + case["Hkv"] * 4 * case["d"]), flops=0)


# --------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, bs, B = case["op"], case["bs"], case["B"]
    table = st["block_table"].cpu().numpy().astype(np.int64)
    if op == "bounds":
        out = st["bounds"].double()
        for b in range(B):
            for first in range(st["start"][b] // bs, st["lens"][b] // bs, 512):
                ids = torch.from_numpy(table[b, first:min(first + 512, st["lens"][b] // bs)]).cuda()
                k = st["k_cache"][ids].double()
                hi, lo = k.max(2).values, k.min(2).values
                big = torch.maximum(hi, -lo).amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(big / TOP))
                e = torch.where(TOP * 2.0 ** (e - 1) >= big, e - 1, torch.where(TOP * 2.0 ** e < big, e + 1, e))
                e = torch.where(big > 0, e, GRID_LO).clamp(GRID_LO, GRID_HI)
                out[ids] = torch.stack([torch.ceil(hi * 2.0 ** -e), torch.floor(lo * 2.0 ** -e)], 2) * (2.0 ** e)[:, :, None]
        return out
    if op == "select":
        return _exact_select(case, st, table)
    if op == "attend":
        return _exact_attend(case, st, table)
    refs = st["refs"].cpu().numpy().astype(np.int64)
    if op == "fork":
        src, lens = st["src"].tolist(), st["lens"]
        new = np.full((len(src), table.shape[1]), -1, dtype=np.int64)
        out_len = [0] * len(src)
        for r, s in enumerate(src):
            if s >= 0:
                out_len[r] = lens[s]
                p = -(-lens[s] // bs)
                new[r, :p] = table[s, :p]
        np.subtract.at(refs, table[table >= 0], 1)
        np.add.at(refs, new[new >= 0], 1)
        return _ints(new), _ints(out_len), _ints(refs)
    if op == "reserve":
        return _exact_reserve(case, st, table, refs)
    ids = np.nonzero(refs > 0)[0]
    live = len(ids)
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in ids if p >= live]
    remap = np.full(len(refs), -1, dtype=np.int64)
    remap[ids] = ids
    new = refs.copy()
    for s, t in zip(movers, holes):
        remap[s] = t
        new[t], new[s] = refs[s], 0
        for buf in (st["k_cache"], st["v_cache"], st["bounds"]):
            buf[t] = buf[int(s)]
    moved = np.where(table >= 0, remap[np.maximum(table, 0)], -1)
    return _ints(moved), _ints(new), _ints(remap), _ints([live]), st["k_cache"], st["v_cache"], st["bounds"]


def _exact_reserve(case, st, table, refs):
    bs, n = case["bs"], st["n"]
    for p in st["freed"].tolist():
        if p >= 0:
            refs[p] -= 1
    free = [p for p in range(len(refs)) if refs[p] == 0]
    at, granted = 0, []
    for b, L in enumerate(st["lens"]):
        first, last = L // bs, -(-(L + n) // bs)
        want = []
        for i in range(first, last):
            p = table[b, i]
            if p < 0 or (i == first and L % bs and refs[p] > 1):
                want.append(i)
        if at + len(want) > len(free):
            granted.append(-1)
            at = len(free) if want else at
            continue
        for i in want:
            t, p = free[at], table[b, i]
            at += 1
            if p >= 0:
                for cache in (st["k_cache"], st["v_cache"]):
                    cache[t, :, : L % bs] = cache[int(p), :, : L % bs]
                refs[p] -= 1
            table[b, i], refs[t] = t, 1
        granted.append(len(want))
    return _ints(table), _ints(refs), _ints(granted), st["k_cache"], st["v_cache"]


def _exact_select(case, st, table):
    B, m, Hkv, d = case["B"], case["m"], case["Hkv"], case["d"]
    g, cap, W = case["Hq"] // Hkv, st["cap"], (case["m"] + 63) // 64
    pages = np.full((B, Hkv, cap), -1, dtype=np.int64)
    count = np.zeros((B, Hkv), dtype=np.int64)
    words = np.zeros((B, Hkv, cap, W), dtype=np.uint64)
    for b in range(B):
        nf = st["full"][b]
        ids = torch.from_numpy(table[b, :nf]).cuda()
        for h in range(Hkv):
            if nf == 0:
                continue
            q = st["q"][b, :, h * g:(h + 1) * g].double()                       # [m, g, d]
            big = q.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -200)
            e = torch.ceil(torch.log2(big / TOP))
            e = torch.where(TOP * 2.0 ** (e - 1) >= big, e - 1, torch.where(TOP * 2.0 ** e < big, e + 1, e))
            e = e.clamp(GRID_LO, GRID_HI)
            q = torch.round(q * 2.0 ** -e) * 2.0 ** e
            bnd = st["bounds"][ids, h].double()                                 # [nf, 2, d]
            q2 = torch.cat([q.clamp(min=0), q.clamp(max=0)], -1)
            s = (q2.view(m * g, 2 * d) @ bnd.reshape(nf, 2 * d).T).view(m, g, nf).amax(1).cpu().numpy()
            for i in range(m):
                keep = set(range(min(st["first"], nf))) | set(range(max(0, nf - st["recent"]), nf))
                for p in np.lexsort((np.arange(nf), -s[i])):
                    if len(keep) >= st["n"]:
                        break
                    keep.add(int(p))
                for p in keep:
                    words[b, h, p, i >> 6] |= np.uint64(1 << (i & 63))
            kept = np.nonzero(words[b, h].any(-1))[0]
            count[b, h] = len(kept)
            pages[b, h, :len(kept)] = kept
            row = words[b, h, kept].copy()
            words[b, h] = 0
            words[b, h, :len(kept)] = row
    return _ints(pages), _ints(count), torch.from_numpy(words.view(np.int64)).cuda()


def _exact_attend(case, st, table):
    B, m, Hq, Hkv, d, bs = (case[k] for k in ("B", "m", "Hq", "Hkv", "d", "bs"))
    g = Hq // Hkv
    out = torch.empty(B, m, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, m, Hq, dtype=torch.float64, device="cuda")
    pages = st["selection"]["pages"].cpu().numpy()
    words = st["selection"]["node_mask"].cpu().numpy().view(np.uint64)
    tree = st["mask"].cpu().numpy().view(np.uint64)
    node = np.arange(m)
    for b in range(B):
        L = st["lens"][b]
        tail = np.arange(L // bs * bs, L + m)
        own_bits = (tree[b][:, node >> 6] >> (node & 63).astype(np.uint64)) & np.uint64(1)      # [m, m]
        tseen = np.concatenate([np.ones((m, L % bs), dtype=bool), own_bits.astype(bool)], 1)
        for h in range(Hkv):
            u = pages[b, h][pages[b, h] >= 0]
            pos = np.concatenate([(u[:, None] * bs + np.arange(bs)).reshape(-1), tail]).astype(np.int64)
            chosen = ((words[b, h, :len(u)][:, node >> 6] >> (node & 63).astype(np.uint64)) & np.uint64(1)).astype(bool).T
            seen = torch.from_numpy(np.concatenate([np.repeat(chosen, bs, 1), tseen], 1)).cuda()
            where = torch.from_numpy(table[b][pos // bs]).cuda()
            slot = torch.from_numpy(pos % bs).cuda()
            k = st["k_cache"][where, h, slot].double()
            v = st["v_cache"][where, h, slot].double()
            for j in range(g):
                x = st["q"][b, :, h * g + j].double() @ k.T / math.sqrt(d)
                x = x.masked_fill(~seen, -math.inf)
                l = torch.logsumexp(x, -1)
                out[b, :, h * g + j] = torch.exp(x - l[:, None]) @ v
                lse[b, :, h * g + j] = l
    return out, lse
