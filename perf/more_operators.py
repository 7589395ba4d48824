"""Cases for measuring the paged cache in 8 bits: quantising K and V rows as they are written, reading them back, tree
attention over the codes, and committing the accepted path.

Shared notation: B sequences, Hkv KV heads (Hq query heads on them, g = Hq / Hkv), d head dim, pages of ``bs`` tokens of which
every ``sb`` have one scale per head, m tree nodes, a prefix of L tokens.  A cache holds e4m3 codes [pages, Hkv, bs, d] beside
fp32 scales [pages, Hkv, bs / sb]; a value is code * scale.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
EXP_LO, EXP_HI = -40, 40          # scales are powers of two in this range


# --------------------------------------------------------------------------------------------------- cases
def listed():
    bf, f32 = "bf16", "f32"
    return [
        # a long-context batch's prompts go into the cache
        dict(name="write_prompt", op="write", B=4, n=32768, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=0, hi=0),
        # the rows of 60-node trees behind ragged prefixes, as slices of a fused projection's output
        dict(name="write_tree", op="write", B=16, n=60, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=1024, hi=8192),
        # plain decode: one token of each of 64 sequences
        dict(name="write_token", op="write", B=64, n=1, Hkv=8, d=128, bs=64, sb=64, dtype=bf, lo=100, hi=8192),
        # plain decode over ragged contexts
        dict(name="attend_token", op="attend", B=8, m=1, Hq=32, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=1024, hi=8192),
        # long contexts, a chain of eight drafted tokens: bound by the cache's bytes
        dict(name="attend_chain", op="attend", B=4, m=8, Hq=32, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=32768, hi=32768),
        # 60-node trees on 64 heads, a batch of sixteen
        dict(name="attend_tree", op="attend", B=16, m=60, Hq=64, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=4096, hi=4096),
        # long contexts, 64-node trees
        dict(name="attend_long", op="attend", B=4, m=64, Hq=32, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=32768, hi=32768),
        # a small model in 32 bits
        dict(name="attend_f32", op="attend", B=2, m=8, Hq=8, Hkv=2, d=64, bs=16, sb=8, dtype=f32, lo=150, hi=700),
        # a context taken back out of the cache, for an engine that wants it in bf16
        dict(name="read_prompt", op="read", B=2, n=8192, Hkv=8, d=128, bs=16, sb=16, dtype=bf, lo=8000, hi=8192, new=0),
        # the last rows of each sequence, in 32 bits
        dict(name="read_tail", op="read", B=16, n=64, Hkv=8, d=128, bs=16, sb=16, dtype=f32, lo=1024, hi=8192, new=64),
        # after verifying 60-node trees: a handful of rows kept in each sequence
        dict(name="commit_tree", op="commit", B=16, m=60, Hkv=8, d=128, bs=16, sb=16, lo=1024, hi=8192, most=7),
        # larger trees, deeper acceptances, larger pages
        dict(name="commit_deep", op="commit", B=64, m=128, Hkv=8, d=128, bs=64, sb=64, lo=1024, hi=4096, most=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "write", "attend", "attend", "attend", "read", "commit"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    Hq, Hkv = rng.choice([(32, 32), (32, 8), (64, 8), (8, 2), (28, 4), (4, 4)])
    d = rng.choice([128, 128, 128, 64])
    bs = rng.choice([16, 16, 32, 64, 128])
    sb = rng.choice([bs, bs, 16, 4, 1])
    hi = _log(rng, 20, 32768)
    lo = rng.choice([hi, max(0, hi // 2 - rng.randint(0, 9)), rng.randint(0, hi)])
    B = _log(rng, 1, 32)
    shape = dict(Hkv=Hkv, d=d, bs=bs, sb=sb)
    if op == "attend":
        m = rng.choice([1, rng.randint(2, 33), rng.randint(34, 128)])
        if dtype == "f32":
            # 32-bit queries are for small work
            hi, lo, m = min(hi, 4096), min(lo, 4096), min(m, 32)
            Hq, shape["Hkv"] = rng.choice([(8, 2), (4, 4), (14, 2)])
        else:
            shape["d"] = d = 128
        while B > 1 and (B * m * Hq * hi > 4 * 64 * 32 * 32768 or B * hi * shape["Hkv"] > 4 * 32768 * 8):
            B -= 1
        return dict(op=op, B=B, m=m, Hq=Hq, dtype=dtype, lo=lo, hi=hi, **shape)
    room = 4 * 32768 * 8 * 128 * 2 // (Hkv * d * (4 if dtype == "f32" else 2))      # rows that the largest case has
    if op == "commit":
        m = rng.randint(2, 128)
        while B > 1 and B * (hi + m) > room:
            B -= 1
        return dict(op=op, B=B, m=m, lo=lo, hi=hi, most=rng.randint(1, min(m, 17)), **shape)
    n = rng.choice([1, rng.randint(2, 128), _log(rng, 128, 32768)])
    while B > 1 and B * (hi + n) > room:
        B -= 1
    if op == "read":
        return dict(op=op, B=B, n=n, dtype=dtype, lo=lo, hi=hi, new=rng.choice([0, n]), **shape)
    return dict(op=op, B=B, n=n, dtype=dtype, lo=lo, hi=hi, **shape)


# -------------------------------------------------------------------------------------------------- inputs
def _lens(case, seed):
    """Lengths spread over the case's range, in another order for each seed (a pool's size goes by the case alone)."""
    r = random.Random(case["hi"] * 65537 + case["B"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    random.Random(seed * 7919 + 13).shuffle(lens)
    return lens


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _tables(lens, more, bs, hi, seed):
    """Block tables with pages for every sequence's length and ``more`` tokens, out of a shuffled pool."""
    pages = [-(-(n + more) // bs) for n in lens]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(1, -(-(hi + more) // bs))
    rows, at = [], 0
    for p in pages:
        rows.append(perm[at:at + p] + [-1] * (width - p))
        at += p
    return _ints(rows), total


def _mask_words(B, m, seed):
    r = random.Random(seed + 5)
    words = np.zeros((B, m, (m + 63) // 64), dtype=np.uint64)
    for b in range(B):
        par = [-1] + [r.randint(max(0, i // 2 - 3), i - 1) for i in range(1, m)]
        for i in range(m):
            j = i
            while j >= 0:
                words[b, i, j >> 6] |= np.uint64(1 << (j & 63))
                j = par[j]
    return torch.from_numpy(words.view(np.int64)).cuda()


def _paths(B, m, most, seed):
    """Accepted paths: the root, then increasing nodes, -1 behind."""
    r = random.Random(seed + 9)
    rows, lens = [], []
    for _ in range(B):
        a = r.randint(1, most)
        rows.append([0] + sorted(r.sample(range(1, m), a - 1)) + [-1] * (m - a))
        lens.append(a)
    return _ints(rows), _ints(lens)


def _rows(shape, g, dt, big):
    """K or V rows: channels differ in size, a few by a lot (``big``), as those of keys do."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    size = torch.rand(shape[-2:], generator=g, device="cuda") * 1.5 + 0.5
    if big:
        size = torch.where(torch.rand(shape[-2:], generator=g, device="cuda") < 0.03, size * 8, size)
    return x.mul_(size.to(dt))


def _cache(nb, case, g, big):
    """A filled cache: codes and scales of normal rows, one page of zeros."""
    Hkv, bs, d, sb = case["Hkv"], case["bs"], case["d"], case["sb"]
    x = _rows((nb, bs, Hkv, d), g, torch.bfloat16, big).transpose(1, 2).reshape(nb, Hkv, bs // sb, sb, d)
    x[0] = 0
    codes = torch.empty((nb, Hkv, bs // sb, sb, d), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((nb, Hkv, bs // sb), device="cuda")
    for at in range(0, nb, 4096):
        part = x[at:at + 4096].float()
        s = _scale(part.abs().amax((-1, -2)))
        scale[at:at + 4096] = s
        codes[at:at + 4096] = (part / s[..., None, None]).to(torch.float8_e4m3fn)
    return codes.view(nb, Hkv, bs, d), scale


def prepare(case, seed):
    g = _gen(seed)
    op, B, bs, Hkv, d = case["op"], case["B"], case["bs"], case["Hkv"], case["d"]
    lens = _lens(case, seed)
    more = dict(write=case.get("n"), attend=case.get("m"), commit=case.get("m"), read=0)[op]
    table, nb = _tables(lens, more, bs, case["hi"], seed)
    st = dict(case=case, block_table=table)
    st["k_cache"], st["k_scale"] = _cache(nb, case, g, True)
    st["v_cache"], st["v_scale"] = _cache(nb, case, g, False)
    if op == "write":
        n, dt = case["n"], _dtype(case)
        st["start_len"] = _ints(lens)
        if n > 1 and B > 1:
            # prompts and trees of a batch are not all of one length
            r = random.Random(seed + 3)
            st["length"] = _ints([n] + [r.randint(n - n // 8, n) for _ in range(B - 1)])
        else:
            st["length"] = _ints([n] * B)
        # the projection gives q, k and v side by side; k and v are views of it (a prompt's come by themselves)
        width = 3 * Hkv if n <= 4096 else 2 * Hkv
        rows = _rows((B, n, width, d), g, dt, True)
        st["k"], st["v"] = rows[:, :, width - 2 * Hkv:width - Hkv], rows[:, :, width - Hkv:]
    elif op == "attend":
        m, Hq, dt = case["m"], case["Hq"], _dtype(case)
        # nodes of one tree ask for much the same: a common part of each head and one of each node's own
        q = torch.randn(B, m, Hq, d, generator=g, device="cuda") * 0.6
        st["q"] = (q + torch.randn(B, 1, Hq, d, generator=g, device="cuda") * 0.8).to(dt)
        st.update(prefix_len=_ints(lens), max_prefix=case["hi"], mask=_mask_words(B, m, seed))
    elif op == "read":
        st["prefix_len"] = _ints(lens)
        st["start_len"] = _ints([max(0, L - case["new"]) if case["new"] else 0 for L in lens])
    else:
        st["prefix_len"] = _ints(lens)
        st["accept_path"], st["accept_len"] = _paths(B, case["m"], case["most"], seed)
    return st


# --------------------------------------------------------------------------------------------- plain forms
def _scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e, e between the two limits."""
    f, e = torch.frexp(amax)                                   # amax = f * 2^e, f in [1/2, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (f > 0.875).int()).clamp(EXP_LO, EXP_HI)
    return torch.exp2(torch.where(amax > 0, e, EXP_LO).float())


def _bytes_of(cache):
    return cache.view(torch.uint8)


def _values(cache, scale, page, row, sb):
    """Values [..., Hkv, d] of rows ``row`` of pages ``page``, in 32 bits."""
    codes = _bytes_of(cache)[page, :, row].view(torch.float8_e4m3fn)
    return codes.float() * scale[page, :, row // sb].unsqueeze(-1)


def _plain_write(cache, scale, x, table, start, length, bs, sb):
    """Rows x [B, n, Hkv, d] become positions start .. start + length - 1, block of sb by block."""
    B, n = x.shape[:2]
    start, length = start.long()[:, None], length.long()[:, None]
    blocks = (n + 2 * sb - 2) // sb
    pos = start // sb * sb + torch.arange(blocks * sb, device="cuda")                           # [B, P]
    t = pos - start
    new = (t >= 0) & (t < length)
    touched = new.view(B, blocks, sb).any(-1)
    live = touched.repeat_interleave(sb, 1) & (t < length)                                      # kept rows and new ones
    page = table.long().gather(1, (pos // bs).clamp(max=table.shape[1] - 1)).clamp(min=0)
    val = x[torch.arange(B, device="cuda")[:, None], t.clamp(0, n - 1)].float()                 # [B, P, Hkv, d]
    kept = live & ~new
    val[kept] = _values(cache, scale, page[kept], (pos % bs)[kept], sb)
    val = val * live[..., None, None]
    val = val.view(B, blocks, sb, *x.shape[2:])
    s = _scale(val.abs().amax((2, 4)))                                                          # [B, blocks, Hkv]
    codes = (val / s[:, :, None, :, None]).to(torch.float8_e4m3fn).flatten(1, 2)
    _bytes_of(cache)[page[live], :, (pos % bs)[live]] = _bytes_of(codes)[live]
    first = pos.view(B, blocks, sb)[:, :, 0]
    scale[page.view(B, blocks, sb)[:, :, 0][touched], :, (first % bs // sb)[touched]] = s[touched]


def _plain_read(st):
    c = st["case"]
    n, bs = c["n"], c["bs"]
    pos = st["start_len"].long()[:, None] + torch.arange(n, device="cuda")
    there = pos < st["prefix_len"].long()[:, None]
    page = st["block_table"].long().gather(1, (pos // bs).clamp(max=st["block_table"].shape[1] - 1)).clamp(min=0)
    return tuple((_values(st[a + "_cache"], st[a + "_scale"], page, pos % bs, c["sb"]) * there[..., None, None]).to(_dtype(c))
                 for a in ("k", "v"))


def _plain_commit(st):
    c, table = st["case"], st["block_table"].long()
    bs, sb, m = c["bs"], c["sb"], c["m"]
    L, a = st["prefix_len"].long(), st["accept_len"].long()
    pos = L[:, None] + st["accept_path"].long().clamp(min=0)
    page = table.gather(1, pos // bs).clamp(min=0)
    rows = [_values(st[x + "_cache"], st[x + "_scale"], page, pos % bs, sb) for x in ("k", "v")]
    for x, r in zip(("k", "v"), rows):
        _plain_write(st[x + "_cache"], st[x + "_scale"], r, table, L, a, bs, sb)
    keep, used = -(-(L + a) // bs), -(-(L + m) // bs)
    at = torch.arange(table.shape[1], device="cuda")
    gone = at + keep[:, None] < used[:, None]
    freed = torch.where(gone, table.gather(1, (at + keep[:, None]).clamp(max=table.shape[1] - 1)), -1)
    left = torch.where((at >= keep[:, None]) & (at < used[:, None]), -1, table)
    return left.int(), (L + a).int(), freed.int(), (used - keep).int()


def _plain_attend(st):
    c = st["case"]
    B, m, Hq, Hkv, d, bs = c["B"], c["m"], c["Hq"], c["Hkv"], c["d"], c["bs"]
    g, table = Hq // Hkv, st["block_table"].long()
    there = table >= 0
    keys = table.shape[1] * bs

    def rows(a):                                                                        # [B, Hkv, keys, d]
        codes = _bytes_of(st[a + "_cache"])[table.clamp(min=0)].view(torch.float8_e4m3fn)
        val = codes.float().unflatten(3, (bs // c["sb"], c["sb"])) * st[a + "_scale"][table.clamp(min=0)][..., None, None]
        return (val.flatten(3, 4) * there[:, :, None, None, None]).transpose(1, 2).flatten(2, 3)

    t = torch.arange(keys, device="cuda") - st["prefix_len"].long()[:, None]             # [B, keys]
    at = t.clamp(0, m - 1)
    word = st["mask"].gather(2, (at // 64)[:, None].expand(-1, m, -1))
    seen = (t < 0)[:, None] | ((t < m)[:, None] & (((word >> (at % 64)[:, None]) & 1) == 1))   # [B, m, keys]
    q = st["q"].float().view(B, m, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, m * g, d)
    x = (q @ rows("k").transpose(2, 3)).view(B, Hkv, m, g, keys) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    o = (e.view(B, Hkv, m * g, keys) @ rows("v")).view(B, Hkv, m, g, d) / z
    lse = (top + torch.log(z)).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4).reshape(B, m, Hq, d).to(_dtype(c)), lse.permute(0, 2, 1, 3).reshape(B, m, Hq)


def run(st):
    c = st["case"]
    op = c["op"]
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if not own:
        if op == "write":
            for a in ("k", "v"):
                _plain_write(st[a + "_cache"], st[a + "_scale"], st[a], st["block_table"], st["start_len"], st["length"],
                             c["bs"], c["sb"])
            return cache
        if op == "commit":
            return _plain_commit(st) + cache
        return _plain_attend(st) if op == "attend" else _plain_read(st)
    import speculative_decoding_tree_eagle_gb300 as ts
    if op == "write":
        ts.kv_write_fp8(st["k"], st["v"], *cache, st["block_table"], st["start_len"], length=st["length"])
        return cache
    if op == "attend":
        return ts.tree_attention_fp8(st["q"], *cache, st["block_table"], st["prefix_len"], st["mask"],
                                     max_prefix=st["max_prefix"])
    if op == "read":
        return ts.kv_read_fp8(*cache, st["block_table"], st["prefix_len"], c["n"], start_len=st["start_len"], dtype=_dtype(c))
    r = ts.kv_commit_fp8(*cache, st["block_table"], st["prefix_len"], st["accept_path"], st["accept_len"])
    return (r["block_table"], r["prefix_len"], r["freed_blocks"], r["freed_count"]) + cache


# --------------------------------------------------------------------------------------------------- costs
def work(case):
    op, B, bs, sb = case["op"], case["B"], case["bs"], case["sb"]
    mean = (case["lo"] + case["hi"]) / 2
    size = 4 if case.get("dtype") == "f32" else 2
    head = case["Hkv"] * (case["d"] + 4 / sb)                  # bytes of a token's K (or V) codes and scales
    row = case["Hkv"] * case["d"] * size
    if op == "write":
        n = case["n"] if case["n"] == 1 or B == 1 else case["n"] * (1 - (B - 1) / B / 16)
        kept = 0 if case["hi"] == 0 else (sb - 1) / 2          # rows of the first block that were there
        return dict(bytes=B * (2 * n * row + 2 * n * head + 4 * kept * head + 4 * (n / bs + 1)), flops=8 * B * n * case["Hkv"] * case["d"])
    if op == "read":
        n = min(case["n"], case["new"] or case["n"], mean)
        return dict(bytes=2 * B * (n * (head + row) + (case["n"] - n) * row), flops=2 * B * n * case["Hkv"] * case["d"])
    if op == "commit":
        a = (1 + case["most"]) / 2
        width = -(-(case["hi"] + case["m"]) // bs)
        return dict(bytes=2 * B * (2 * a + (sb - 1)) * head + 12 * B * width, flops=8 * B * a * case["Hkv"] * case["d"])
    m, Hq, d = case["m"], case["Hq"], case["d"]
    return dict(bytes=2 * B * m * Hq * d * size + 4 * B * m * Hq + 2 * B * (mean + m) * head + 4 * B * (mean + m) / bs,
                flops=4.0 * B * m * Hq * d * (mean + (m + 1) / 2))


# --------------------------------------------------------------------------- the definitions, in 64 bits
def _e4m3(x):
    """The nearest of e4m3's values (three fraction bits, exponents from -6, at most 448), ties to even."""
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _two_to(e):
    """2^e for whole e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_write(cache, scale, rows, table, start, bs, sb):
    """cache, scale: float64 copies that change; rows [len, Hkv, d] float64; one sequence."""
    end = start + rows.shape[0]
    for first in range(start // sb * sb, end, 1024 * sb):
        last = min(first + 1024 * sb, -(-end // sb) * sb)
        pos = torch.arange(first, last, device="cuda")
        page, row = table[(pos // bs).clamp(max=table.numel() - 1)], pos % bs
        old = cache[page, :, row] * scale[page, :, row // sb][..., None]
        val = torch.where((pos < start)[:, None, None], old, rows[(pos - start).clamp(0, rows.shape[0] - 1)])
        val = torch.where((pos < end)[:, None, None], val, 0.0)
        big = val.abs().amax(-1).view(-1, sb, val.shape[1]).amax(1)                        # [blocks, Hkv]
        e = torch.ceil(torch.log2(big / E4M3_MAX))
        e = torch.where(big > 0, e, EXP_LO).clamp(EXP_LO, EXP_HI)
        e = torch.where(E4M3_MAX * _two_to(e - 1) >= big, e - 1, torch.where(E4M3_MAX * _two_to(e) < big, e + 1, e))
        e = e.clamp(EXP_LO, EXP_HI)
        code = _e4m3(val * _two_to(-e).repeat_interleave(sb, 0)[..., None])
        mine = pos < end
        cache[page[mine], :, row[mine]] = code[mine]
        scale[page[::sb], :, row[::sb] // sb] = _two_to(e)


def exact(case, seed):
    st = prepare(case, seed)
    op, B, bs, sb = case["op"], case["B"], case["bs"], case["sb"]
    table = st["block_table"].long()
    if op in ("write", "commit"):
        cache = [st[x].double() for x in ("k_cache", "v_cache", "k_scale", "v_scale")]
        start = st["start_len" if op == "write" else "prefix_len"].tolist()
        count = st["length" if op == "write" else "accept_len"].tolist()
        for b in range(B):
            for i, a in enumerate("kv"):
                codes, scale = cache[i], cache[2 + i]
                if op == "write":
                    rows = st[a][b, :count[b]].double()
                else:
                    pos = start[b] + st["accept_path"][b, :count[b]].long()
                    page, row = table[b][pos // bs], pos % bs
                    rows = codes[page, :, row] * scale[page, :, row // sb][..., None]
                _exact_write(codes, scale, rows, table[b], start[b], bs, sb)
        if op == "write":
            return tuple(cache)
        new, freed = table.cpu().numpy().copy(), np.full(table.shape, -1, dtype=np.int64)
        gone = []
        for b in range(B):
            keep, used = -(-(start[b] + count[b]) // bs), -(-(start[b] + case["m"]) // bs)
            gone.append(used - keep)
            freed[b, :used - keep] = new[b, keep:used]
            new[b, keep:used] = -1
        return (_ints(new), _ints([s + c for s, c in zip(start, count)]), _ints(freed), _ints(gone)) + tuple(cache)
    lens = st["prefix_len"].tolist()
    if op == "read":
        out = []
        for a in ("k", "v"):
            o = torch.zeros(B, case["n"], case["Hkv"], case["d"], dtype=torch.float64, device="cuda")
            for b in range(B):
                pos = torch.arange(int(st["start_len"][b]), min(lens[b], int(st["start_len"][b]) + case["n"]), device="cuda")
                page, row = table[b][pos // bs], pos % bs
                o[b, :pos.numel()] = (st[a + "_cache"].view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).double()
                                      * st[a + "_scale"][page, :, row // sb].double()[..., None])
            out.append(o)
        return tuple(out)
    m, Hq, Hkv, d = case["m"], case["Hq"], case["Hkv"], case["d"]
    g = Hq // Hkv
    out = torch.empty(B, m, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, m, Hq, dtype=torch.float64, device="cuda")
    node = torch.arange(m, device="cuda")
    for b in range(B):
        L = lens[b]
        ids = table[b, :-(-(L + m) // bs)]
        bits = (st["mask"][b][:, node // 64] >> (node % 64)) & 1                       # [m, m]
        seen = torch.cat([torch.ones(m, L, dtype=torch.bool, device="cuda"), bits == 1], 1)
        for h in range(Hkv):
            k, v = [(st[a + "_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double().view(-1, sb, d)
                     * st[a + "_scale"][ids, h].double().view(-1, 1, 1)).view(-1, d)[:L + m] for a in ("k", "v")]
            q = st["q"][b, :, h * g:(h + 1) * g].double()
            x = torch.einsum("ihc,jc->ihj", q, k) / math.sqrt(d)
            x = torch.where(seen[:, None], x, -math.inf)
            lse[b, :, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
            out[b, :, h * g:(h + 1) * g] = torch.einsum("ihj,jc->ihc", torch.softmax(x, -1), v)
    return out, lse
