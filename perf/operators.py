"""Measured cases of the paged 8-bit KV cache: append, attention over it, and its page operations.

The cache of one layer holds K and V codes [pages, kv_heads, page_tokens, head_dim] in 8 bits
(int8 or e4m3) and one fp32 scale for each block of 16 tokens and head, so that a stored value is
code * scale.  Sequences (rows) list their pages in an int32 table; refs counts the table entries
that name a page (0 = free).

Operators, with R rows and T new tokens (row r owns starts[r] .. starts[r+1] of them, or token r):

  append   A block's scale only grows: s' = max(s, max(amax, 2^-80) / top) over the finite new
           values of the block (s = 0 if the block holds no earlier token); earlier codes become
           rnd(code * s / s'), new ones rnd(x / s') (a product with the fp32 reciprocal of s'),
           clamped to +-top, top = 127 (int8) or 448 (e4m3); NaN is stored as 0.
  attend   out = softmax(scale q K^T) V for query i of a row at position len - n + i, over the keys
           j <= position (and j > position - window), lse = log of the softmax's sum; a query that
           sees no key gives 0 and -inf.
  fork     new rows that list (a prefix of) their parents' pages, with the reference counts that
           follow; then reserve: pages for the tokens to come, lowest free index first, and a copy
           of a partly filled last page that other rows list too.
  compact  the k-th live page with an index >= the number of live pages moves to the k-th hole.
"""
import math

import torch

own = False

BLOCK = 16
FLOOR = 2.0 ** -80
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


# ---- cases ---------------------------------------------------------------------------------------

def _case(op, **kw):
    c = {"op": op, "rows": 1, "new": 1, "len": 1, "ragged": False, "kv_heads": 8, "group": 6, "head_dim": 128,
         "page": 64, "dtype": "fp16", "code": "int8", "window": 0, "layers": 1}
    c.update(kw)
    return c


def listed():
    return [
        # a decode step of a small batch: one token for each of 16 sequences of the 27B-class layer
        # (K/V projections 1024 wide: 8 heads of 128), every block partly filled
        _case("append", name="append_step", rows=16, len=1500, ragged=True),
        # a scheduler's prefill chunk: several prompts' ragged pieces, some behind a cached prefix
        _case("append", name="append_chunk", rows=5, new=2049, len=3000, ragged=True, dtype="bf16", code="e4m3", page=32),
        # the largest admission: four prompts of 16K tokens at once
        _case("append", name="append_prompts", rows=4, new=16384, len=0),
        # one user's chat, one token: latency counts
        _case("attend", name="attend_one", rows=1, len=701),
        # continuous batching: 32 sequences of mixed lengths, some slots empty
        _case("attend", name="attend_step", rows=32, len=8191, ragged=True, dtype="bf16"),
        # few sequences with very long contexts
        _case("attend", name="attend_long", rows=4, len=130001, code="e4m3", page=128),
        # speculative verification: four draft tokens and the last sampled one, per sequence
        _case("attend", name="attend_verify", rows=8, new=5, len=16000, ragged=True),
        # the other split of the same projections (24 and 4 heads of 256), sliding window
        _case("attend", name="attend_window", rows=24, len=6000, ragged=True, kv_heads=4, head_dim=256, window=4096,
              dtype="bf16", page=16),
        # a prefill chunk behind a cached prefix
        _case("attend", name="attend_chunk", rows=1, new=2048, len=8192, dtype="bf16"),
        # first chunks of ragged prompts, small heads, odd group
        _case("attend", name="attend_prompts", rows=4, new=3001, len=3001, ragged=True, kv_heads=2, group=7, head_dim=64,
              page=32, code="e4m3"),
        # beams: 64 children of 16 parents, cut back to the verified tokens, then room for one token
        _case("fork", name="fork_beams", rows=16, new=64, len=4000, ragged=True, layers=4),
        # a fragmented pool (60% live) before a large admission
        _case("compact", name="compact_pool", rows=48, len=3276, layers=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "fork", "compact"])
    head_dim, kv_heads, group = rng.choice([(128, 8, 6), (256, 4, 6), (64, 2, 7), (128, 4, 1), (128, 2, 16), (64, 8, 3)])
    c = _case(op, kv_heads=kv_heads, group=group, head_dim=head_dim, page=rng.choice([16, 32, 64, 128]),
              dtype=rng.choice(["fp16", "bf16"]), code=rng.choice(["int8", "int8", "e4m3"]), ragged=rng.random() < 0.7)
    token = kv_heads * head_dim  # values of one token's K
    if op == "append":
        c["rows"] = _log(rng, 1, 64)
        c["new"] = rng.choice([1, _log(rng, 2, max(2, min(16384, 65536 // c["rows"])))])
        c["len"] = _log(rng, 1, 4000)
    elif op == "attend":
        if rng.random() < 0.6:  # single tokens and verification
            c["new"] = rng.choice([1, 1, rng.randint(2, 9)])
            c["rows"] = _log(rng, 1, 64)
            most = 500_000_000 // (token * c["rows"])
            c["len"] = _log(rng, c["new"], max(c["new"] + 1, min(131072, most)))
        else:  # chunks and prompts
            c["rows"] = _log(rng, 1, 6)
            heads = kv_heads * group
            c["new"] = _log(rng, 16, 3000)
            c["len"] = c["new"] + rng.choice([0, _log(rng, 1, 6000)])
            while c["rows"] > 1 and c["rows"] * heads * c["new"] * c["len"] > 700_000_000:
                c["rows"] -= 1
        if rng.random() < 0.25:
            c["window"] = _log(rng, 16, 4096)
    elif op == "fork":
        c["rows"] = _log(rng, 1, 32)
        c["new"] = _log(rng, 1, 96)
        c["len"] = _log(rng, 1, 4000)
        c["layers"] = rng.randint(1, 4)
    else:
        c["rows"] = _log(rng, 1, 48)
        c["len"] = _log(rng, 16, max(17, min(3276, 157_000_000 // (token * c["rows"]))))
        c["layers"] = rng.randint(1, 2)
    return c


def _ceil(a, b):
    return -(-a // b)


def _lens(c):
    """Lengths of the rows (before an append; with the new tokens otherwise), from the case alone."""
    n = []
    for r in range(c["rows"]):
        u = (r * 0.6180339887498949) % 1.0
        length = c["len"] if r == 0 or not c["ragged"] else int(c["len"] * u ** 1.5)
        if c["ragged"] and c["op"] == "attend" and c["new"] == 1 and r % 11 == 3:
            length = 0  # an empty slot of the batch
        n.append(length)
    return n


def _news(c):
    """New tokens of each row."""
    lens = _lens(c)
    n = []
    for r in range(c["rows"]):
        u = (0.37 + r * 0.7548776662466927) % 1.0
        k = c["new"] if r == 0 or not c["ragged"] or c["new"] == 1 else 1 + int((c["new"] - 1) * u)
        if c["op"] == "attend" and c["new"] > 1:
            k = min(k, lens[r])
        n.append(k)
    return n


def _visible(c):
    """(pairs of query and key, keys that are read) over the rows, for one head."""
    pairs = keys = 0
    for length, n in zip(_lens(c), _news(c)):
        lo = length
        for i in range(n):
            p = length - n + i
            if p < 0:
                continue
            first = max(0, p + 1 - c["window"]) if c["window"] else 0
            pairs += p + 1 - first
            lo = min(lo, first)
        keys += length - lo
    return pairs, keys


def work(case):
    c = case
    d, hk = c["head_dim"], c["kv_heads"]
    if c["op"] == "append":
        t = sum(_news(c))
        blocks = sum(_ceil(b + n, BLOCK) - b // BLOCK for b, n in zip(_lens(c), _news(c)))
        return {"bytes": 2 * hk * (t * d * 3 + blocks * 4) + 8 * c["rows"], "flops": 2 * t * hk * d * 4}
    if c["op"] == "attend":
        pairs, keys = _visible(c)
        t, hq = sum(_news(c)), hk * c["group"]
        return {"bytes": 2 * hk * (keys * d + 4 * _ceil(keys, BLOCK)) + t * hq * (4 * d + 4) + 4 * _ceil(keys, c["page"]),
                "flops": 4 * d * hq * pairs}
    page = 2 * hk * c["page"] * (d + 4 / BLOCK) * c["layers"]
    lens = _lens(c)
    if c["op"] == "fork":
        entries = sum(_ceil(x, c["page"]) for x in lens)
        kids = [_keep(c, i, lens[i % c["rows"]]) for i in range(c["new"])]
        copies = 0  # partly filled last pages that other children list, but for one keeper of each
        for p in range(c["rows"]):
            own_kids = kids[p::c["rows"]]
            for slot in {x // c["page"] for x in own_kids if x % c["page"]}:
                lists = sum(_ceil(x, c["page"]) > slot for x in own_kids)
                ends = sum(x // c["page"] == slot and x % c["page"] > 0 for x in own_kids)
                copies += 0 if lists == 1 else ends - (lists == ends)
        return {"bytes": 2 * page * copies + 4 * (entries + sum(_ceil(x, c["page"]) for x in kids) + 2 * _pool(c)),
                "flops": 0}
    live, pool = sum(_ceil(x, c["page"]) for x in lens), _pool(c)
    return {"bytes": 2 * page * live * (pool - live) / pool + 8 * (live + pool), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------

def _keep(c, i, length):
    """Verified tokens that child i keeps of a parent of this length."""
    return max(0, length - (i * 5) % 7)


def _pool(c):
    """Pages of the pool."""
    lens, news = _lens(c), _news(c)
    if c["op"] == "append":
        return sum(_ceil(x + n, c["page"]) for x, n in zip(lens, news)) + 3
    live = sum(_ceil(x, c["page"]) for x in lens)
    if c["op"] == "fork":
        return live + 2 * c["new"] + 8
    if c["op"] == "compact":
        return _ceil(live * 5, 3) + 1
    return live + 3


def _codes(c, shape, g, dev):
    x = torch.randn(shape, generator=g, device=dev)
    if c["code"] == "int8":
        return x.mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rows, hk, d, pt, pool = c["rows"], c["kv_heads"], c["head_dim"], c["page"], _pool(c)
    lens, news = _lens(c), _news(c)
    dt = DTYPES[c["dtype"]]
    held = [x + n for x, n in zip(lens, news)] if c["op"] == "append" else lens
    pages = [_ceil(x, pt) for x in held]
    width = max(1, max(pages) + (1 if c["op"] == "fork" else 0))
    # every page's place in the pool is random, as after a while of serving
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    slot, first = [], 0
    for n in pages:
        slot.append([first + j if j < n else -1 for j in range(width)])
        first += n
    slot = torch.tensor(slot, dtype=torch.int64, device=dev)
    table = torch.where(slot >= 0, perm[slot.clamp(min=0)], torch.full_like(slot, -1, dtype=torch.int32)).contiguous()
    refs = torch.zeros(pool, dtype=torch.int32, device=dev)
    refs[perm[:first].long()] = 1
    shape = (c["layers"], pool, hk, pt, d)
    st = {"case": c, "table": table, "refs": refs, "lens": torch.tensor(held, dtype=torch.int32, device=dev)}
    for n in ("k", "v"):
        st[n] = _codes(c, shape, g, dev)
        mean = (1 / 34.0) if c["code"] == "int8" else (1 / 110.0)
        st[n + "_scales"] = torch.randn(shape[:3] + (pt // BLOCK,), generator=g, device=dev).mul_(0.25).exp_().mul_(mean)
    t = sum(news)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    st["starts"] = None if c["new"] == 1 else torch.tensor(starts, dtype=torch.int32, device=dev)
    if c["op"] == "append":
        # K with a few strong channels, as after a rotary projection; k and v are views of one fused buffer
        kv = torch.randn((t, 2, hk, d), generator=g, device=dev)
        kv[:, 0] *= 1 + 5 * (torch.rand((hk, d), generator=g, device=dev) > 0.95)
        kv = kv.to(dt)
        st["new_k"], st["new_v"] = kv[:, 0], kv[:, 1]
        st["base"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    elif c["op"] == "attend":
        st["q"] = torch.randn((t, hk * c["group"], d), generator=g, device=dev).mul_(1.5).to(dt)
    elif c["op"] == "fork":
        par = [i % rows for i in range(c["new"])]
        st["parents"] = torch.tensor(par, dtype=torch.int32, device=dev)
        st["keep"] = torch.tensor([_keep(c, i, lens[p]) for i, p in enumerate(par)], dtype=torch.int32, device=dev)
        st["counts"] = torch.ones(c["new"], dtype=torch.int32, device=dev)
    return st


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact}[op](state)


def _run_own(st, op):
    c = st["case"]
    cache = st.get("cache")
    if cache is None:  # the handle that a serving program keeps over its pools and tables
        from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
        cache = st["cache"] = KVCache(st["k"], st["v"], st["k_scales"], st["v_scales"], st["table"], st["lens"], st["refs"])
    if op == "append":
        cache.append(st["new_k"], st["new_v"], st["base"], st["starts"], max_new=c["new"])
        return _pools(st)
    if op == "attend":
        out, lse = cache.attend(st["q"], st["starts"], max_new=c["new"], max_len=c["len"], window=c["window"])
        return {"out": out, "lse": lse}
    if op == "fork":
        child = cache.fork(st["parents"], st["keep"])
        base, status = child.reserve(st["counts"])
        return {"table": child.table, "lens": child.lens, "refs": child.refs, "base": base, "status": status, **_pools(st)}
    new, moved = cache.compact()
    return {"table": new.table, "refs": new.refs, "moved": moved, **_pools(st)}


def _pools(st):
    return {n: st[n] for n in ("k", "v", "k_scales", "v_scales")}


def _blocks(x):
    """The bytes of a layer's codes [pages, heads, page, d] by blocks of 16 tokens: [pages, heads, page / 16, 16, d]."""
    p, h, pt, d = x.shape
    return x.view(torch.int8).view(p, h, pt // BLOCK, BLOCK, d)


def _move(st, dst, src):
    """Copies pages of every layer's codes and scales."""
    for x in (st["k"].view(torch.int8), st["v"].view(torch.int8), st["k_scales"], st["v_scales"]):
        x[:, dst] = x[:, src]


def _encode(x, code):
    """fp32 quotients to codes: rounded to nearest even, clamped, NaN as 0."""
    x = torch.nan_to_num(x, nan=0.0, posinf=TOP[code], neginf=-TOP[code]).clamp(-TOP[code], TOP[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _plain_append(st):
    c, dev = st["case"], st["table"].device
    pt, code, top = c["page"], c["code"], TOP[c["code"]]
    rows = st["table"].shape[0]
    base = st["base"].long()
    t = st["new_k"].shape[0]
    starts = st["starts"].long() if st["starts"] is not None else torch.arange(rows + 1, device=dev)
    n = starts[1:] - starts[:-1]
    most = c["new"]
    # touched blocks of each row: [rows, nb], their tokens [rows, nb, 16]
    nb = (most + 2 * BLOCK - 2) // BLOCK
    block = base[:, None] // BLOCK + torch.arange(nb, device=dev)
    real = (block * BLOCK < (base + n)[:, None]) & (n[:, None] > 0)
    pos = block[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)
    fresh = (pos >= base[:, None, None]) & (pos < (base + n)[:, None, None])
    older = (pos < base[:, None, None])
    src = (starts[:-1, None, None] + pos - base[:, None, None]).clamp(0, t - 1)
    at, which = torch.nonzero(real, as_tuple=True)
    b, fresh, older, src = block[at, which], fresh[at, which], older[at, which], src[at, which]
    page = st["table"][at, b * BLOCK // pt].long()
    sub = b % (pt // BLOCK)
    for new, pool, scales in ((st["new_k"], st["k"][0], st["k_scales"][0]), (st["new_v"], st["v"][0], st["v_scales"][0])):
        x = new[src].float().permute(0, 2, 1, 3)                       # [blocks, heads, 16, d]
        f = fresh[:, None, :, None]
        mag = torch.where(f & x.isfinite(), x.abs(), torch.zeros_like(x)).amax(dim=(2, 3))
        codes = _blocks(pool)
        old = codes[page, :, sub].view(CODES[code])
        s0 = torch.where(older.any(dim=1)[:, None], scales[page, :, sub], torch.zeros_like(mag))
        s = torch.maximum(s0, mag.clamp(min=FLOOR) * (1.0 / top))
        inv = (torch.ones_like(s) / s)[:, :, None, None]
        kept = _encode(old.float() * s0[:, :, None, None] * inv, code)
        fill = _encode(x * inv, code)
        bits = torch.where(f, fill.view(torch.int8), torch.where(older[:, None, :, None], kept.view(torch.int8), old.view(torch.int8)))
        codes[page, :, sub] = bits
        scales[page, :, sub] = s
    return _pools(st)


def _plain_attend(st):
    c, dev = st["case"], st["table"].device
    hk, grp, d, pt = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    rows, width = st["table"].shape
    lens, q = st["lens"].long(), st["q"]
    t = q.shape[0]
    starts = st["starts"].long() if st["starts"] is not None else torch.arange(rows + 1, device=dev)
    n, most = starts[1:] - starts[:-1], c["new"]
    page = st["table"].clamp(min=0).long()

    def rows_of(codes, scales):  # [rows, heads, tokens, d] in fp32
        x = _blocks(codes[0])[page].view(codes.dtype).float() * scales[0][page][..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(rows, hk, width * pt, d)

    j = torch.arange(width * pt, device=dev)
    held = (j < lens[:, None])[:, None, :, None]
    k = rows_of(st["k"], st["k_scales"]).masked_fill(~held, 0.0)
    v = rows_of(st["v"], st["v_scales"]).masked_fill(~held, 0.0)
    i = torch.arange(most, device=dev)
    at = (starts[:-1, None] + i).clamp(max=t - 1)                      # [rows, most]
    qf = q[at].float().view(rows, most, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(rows, hk, grp * most, d)
    s = (qf @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(rows, hk, grp, most, width * pt)
    pos = (lens - n)[:, None] + i                                      # [rows, most]
    sees = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if c["window"]:
        sees &= j > pos[:, :, None] - c["window"]
    s.masked_fill_(~sees[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = (p.view(rows, hk, grp * most, width * pt) @ v).view(rows, hk, grp, most, d) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (l.log() + m).squeeze(-1)
    real = i < n[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(rows, most, hk * grp, d)[real].to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(rows, most, hk * grp)[real]}


def _uses(table, count, pool):
    """How often each page is listed in the first count[r] entries of the rows."""
    listed_ = torch.arange(table.shape[1], device=table.device) < count[:, None]
    return torch.zeros(pool, dtype=torch.int32, device=table.device).index_add_(
        0, table[listed_].long(), torch.ones_like(table[listed_]))


def _plain_fork(st):
    table, lens, refs, dev = st["table"], st["lens"], st["refs"], st["table"].device
    pt, pool, width = st["case"]["page"], st["refs"].shape[0], st["table"].shape[1]
    # fork
    par = st["parents"].long()
    new_lens = torch.minimum(lens[par], st["keep"])
    filled = (new_lens + pt - 1) // pt
    j = torch.arange(width, device=dev, dtype=torch.int32)
    new = torch.where(j < filled[:, None], table[par], torch.full_like(table[par], -1))
    refs = refs - _uses(table, (lens + pt - 1) // pt, pool) + _uses(new, filled, pool)
    # reserve
    cnt = st["counts"]
    rows = new.shape[0]
    r = torch.arange(rows, device=dev)
    part = (cnt > 0) & (new_lens % pt != 0)
    last = new.gather(1, (new_lens // pt).clamp(max=width - 1).long()[:, None])[:, 0]
    last = torch.where(part, last, torch.full_like(last, -1))
    same = (last[:, None] == last[None, :]) & part[:, None] & part[None, :]
    shared = part & (refs[last.clamp(min=0).long()] > 1)
    keeper = ~(same & (r[None, :] < r[:, None])).any(dim=1) & (same.sum(dim=1) == refs[last.clamp(min=0).long()])
    copy = shared & ~keeper
    end = (new_lens + cnt + pt - 1) // pt
    need = torch.where(cnt > 0, end - filled + copy.int(), torch.zeros_like(cnt))
    before = need.cumsum(0) - need
    free = torch.argsort((refs > 0).int(), stable=True).to(torch.int32)
    first = filled - copy.int()                                       # first table slot that gets a new page
    k = j[None, :] - first[:, None]
    gets = (k >= 0) & (k < need[:, None])
    grown = torch.where(gets, free[(before[:, None] + k).clamp(0, pool - 1).long()], new)
    refs = refs.index_add(0, grown[gets].long(), torch.ones_like(grown[gets]))
    refs = refs.index_add(0, last[copy].long(), -torch.ones_like(last[copy]))
    src, dst = last[copy].long(), free[before[copy].long()].long()
    _move(st, dst, src)
    status = torch.zeros(2, dtype=torch.int32, device=dev)
    return {"table": grown, "lens": new_lens + cnt, "refs": refs, "base": new_lens, "status": status, **_pools(st)}


def _plain_compact(st):
    refs, dev = st["refs"], st["refs"].device
    pool = refs.shape[0]
    live = (refs > 0)
    count = live.sum()
    idx = torch.arange(pool, device=dev)
    src = idx[live & (idx >= count)]
    dst = idx[~live & (idx < count)]
    to = idx.clone()
    to[src] = dst
    new_refs = torch.where(idx < count, refs, torch.zeros_like(refs))
    new_refs[dst] = refs[src]
    filled = (st["lens"] + st["case"]["page"] - 1) // st["case"]["page"]
    held = torch.arange(st["table"].shape[1], device=dev) < filled[:, None]
    table = torch.where(held, to[st["table"].clamp(min=0).long()].to(torch.int32), torch.full_like(st["table"], -1))
    _move(st, dst, src)
    return {"table": table, "refs": new_refs, "moved": (live & (idx >= count)).sum().to(torch.int32).view(1), **_pools(st)}


# ---- in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    """From the definitions, a row at a time, in 64 bits; the page operations compute no numbers."""
    c = case
    if c["op"] not in ("append", "attend"):
        return None
    st = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(c, st)
    return _exact_attend(c, st)


def _exact_append(c, st):
    """The blocks' scales are maxima of the values themselves; codes are whole numbers and have no 64-bit value."""
    pt, top = c["page"], TOP[c["code"]]
    out = {"k": None, "v": None}
    table, starts = st["table"].tolist(), None if st["starts"] is None else st["starts"].tolist()
    base = st["base"].tolist()
    for name in ("k", "v"):
        scales = st[name + "_scales"].double().clone()
        mag = st["new_" + name].double().abs().amax(dim=2)            # [tokens, heads]
        for r, b0 in enumerate(base):
            lo, hi = (r, r + 1) if starts is None else (starts[r], starts[r + 1])
            n = hi - lo
            if n == 0:
                continue
            first, last = b0 // BLOCK, (b0 + n - 1) // BLOCK
            pad = torch.zeros(((last - first + 1) * BLOCK, mag.shape[1]), dtype=torch.float64, device=mag.device)
            pad[b0 - first * BLOCK: b0 - first * BLOCK + n] = mag[lo:hi]
            s = pad.view(-1, BLOCK, mag.shape[1]).amax(dim=1).clamp(min=FLOOR) / top
            blocks = torch.arange(first, last + 1, device=mag.device)
            pages = torch.tensor(table[r], device=mag.device)[blocks * BLOCK // pt]
            sub = blocks % (pt // BLOCK)
            if b0 % BLOCK:
                s[0] = torch.maximum(s[0], scales[0, pages[0], :, sub[0]])
            scales[0, pages, :, sub] = s
        out[name + "_scales"] = scales
    return out


def _exact_attend(c, st):
    hk, grp, d, pt = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    outs, lses = [], []
    lo = 0
    for r, (length, n) in enumerate(zip(_lens(c), _news(c))):
        q = st["q"][lo:lo + n].double().view(n, hk, grp, d)
        lo += n
        o = torch.zeros((n, hk, grp, d), dtype=torch.float64, device=q.device)
        e = torch.full((n, hk, grp), -math.inf, dtype=torch.float64, device=q.device)
        pages = st["table"][r, :_ceil(length, pt)].long()
        pos = torch.arange(length - n, length, device=q.device)
        j = torch.arange(length, device=q.device)
        sees = j[None, :] <= pos[:, None]
        if c["window"]:
            sees &= j[None, :] > pos[:, None] - c["window"]
        for h in range(hk if length else 0):
            kv = [(x.view(torch.int8)[0, pages, h].view(x.dtype).double().view(-1, BLOCK, d) * s[0, pages, h].double().reshape(-1, 1, 1)).view(-1, d)[:length]
                  for x, s in ((st["k"], st["k_scales"]), (st["v"], st["v_scales"]))]
            for g in range(grp):
                s = (q[:, h, g] @ kv[0].T / math.sqrt(d)).masked_fill(~sees, -math.inf)
                e[:, h, g] = torch.logsumexp(s, dim=1)
                some = e[:, h, g] > -math.inf
                o[some, h, g] = torch.exp(s[some] - e[some, h, g, None]) @ kv[1]
        outs.append(o.view(n, hk * grp, d))
        lses.append(e.view(n, hk * grp))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
