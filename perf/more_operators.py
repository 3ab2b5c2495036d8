"""Measured cases of a decode step's operators around the 8-bit KV cache when a tree of tokens is drafted.

A step of speculative decoding with trees: row r (a sequence) has n drafted nodes, tokens
starts[r] .. starts[r + 1] - 1 of the ragged batch, in an order that puts a parent before its
children; parents[i] is the row's own index of node i's parent (-1: a root).  Node 0 is the last
token that the target chose.

  rope      queries and keys of each head, in one pass: y = x / sqrt(mean(x^2) + eps) * w, then the
            first rotary_dim values are turned by the angle position * inv_freq[j]: pair j is
            (j, j + rotary_dim / 2), or (2 j, 2 j + 1) where interleaved.
  tree      attention over the cache for the row's last n tokens: node i sees every token before the
            nodes (a prefix of lens - n) and the nodes whose bit is set in its mask (its ancestors and
            itself); with a window, the prefix tokens j > lens - n + depth[i] - window.
            out = softmax(scale q K^T) V, lse = log of the softmax's sum.
  verify    the nodes' ancestor masks, depths and positions from their parents; then t[i] = argmax of
            node i's logits, and from node 0 on the walk to the lowest child c whose token is t of the
            node before it: its path, the drafts that it accepts, and the target's next token.
  accept    the cache keeps the path's tokens alone: token lens - n + path[k] moves to lens - n + k in
            every layer.  A 16-token block that gets them takes the largest of its tokens' scales;
            codes of another scale are rounded again, rnd(code * s * (1 / s')).  Rows shrink to what
            they keep, and pages that no row lists any more are free.
  logprobs  for each row of logits: log softmax at a given token, the softmax's entropy, how many
            entries come before the token (larger, or equal with a lower index), and the k most likely
            tokens with their log probabilities.
"""
import math

import torch

own = False

BLOCK = 16
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------

def _rope(**kw):
    return {"op": "rope", "tokens": 1, "kv_heads": 8, "group": 6, "head_dim": 128, "rotary": 128, "interleaved": False,
            "dtype": "fp16", "far": 4096, **kw}


def _tree(op, **kw):
    return {"op": op, "rows": 1, "nodes": 26, "len": 701, "ragged": False, "kv_heads": 8, "group": 6, "head_dim": 128,
            "page": 64, "dtype": "fp16", "code": "int8", "window": 0, "layers": 1, **kw}


def _logits(op, **kw):
    return {"op": op, "rows": 1, "nodes": 26, "vocab": 151936, "ragged": False, "dtype": "fp16", "top": 20, **kw}


def listed():
    return [
        # a decode step of a small batch: one token of 16 sequences, 48 query and 8 key heads of 128
        _rope(name="rope_step", tokens=16),
        # a prefill chunk far behind a long prefix
        _rope(name="rope_chunk", tokens=2049, dtype="bf16", far=131072),
        # an admission of several prompts; the other split of the same projections (heads of 256), of
        # which a quarter is rotated in adjacent pairs
        _rope(name="rope_prompts", tokens=16384, kv_heads=4, head_dim=256, rotary=64, interleaved=True, dtype="bf16",
              far=16384),
        # one user's chat: a tree of 26 drafts; latency counts
        _tree("tree", name="tree_one"),
        # a batch of sequences of mixed lengths, trees of up to 64 nodes
        _tree("tree", name="tree_step", rows=8, nodes=64, len=16000, ragged=True, dtype="bf16"),
        # few sequences with very long contexts, small trees
        _tree("tree", name="tree_long", rows=4, nodes=8, len=65001, code="e4m3", page=128),
        # one user's chat: the whole vocabulary for each node of one tree
        _logits("verify", name="verify_one"),
        # 16 trees of up to 64 nodes
        _logits("verify", name="verify_step", rows=16, nodes=64, ragged=True, dtype="bf16"),
        # the accepted path of one tree
        _tree("accept", name="accept_one", layers=4),
        # the accepted paths of a batch, several layers
        _tree("accept", name="accept_step", rows=32, nodes=64, len=3000, ragged=True, layers=8, page=32),
        # a chat's reply with 20 alternatives for each token: one row a step
        _logits("logprobs", name="logprobs_one", nodes=0),
        # the log probabilities of a prompt's own tokens
        _logits("logprobs", name="logprobs_prompt", rows=2049, nodes=0, dtype="bf16", top=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "verify", "verify", "accept", "logprobs", "logprobs"])
    head_dim, kv_heads, group = rng.choice([(128, 8, 6), (256, 4, 6), (64, 2, 7), (128, 4, 1), (128, 2, 16), (64, 8, 3)])
    if op == "rope":
        far = _log(rng, 16, 1 << 20)
        return _rope(tokens=_log(rng, 1, min(16384, 50_000_000 // (kv_heads * (group + 1) * head_dim))), kv_heads=kv_heads,
                     group=group, head_dim=head_dim, rotary=rng.choice([head_dim, head_dim, head_dim // 2, 32, 16]),
                     interleaved=rng.random() < 0.4, dtype=rng.choice(["fp16", "bf16"]), far=far)
    if op in ("verify", "logprobs"):
        c = _logits(op, vocab=rng.choice([_log(rng, 40, 260_000), 151936, 32000, 50257]), ragged=rng.random() < 0.7,
                    dtype=rng.choice(["fp16", "bf16", "fp32"]), top=rng.choice([0, 1, 5, 20, 32]))
        most = min(60_000, 280_000_000 // c["vocab"])  # rows of logits
        if op == "verify":
            c["nodes"] = _log(rng, 1, 128)
            c["rows"] = _log(rng, 1, max(1, min(64, most // c["nodes"])))
        else:
            c["nodes"], c["rows"] = 0, _log(rng, 1, min(4000, most))
            c["top"] = min(c["top"], c["vocab"])
        return c
    c = _tree(op, nodes=_log(rng, 1, 128), ragged=rng.random() < 0.7, kv_heads=kv_heads, group=group, head_dim=head_dim,
              page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["fp16", "bf16"]), code=rng.choice(["int8", "int8", "e4m3"]))
    c["rows"] = _log(rng, 1, 32)
    if op == "tree":
        most = min(100_000, 300_000_000 // (kv_heads * head_dim * c["rows"]),
                   1_000_000_000 // (kv_heads * group * c["rows"] * c["nodes"]))
        c["len"] = c["nodes"] + _log(rng, 1, max(2, most))
        if rng.random() < 0.25:
            c["window"] = _log(rng, 16, 4096)
    else:
        c["layers"] = rng.randint(1, 8)
        c["len"] = c["nodes"] + _log(rng, 1, max(2, min(4000, 400_000_000 // (kv_heads * head_dim * c["rows"] * c["layers"]))))
    return c


def _ceil(a, b):
    return -(-a // b)


def _nodes(c):
    """Nodes of each row."""
    n = []
    for r in range(c["rows"]):
        u = (0.37 + r * 0.7548776662466927) % 1.0
        n.append(c["nodes"] if r == 0 or not c["ragged"] else 1 + int((c["nodes"] - 1) * u))
    return n


def _lens(c):
    """Lengths of the rows, their nodes among them."""
    n = []
    for r, k in enumerate(_nodes(c)):
        u = (r * 0.6180339887498949) % 1.0
        n.append(c["len"] if r == 0 or not c["ragged"] else max(k, int(c["len"] * u ** 1.5)))
    return n


def _parents(c, r, n):
    """A row's tree: node 0 is the root, others hang below a node that is more likely a late one."""
    p = [-1]
    for i in range(1, n):
        u = ((i + 1) * 0.5698402909980532 + r * 0.7548776662466927) % 1.0
        p.append(int(i * (1 - u ** 2)) if i > 4 else 0)
    return [min(x, i - 1) for i, x in enumerate(p)]


def _trees(c):
    """(parents, ancestors and itself, depth) of each row's nodes."""
    found = []
    for r, n in enumerate(_nodes(c)):
        par = _parents(c, r, n)
        seen, depth = [], []
        for i, p in enumerate(par):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        found.append((par, seen, depth))
    return found


def _path(c, r):
    """An accepted path of the row's tree, as verification returns it: nodes from the root down, then -1."""
    par = _parents(c, r, _nodes(c)[r])
    path = [0]
    while True:
        kids = [i for i, p in enumerate(par) if p == path[-1]]
        if not kids or (r * 5 + len(path)) % 7 == 6:
            return path
        path.append(kids[(r + len(path)) % len(kids)])


def _words(c):
    return _ceil(max(1, c["nodes"]), 64)


def work(case):
    c = case
    op = c["op"]
    if op == "rope":
        values = c["tokens"] * c["kv_heads"] * (c["group"] + 1) * c["head_dim"]
        return {"bytes": 4 * values + 4 * c["tokens"] + 4 * c["rotary"] + 4 * c["head_dim"], "flops": 7 * values}
    if op == "tree":
        d, hk = c["head_dim"], c["kv_heads"]
        pairs = keys = 0
        for n, length, (_, seen, depth) in zip(_nodes(c), _lens(c), _trees(c)):
            before = length - n
            for m, e in zip(seen, depth):
                pairs += bin(m).count("1") + (min(before, max(0, c["window"] - e - 1)) if c["window"] else before)
            keys += n + (min(before, c["window"] - 1) if c["window"] else before)
        t, hq = sum(_nodes(c)), hk * c["group"]
        return {"bytes": 2 * hk * (keys * d + 4 * _ceil(keys, BLOCK)) + t * (hq * (4 * d + 4) + 8 * _words(c)) +
                4 * _ceil(keys, c["page"]), "flops": 4 * d * hq * pairs}
    size = {"fp16": 2, "bf16": 2, "fp32": 4}[c["dtype"]]
    if op == "verify":
        t = sum(_nodes(c))
        return {"bytes": t * (c["vocab"] * size + 8 + 8 * _words(c) + 12) + c["rows"] * (12 + 4 * c["nodes"]), "flops": 0}
    if op == "logprobs":
        return {"bytes": c["rows"] * (c["vocab"] * size + 16 + 8 * c["top"]), "flops": 5 * c["rows"] * c["vocab"]}
    token = 2 * c["layers"] * c["kv_heads"] * (c["head_dim"] + 4)
    moved = sum(sum(k != p for k, p in enumerate(_path(c, r))) for r in range(c["rows"]))
    entries = sum(_ceil(x, c["page"]) for x in _lens(c))
    return {"bytes": 2 * token * moved + 4 * (2 * entries + 2 * _pool(c)) + c["rows"] * (12 + 4 * c["nodes"]), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------

def _pool(c):
    return sum(_ceil(x, c["page"]) for x in _lens(c)) + 3


def _inv_freq(c):
    return [10000.0 ** (-2.0 * j / c["rotary"]) for j in range(c["rotary"] // 2)]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(c):
    s = [0]
    for n in _nodes(c):
        s.append(s[-1] + n)
    return s


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "rope":
        t, hk, hq, d = c["tokens"], c["kv_heads"], c["kv_heads"] * c["group"], c["head_dim"]
        # q, k and v of one fused projection; the norms' weights as trained ones spread
        qkv = (normal(t, hq + 2 * hk, d) * (1 + 3 * torch.rand((1, hq + 2 * hk, 1), generator=g, device=dev))).to(dt)
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        st["q_weight"], st["k_weight"] = ((1 + 0.3 * normal(d)).to(dt) for _ in range(2))
        first = int(torch.randint(0, max(1, c["far"] - t), (1,), generator=g, device=dev).item())
        st["positions"] = (first + torch.arange(t, device=dev)).to(torch.int32)
        st["inv_freq"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device=dev)
        return st
    if c["op"] == "logprobs":
        x = normal(c["rows"], c["vocab"]).mul_(2.5)
        # the given tokens are those that such a model would say: the largest of a few draws
        tries = torch.randint(0, c["vocab"], (c["rows"], 4096), generator=g, device=dev)
        best = (x.gather(1, tries) + 1.5 * normal(c["rows"], 4096)).argmax(dim=1)
        st["logits"], st["tokens"] = x.to(dt), tries.gather(1, best[:, None])[:, 0].to(torch.int32)
        return st
    trees = _trees(c)
    st["starts"] = _i32(_starts(c))
    st["parents"] = _i32([p for par, _, _ in trees for p in par])
    if c["op"] == "verify":
        t = sum(_nodes(c))
        x = normal(t, c["vocab"]).mul_(2.5)
        tok = torch.randint(0, c["vocab"], (t,), generator=g, device=dev)
        # the target agrees with one child of most nodes on the way down
        lo = torch.tensor(_starts(c)[:-1], device=dev)
        agreed = [[_starts(c)[r] + n for n in _path(c, r)] for r in range(c["rows"])]
        above = torch.tensor([i for p in agreed for i in p[:-1]], dtype=torch.int64, device=dev)
        below = torch.tensor([i for p in agreed for i in p[1:]], dtype=torch.int64, device=dev)
        x[above, tok[below]] = 20.0
        st["logits"], st["tokens"] = x.to(dt), tok.to(torch.int32)
        st["base"] = (torch.randint(0, 4000, lo.shape, generator=g, device=dev)).to(torch.int32)
        return st
    rows, hk, d, pt, pool = c["rows"], c["kv_heads"], c["head_dim"], c["page"], _pool(c)
    lens = _lens(c)
    pages = [_ceil(x, pt) for x in lens]
    width = max(pages)
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    slot, first = [], 0
    for n in pages:
        slot.append([first + j if j < n else -1 for j in range(width)])
        first += n
    slot = torch.tensor(slot, dtype=torch.int64, device=dev)
    st["table"] = torch.where(slot >= 0, perm[slot.clamp(min=0)], torch.full_like(slot, -1, dtype=torch.int32)).contiguous()
    st["refs"] = torch.zeros(pool, dtype=torch.int32, device=dev)
    st["refs"][perm[:first].long()] = 1
    st["lens"] = _i32(lens)
    shape = (c["layers"], pool, hk, pt, d)
    for n in ("k", "v"):
        x = normal(*shape)
        if c["code"] == "int8":
            st[n] = x.mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
        else:
            st[n] = x.mul_(110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        mean = (1 / 34.0) if c["code"] == "int8" else (1 / 110.0)
        st[n + "_scales"] = normal(*shape[:3], pt // BLOCK).mul_(0.25).exp_().mul_(mean)
    if c["op"] == "tree":
        st["q"] = normal(sum(_nodes(c)), hk * c["group"], d).mul_(1.5).to(dt)
        # a static tree's masks are the plan that a program keeps; every layer reads them
        w = _words(c)
        bits = [[(m >> 64 * i) & (2 ** 64 - 1) for i in range(w)] for _, seen, _ in trees for m in seen]
        st["mask"] = torch.tensor([[b - 2 ** 64 if b >= 2 ** 63 else b for b in row] for row in bits], device=dev)
        st["depth"] = _i32([x for _, _, depth in trees for x in depth])
    else:
        paths = [_path(c, r) for r in range(rows)]
        st["path"] = _i32([p + [-1] * (c["nodes"] - len(p)) for p in paths])
    return st


# ---- one pass ------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify, "accept": _plain_accept,
            "logprobs": _plain_logprobs}[op](state)


def _run_own(st, op):
    import bit_quantized_decode_unpack_gb300 as bqd
    c = st["case"]
    if op == "rope":
        plan = st.get("plan")
        if plan is None:  # a layer's weights and frequencies
            plan = st["plan"] = bqd.QKNormRope(c["head_dim"], st["inv_freq"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                                               eps=EPS, interleaved=c["interleaved"])
        q, k = plan(st["q"], st["k"], st["positions"])
        return {"q": q, "k": k}
    if op == "logprobs":
        r = bqd.token_logprobs(st["logits"], st["tokens"], top=c["top"])
        return {"logprob": r.logprob, "entropy": r.entropy, "rank": r.rank, "top_ids": r.top_ids, "top_logprobs": r.top_logprobs}
    if op == "verify":
        mask, depth, positions = bqd.tree_mask(st["parents"], st["starts"], words=_words(c), base=st["base"])
        accepted, token, path = bqd.spec_tree_verify(st["logits"], st["tokens"], st["parents"], st["starts"],
                                                     max_path=c["nodes"])
        return {"mask": mask, "depth": depth, "positions": positions, "accepted": accepted, "next": token, "path": path}
    cache = st.get("cache")
    if cache is None:  # the handle that a serving program keeps over its pools and tables
        cache = st["cache"] = bqd.KVCache(st["k"], st["v"], st["k_scales"], st["v_scales"], st["table"], st["lens"], st["refs"])
    if op == "tree":
        out, lse = cache.attend(st["q"], st["starts"], mask=st["mask"], depth=st["depth"], max_new=c["nodes"],
                                max_len=c["len"], window=c["window"])
        return {"out": out, "lse": lse}
    new = cache.accept(st["path"], st["starts"])
    return {"table": new.table, "lens": new.lens, "refs": new.refs, **_pools(st)}


def _pools(st):
    return {n: st[n] for n in ("k", "v", "k_scales", "v_scales")}


def _plain_rope(st):
    c = st["case"]
    half = c["rotary"] // 2
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * w.float()
        r = x[..., :c["rotary"]]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((a, b), dim=-1).flatten(2) if c["interleaved"] else torch.cat((a, b), dim=-1)
        return torch.cat((r, x[..., c["rotary"]:]), dim=-1)

    return {"q": turned(st["q"], st["q_weight"]).to(st["q"].dtype), "k": turned(st["k"], st["k_weight"]).to(st["k"].dtype)}


def _plain_logprobs(st):
    x, k = st["logits"].float(), st["case"]["top"]
    rows, vocab = x.shape
    tok = st["tokens"].long()[:, None]
    i = torch.arange(vocab, device=x.device)
    m = x.amax(dim=1, keepdim=True)
    d = x - m
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    entropy = total.log()[:, 0] - (e.mul_(d).sum(dim=1) / total[:, 0])
    at = x.gather(1, tok)
    rank = ((x > at) | ((x == at) & (i < tok))).sum(dim=1).to(torch.int32)
    # the k first by value, then by index: a whole number that orders like both
    bits = (x + 0.0).view(torch.int32).long()
    keys = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits) * 2 ** 32 + (2 ** 32 - 1 - i)
    ids = torch.topk(keys, k, dim=1).indices
    return {"logprob": (d.gather(1, tok) - total.log())[:, 0], "entropy": entropy, "rank": rank,
            "top_ids": ids.to(torch.int32), "top_logprobs": d.gather(1, ids) - total.log()}


def _batch(st, rows, most):
    """(real [rows, most], index into the ragged tokens [rows, most], nodes of each row)."""
    starts = st["starts"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(most, device=starts.device)
    return i < n[:, None], (starts[:-1, None] + i).clamp(max=int(st["parents"].shape[0]) - 1), n


def _plain_verify(st):
    c, dev = st["case"], st["starts"].device
    rows, most, words = c["rows"], c["nodes"], _words(c)
    real, at, n = _batch(st, rows, most)
    i = torch.arange(most, device=dev)
    par = torch.where(real, st["parents"].long()[at], torch.full_like(at, -1))
    # ancestors: walks along parent edges of any length
    step = (par[:, :, None] == i).double() + torch.eye(most, dtype=torch.float64, device=dev)
    seen = torch.matrix_power(step, most) > 0                          # [rows, node, ancestor]
    bits = torch.nn.functional.pad(seen, (0, 64 * words - most)).view(rows, most, words, 64).long()
    mask = (bits << torch.arange(64, device=dev)).sum(dim=3)
    depth = seen.sum(dim=2) - 1
    positions = st["base"].long()[:, None] + depth
    t = st["logits"].float().argmax(dim=1)
    tok = st["tokens"].long()[at]
    said = torch.where(par >= 0, t[at].gather(1, par.clamp(min=0)), torch.full_like(par, -1))
    agrees = (said == tok) & (par >= 0) & real
    twin = (par[:, :, None] == par[:, None, :]) & agrees[:, None, :] & (i < i[:, None])   # an earlier child that agrees
    fine = (agrees & ~twin.any(dim=2)) | (i == 0)
    on = (seen <= fine[:, None, :]).all(dim=2) & seen[:, :, 0] & real  # every node from the root down agrees
    count = on.sum(dim=1)
    order = torch.argsort(torch.where(on, i, i + most), dim=1)
    path = torch.where(i < count[:, None], order, torch.full_like(order, -1))
    last = at.gather(1, path.gather(1, (count - 1).clamp(min=0)[:, None]).clamp(min=0))[:, 0]
    as_i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"mask": mask[real], "depth": as_i32(depth[real]), "positions": as_i32(positions[real]),
            "accepted": as_i32(count - 1), "next": as_i32(t[last]), "path": as_i32(path)}


def _blocks(x):
    """The bytes of codes [layers, pages, heads, page, d] by blocks of 16 tokens: [layers, pages, heads, page / 16, 16, d]."""
    la, p, h, pt, d = x.shape
    return x.view(torch.int8).view(la, p, h, pt // BLOCK, BLOCK, d)


def _plain_tree(st):
    c, dev = st["case"], st["table"].device
    hk, grp, d, pt = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    rows, width = st["table"].shape
    most, lens = c["nodes"], st["lens"].long()
    starts = st["starts"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(most, device=dev)
    real, at = i < n[:, None], (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    page = st["table"].clamp(min=0).long()

    def rows_of(codes, scales):  # [rows, heads, tokens, d] in fp32
        x = _blocks(codes)[0][page].view(codes.dtype).float() * scales[0][page][..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(rows, hk, width * pt, d)

    j = torch.arange(width * pt, device=dev)
    held = (j < lens[:, None])[:, None, :, None]
    k = rows_of(st["k"], st["k_scales"]).masked_fill(~held, 0.0)
    v = rows_of(st["v"], st["v_scales"]).masked_fill(~held, 0.0)
    qf = st["q"][at].float().view(rows, most, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(rows, hk, grp * most, d)
    s = (qf @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(rows, hk, grp, most, width * pt)
    before = (lens - n)[:, None, None]                                 # tokens that every node may see
    node = (j - before).clamp(0, 64 * st["mask"].shape[1] - 1).expand(rows, most, -1)
    bit = (st["mask"][at].gather(2, node >> 6) >> (node & 63)) & 1
    prefix = (j < before).expand(rows, most, -1)
    if c["window"]:
        prefix = prefix & (j > before + st["depth"].long()[at][:, :, None] - c["window"])
    sees = prefix | ((j >= before) & (j < lens[:, None, None]) & (bit > 0))
    s.masked_fill_(~sees[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.view(rows, hk, grp * most, width * pt) @ v).view(rows, hk, grp, most, d) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (total.log() + m).squeeze(-1)
    out = o.permute(0, 3, 1, 2, 4).reshape(rows, most, hk * grp, d)[real].to(st["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(rows, most, hk * grp)[real]}


def _encode(x, code):
    """fp32 quotients to codes: rounded to nearest even, clamped, NaN as 0."""
    x = torch.nan_to_num(x, nan=0.0, posinf=TOP[code], neginf=-TOP[code]).clamp(-TOP[code], TOP[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _plain_accept(st):
    c, dev = st["case"], st["table"].device
    pt, code = c["page"], c["code"]
    rows, width = st["path"].shape
    lens, starts = st["lens"].long(), st["starts"].long()
    base = lens - (starts[1:] - starts[:-1])
    kept = (st["path"] >= 0).sum(dim=1)
    # the blocks that get tokens, by row, and where their tokens come from: [rows, blocks, 16]
    nb = (width + 2 * BLOCK - 2) // BLOCK
    block = base[:, None] // BLOCK + torch.arange(nb, device=dev)
    gets = (block * BLOCK < (base + kept)[:, None]) & (kept[:, None] > 0)
    pos = block[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)
    k = pos - base[:, None, None]
    moved = st["path"].long().gather(1, k.clamp(0, width - 1).flatten(1)).view_as(k) + base[:, None, None]
    src = torch.where(k < 0, pos, moved)
    fresh = (k < kept[:, None, None])                                  # tokens that the block holds afterwards
    r, b = torch.nonzero(gets, as_tuple=True)
    src, fresh, block = src[r, b].clamp(min=0), fresh[r, b], block[r, b]
    page = st["table"][r, block * BLOCK // pt].long()
    sub = block % (pt // BLOCK)
    spage = st["table"][r[:, None], (src // pt).clamp(max=st["table"].shape[1] - 1)].clamp(min=0).long()
    ssub, slot = src % pt // BLOCK, src % BLOCK
    for pool, scales in ((st["k"], st["k_scales"]), (st["v"], st["v_scales"])):
        codes = _blocks(pool)
        la, hd = codes.shape[0], codes.shape[2]
        x = codes.permute(1, 3, 4, 0, 2, 5)[spage, ssub, slot].view(CODES[code])      # [blocks, 16, layers, heads, d]
        s0 = scales.permute(1, 3, 0, 2)[spage, ssub]                                   # [blocks, 16, layers, heads]
        f = fresh[:, :, None, None]
        s = torch.where(f, s0, torch.zeros_like(s0)).amax(dim=1)                       # [blocks, layers, heads]
        inv = (torch.ones_like(s) / s)[:, None, :, :, None]
        again = _encode(x.float() * s0[..., None] * inv, code).view(torch.int8)
        bits = torch.where((s0 == s[:, None])[..., None], x.view(torch.int8), again)
        dst = codes.permute(1, 3, 0, 2, 4, 5)                                          # [pages, blocks, layers, heads, 16, d]
        old = dst[page, sub]
        dst[page, sub] = torch.where(f[..., None], bits, old.permute(0, 3, 1, 2, 4)).permute(0, 2, 3, 1, 4)
        scales.permute(1, 3, 0, 2)[page, sub] = s
    # the rows' lists and counts
    new_lens = torch.where(starts[1:] > starts[:-1], base + kept, lens)
    listed_ = torch.arange(st["table"].shape[1], device=dev)
    before = listed_ < ((lens + pt - 1) // pt)[:, None]
    after = listed_ < ((new_lens + pt - 1) // pt)[:, None]
    gone = st["table"][before & ~after].long()
    refs = st["refs"].index_add(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    return {"table": torch.where(after, st["table"], torch.full_like(st["table"], -1)), "lens": new_lens.to(torch.int32),
            "refs": refs, **_pools(st)}


# ---- in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    """From the definitions, in 64 bits; what is a whole number has no such value."""
    c = case
    if c["op"] == "verify":
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "accept": _exact_accept, "logprobs": _exact_logprobs}[c["op"]](c, st)


def _exact_rope(c, st):
    freq = torch.tensor(_inv_freq(c), dtype=torch.float64, device="cuda")
    turn = torch.exp(1j * st["positions"].double()[:, None, None] * freq)
    rot = c["rotary"]
    outs = {}
    for n in ("q", "k"):
        parts = []
        for t0 in range(0, c["tokens"], 1024):
            x = st[n][t0:t0 + 1024].double()
            x = x / (x.square().mean(dim=2, keepdim=True) + EPS).sqrt() * st[n + "_weight"].double()
            r = x[..., :rot]
            z = r.unflatten(2, (rot // 2, 2)) if c["interleaved"] else r.unflatten(2, (2, rot // 2)).transpose(2, 3)
            z = torch.complex(z[..., 0], z[..., 1]) * turn[t0:t0 + 1024]
            z = torch.view_as_real(z)
            x[..., :rot] = (z if c["interleaved"] else z.transpose(2, 3)).flatten(2)
            parts.append(x)
        outs[n] = torch.cat(parts)
    return outs


def _exact_tree(c, st):
    hk, grp, d, pt = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    outs, lses, lo = [], [], 0
    for r, (length, n, (_, seen, depth)) in enumerate(zip(_lens(c), _nodes(c), _trees(c))):
        q = st["q"][lo:lo + n].double().view(n, hk, grp, d)
        lo += n
        before = length - n
        sees = torch.ones((n, length), dtype=torch.bool)
        for i in range(n):
            sees[i, before:] = torch.tensor([bool(seen[i] >> j & 1) for j in range(n)])
            if c["window"]:
                sees[i, :max(0, min(before, before + depth[i] - c["window"] + 1))] = False
        sees = sees.to(q.device)
        o = torch.zeros((n, hk, grp, d), dtype=torch.float64, device=q.device)
        e = torch.zeros((n, hk, grp), dtype=torch.float64, device=q.device)
        pages = st["table"][r, :_ceil(length, pt)].long()
        for h in range(hk):
            kv = [(x.view(torch.int8)[0, pages, h].view(x.dtype).double().view(-1, BLOCK, d) *
                   s[0, pages, h].double().reshape(-1, 1, 1)).view(-1, d)[:length]
                  for x, s in ((st["k"], st["k_scales"]), (st["v"], st["v_scales"]))]
            s = (q[:, h].reshape(n * grp, d) @ kv[0].T / math.sqrt(d)).view(n, grp, length).masked_fill(~sees[:, None], -math.inf)
            e[:, h] = torch.logsumexp(s, dim=2)
            o[:, h] = (torch.exp(s - e[:, h, :, None]).view(n * grp, length) @ kv[1]).view(n, grp, d)
        outs.append(o.view(n, hk * grp, d))
        lses.append(e.view(n, hk * grp))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_accept(c, st):
    """A block's scale is the largest of those of the tokens that it holds; codes are whole numbers."""
    out = {"table": None, "lens": None, "refs": None, "k": None, "v": None}
    pt = c["page"]
    table = st["table"].tolist()
    for name in ("k_scales", "v_scales"):
        old, new = st[name].double(), st[name].double().clone()
        for r, (length, n) in enumerate(zip(_lens(c), _nodes(c))):
            base, path = length - n, _path(c, r)
            end = base + len(path)
            for b in range(base // BLOCK, _ceil(end, BLOCK)):
                at = [p if p < base else base + path[p - base] for p in range(b * BLOCK, min(end, (b + 1) * BLOCK))]
                src = sorted({p // BLOCK for p in at})
                s = torch.stack([old[:, table[r][x * BLOCK // pt], :, x % (pt // BLOCK)] for x in src]).amax(dim=0)
                new[:, table[r][b * BLOCK // pt], :, b % (pt // BLOCK)] = s
        out[name] = new
    return out


def _exact_logprobs(c, st):
    outs = {"logprob": [], "entropy": [], "top_logprobs": []}
    step = max(1, 40_000_000 // c["vocab"])
    for r0 in range(0, c["rows"], step):
        x = st["logits"][r0:r0 + step].double()
        lp = torch.log_softmax(x, dim=1)
        outs["logprob"].append(lp.gather(1, st["tokens"][r0:r0 + step].long()[:, None])[:, 0])
        outs["entropy"].append(-(lp.exp() * lp).sum(dim=1))
        outs["top_logprobs"].append(torch.sort(lp, dim=1, descending=True).values[:, :c["top"]].clone())
    return {"rank": None, "top_ids": None, **{n: torch.cat(x) for n, x in outs.items()}}
