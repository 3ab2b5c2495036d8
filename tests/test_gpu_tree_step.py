"""The operators of a step with trees of drafts together, as a program runs them: against the oracle stage
by stage, captured in graphs and replayed, on a stream of its own, and in the example's decoding loop."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest

import bit_quantized_decode_unpack_gb300 as bqd
import oracle.draft_step as od
import oracle.kv_cache as okv
from _kv_util import F16_HALF, assert_same, i32, random_cache, starts_of, to_library
from test_gpu_draft_trees import _parents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "tree_decode", Path(__file__).resolve().parent.parent / "examples" / "tree_decode.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Step:
    """One layer's step over static inputs; every call of run() computes the whole of it."""

    def __init__(self, seed, lens, news, fmt="int8", d=64, hk=2, grp=3, vocab=1003, long=0):
        import torch
        rng = np.random.default_rng(seed)
        self.news, self.starts, self.d, self.hk, self.hq = news, starts_of(news), d, hk, hk * grp
        self.c = random_cache(rng, lens, heads=hk, d=d, pt=16, fmt=fmt, spare=sum(-(-n // 16) + 1 for n in news),
                              row_pages=long or -(-(max(lens) + max(news)) // 16))
        t = sum(news)
        self.qkv = torch.from_numpy(rng.standard_normal((t, self.hq + 2 * hk, d)).astype(np.float32)).cuda().half()
        self.freq = [1000.0 ** (-2 * j / d) for j in range(d // 2)]
        self.w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda().half() for _ in range(2)]
        self.rope = bqd.QKNormRope(d, self.freq, q_weight=self.w[0], k_weight=self.w[1])
        self.parents = _parents(rng, news)
        self.par, self.st, self.counts = i32(self.parents), i32(self.starts), i32(news)
        x = rng.standard_normal((t, vocab)).astype(np.float32)
        self.drafted = rng.integers(0, vocab, t)
        for lo, hi in zip(self.starts[:-1], self.starts[1:]):
            for i in range(1, hi - lo):
                if rng.random() < 0.7:
                    x[lo + self.parents[lo + i], self.drafted[lo + i]] = 8 + rng.random()
        self.logits, self.nodes = torch.from_numpy(x).cuda(), i32(self.drafted)
        self.cache = to_library(self.c)
        self.kept = self.cache.fork(i32(range(len(lens))))  # the state that a run leaves
        self.first = {n: getattr(self.cache, n).clone() for n in ("k", "v", "k_scales", "v_scales", "table", "lens", "refs")}

    def reset(self):
        import torch
        for n, t in self.first.items():
            getattr(self.cache, n).view(torch.uint8).copy_(t.view(torch.uint8))

    def run(self):
        hq, hk, most = self.hq, self.hk, max(self.news)
        base, status = self.cache.reserve(self.counts)
        mask, depth, positions = bqd.tree_mask(self.par, self.st, base=base)
        q, k = self.rope(self.qkv[:, :hq], self.qkv[:, hq:hq + hk], positions)
        self.cache.append(k, self.qkv[:, hq + hk:], base, self.st, max_new=most)
        out, lse = self.cache.attend(q, self.st, mask=mask, depth=depth, max_new=most)
        accepted, token, path = bqd.spec_tree_verify(self.logits, self.nodes, self.par, self.st, max_path=most)
        said = bqd.token_logprobs(self.logits, self.nodes, 5)
        self.cache.accept(path, self.st, out=self.kept)
        return {"base": base, "status": status, "mask": mask, "positions": positions, "q": q, "k": k, "out": out, "lse": lse,
                "accepted": accepted, "token": token, "path": path, **said._asdict(), "lens": self.kept.lens, "table": self.kept.table,
                "refs": self.kept.refs, "k_scales": self.cache.k_scales, "v_scales": self.cache.v_scales}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_step_stage_by_stage(fmt):
    s = Step(1, [40, 0, 33, 200], [26, 5, 1, 64], fmt)
    r = s.run()
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    base, status = okv.reserve(s.c, s.news)
    assert status == [0, 0] and r["base"].tolist() == base.tolist()
    seen, depth = od.tree_mask(s.parents, s.starts)
    pos = np.repeat(base, s.news) + depth
    assert r["positions"].tolist() == pos.tolist()
    hq, hk = s.hq, s.hk
    for name, x, w in (("q", s.qkv[:, :hq], s.w[0]), ("k", s.qkv[:, hq:hq + hk], s.w[1])):
        want, bound = od.norm_rope(n(x), pos, s.freq, n(w))
        assert np.all(np.abs(n(r[name]) - want) <= bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)
    okv.append(s.c, n(r["k"]), n(s.qkv[:, hq + hk:]), base, s.starts)  # (what the library rounded goes in)
    want, _, bound, _ = od.masked_attend(s.c, n(r["q"]), s.starts, seen)
    assert np.all(np.abs(n(r["out"]) - want) <= bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)
    accepted, token, path, _ = od.tree_verify(s.logits.cpu().numpy(), s.drafted, s.parents, s.starts, 64)
    assert r["accepted"].tolist() == accepted.tolist() and r["token"].tolist() == token.tolist() and accepted.max() >= 2
    assert_same(s.kept, od.accept(s.c, path, s.starts))
    want, _ = od.token_logprobs(s.logits.cpu().numpy(), s.drafted, 5)
    assert (r["top_ids"].cpu().numpy() == want["top_ids"]).all() and (r["rank"].cpu().numpy() == want["rank"]).all()


def _equal(a, b):
    import torch
    for name in a:
        assert torch.equal(a[name].contiguous().view(torch.uint8), b[name].contiguous().view(torch.uint8)), name


@pytest.mark.parametrize("big", [False, True])
def test_captured_and_replayed(big):
    """Two graphs of two states, replayed in turn and with other inputs, give what eager calls give."""
    import torch
    shapes = dict(d=128, grp=6, hk=4, long=9000) if big else {}  # (planned long: the tile kernel)
    steps = [Step(2, [600, 90] if big else [60, 9], [64, 30], **shapes), Step(3, [17, 300], [33, 64], **shapes)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for s in steps:
        assert (s.cache.attend_workspace(s.hq, sum(s.news), max(s.news), masked=True) > 1 << 24) == big
        s.run()
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(s.run())
        graphs.append(g)
    for turn in range(3):
        for s in steps:
            s.reset()
            if turn:
                s.qkv.mul_(-0.5), s.logits.copy_(s.logits.flip(0))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, got in zip(steps, outs):
            got = {k: v.clone() for k, v in got.items()}
            s.reset()
            _equal(s.run(), got)


def test_on_a_stream_of_its_own():
    import torch
    s, side = Step(4, [70, 33], [26, 40]), torch.cuda.Stream()
    want = {k: v.clone() for k, v in s.run().items()}
    torch.cuda.synchronize()
    s.reset()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.run()
    side.synchronize()
    _equal(want, got)
    # and by the argument
    pos = torch.zeros(len(s.parents), dtype=torch.int32, device="cuda")
    a = bqd.spec_tree_verify(s.logits, s.nodes, s.par, s.st, max_path=9, stream=side)
    b = bqd.token_logprobs(s.logits, s.nodes, 3, stream=side)
    m = bqd.tree_mask(s.par, s.st, stream=side)
    q, _ = s.rope(s.qkv, None, pos, stream=side)
    side.synchronize()
    assert a[0].tolist() == bqd.spec_tree_verify(s.logits, s.nodes, s.par, s.st, max_path=9)[0].tolist()
    assert b.rank.tolist() == bqd.token_logprobs(s.logits, s.nodes, 3).rank.tolist()
    assert m[1].tolist() == bqd.tree_mask(s.par, s.st)[1].tolist() and torch.equal(q, s.rope(s.qkv, None, pos)[0])


# ---- waits that run out --------------------------------------------------------------------------

@pytest.mark.parametrize("d,grp,lens,news", [(128, 6, [900, 400], [64, 40]), (128, 6, [2500, 900], [20, 8]), (64, 6, [700], [64]),
                                             (256, 6, [900, 130], [64, 3])])
def test_waits_that_run_out_anywhere(d, grp, lens, news):
    """In the tile kernel of masked calls: a CTA lets what it issued finish; a call whose waits all came through has
    the right answer, another is reported by bqd_device_status, and the calls after it are clean."""
    import torch
    from _kv_util import rounded
    rng = np.random.default_rng(d + len(lens))
    c = random_cache(rng, lens, heads=2, d=d, pt=64, row_pages=60000)
    q, qd = rounded(rng.standard_normal((sum(news), 2 * grp, d)), "float16")
    seen, _ = od.tree_mask(_parents(rng, news), starts_of(news))
    lib, qq, starts = to_library(c), q.cuda(), i32(starts_of(news))
    mask = torch.from_numpy(od.mask_words(seen, 1)).cuda()
    assert lib.attend_workspace(2 * grp, sum(news), max(news), masked=True) > 1 << 24
    want, _, bound, _ = od.masked_attend(c, qd, starts_of(news), seen)
    tol = bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25

    def call():
        out, _ = lib.attend(qq, starts, mask=mask, max_new=max(news))
        status = bqd.device_status()
        return status, np.all(np.abs(out.double().cpu().numpy() - want) <= tol)

    assert call() == (0, True)
    statuses = []
    for limit in (1, 300, 1000, 2000, 4000, 7000, 12000, 19000, 25000, 50000, 100000):
        for _ in range(3):
            bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, limit)
            try:
                status, right = call()
            finally:
                bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, 0)
            assert status == 7 or (status == 0 and right)
            statuses.append(status)
            assert call() == (0, True)
    assert statuses[0] == 7


# ---- the example ----------------------------------------------------------------------------------

def _prompts():
    import torch
    gen = torch.Generator().manual_seed(5)
    return [torch.randint(0, 1000, (n,), generator=gen).tolist() for n in (2, 90, 31, 1)]


@pytest.mark.parametrize("kw", [dict(page_tokens=16), dict(page_tokens=64, format="e4m3")])
def test_trees_change_nothing_but_the_speed(example, kw):
    model, prompts = example.Decoder(), _prompts()
    plain, lp, _, none, steps = example.generate(model, prompts, 12, draft=lambda r, s: ([], []), **kw)
    assert none == 0 and steps == 12 and all(len(s) == len(p) + 12 for s, p in zip(plain, prompts))

    def oracle(row, seq):
        """What the model says next, with a wrong branch beside each node of it."""
        say = (plain[row][len(seq):] + [0, 0, 0])[:3]
        return [0, 0, 2, 2, 4, 4], [(say[0] + 1) % 1000, say[0], say[1], (say[1] + 7) % 1000, 5, say[2]][:6]

    fast, lp2, cache, hits, quick = example.generate(model, prompts, 12, draft=oracle, **kw)
    # a block's scale may remember a rejected token, and other batch shapes round differently: the first tokens agree,
    # and most drafts are taken
    for a, b, p, x, y in zip(plain, fast, prompts, lp, lp2):
        assert a[:len(p) + 1] == b[:len(p) + 1] and abs(x[0] - y[0]) < 0.1
    assert hits >= 12 and quick < steps
    assert cache.lens.tolist() == [len(s) - 1 for s in fast]
    assert int((cache.refs > 0).sum()) == sum(-(-(len(s) - 1) // kw["page_tokens"]) for s in fast)


def test_main_runs(example, capsys):
    example.main()
    assert "drafts accepted" in capsys.readouterr().out
