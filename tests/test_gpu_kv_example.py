"""The example's decoding path: the tokens do not depend on the drafts, on the split of a prompt
into chunks, or on the cache's page size beyond what its rounding allows, and they agree with a
model that keeps no cache."""
import importlib.util
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "cached_decode", Path(__file__).resolve().parent.parent / "examples" / "cached_decode.py")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _prompts():
    import torch
    gen = torch.Generator().manual_seed(5)
    return [torch.randint(0, 1000, (n,), generator=gen).tolist() for n in (2, 90, 31, 17)]


@pytest.mark.parametrize("kw", [dict(page_tokens=16), dict(page_tokens=64, format="e4m3")])
def test_drafts_change_nothing_but_the_speed(example, kw):
    model, prompts = example.Decoder(), _prompts()
    plain, _, _ = example.generate(model, prompts, 12, drafts=1, **kw)
    # drafts that are what the model says: all accepted while they last
    oracle = lambda row, seq, n: (plain[row][len(seq):] + [0] * n)[:n]
    fast, cache, hits = example.generate(model, prompts, 12, drafts=4, draft=oracle, **kw)
    # a block's scale may remember a rejected token, and other batch shapes round differently: the first
    # tokens agree, and most drafts are taken
    for a, b, p in zip(plain, fast, prompts):
        assert a[:len(p) + 1] == b[:len(p) + 1]
    assert hits >= 12
    assert cache.lens.tolist() == [len(s) - 1 for s in fast]
    assert int((cache.refs > 0).sum()) == sum(-(-(len(s) - 1) // kw["page_tokens"]) for s in fast)


def test_logits_agree_with_a_model_without_a_cache(example):
    """fp16 attention over unquantised keys and values, the same layers otherwise.  8 bits a value
    (half a step of 1/127 of a block's largest) leave the logits within a few percent."""
    import torch
    model, prompts = example.Decoder(), _prompts()
    counts = [len(p) for p in prompts]
    tokens = torch.tensor(sum(prompts, []), device="cuda")
    cache = model.new_cache(4, 8, 40, page_tokens=16)
    got = model(tokens, counts, cache, 128)
    x = model.embed[tokens]
    norm = lambda t: torch.nn.functional.rms_norm(t, (64,))
    for layer in model.layers:
        q, k = norm(layer.q(x).view(-1, 8, 64)).float(), norm(layer.k(x).view(-1, 2, 64)).float()
        v, outs, at = layer.v(x).view(-1, 2, 64).float(), [], 0
        for n in counts:
            s = torch.einsum("ihd,jhd->hij", q[at:at + n], k[at:at + n].repeat_interleave(4, dim=1)) / 8
            s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
            outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v[at:at + n].repeat_interleave(4, dim=1)))
            at += n
        x = x + layer.o(torch.cat(outs).half().view(len(tokens), -1))
    want = torch.nn.functional.rms_norm(x, (512,)).float() @ model.embed.float().T
    assert (got - want).norm() / want.norm() < 0.03


def test_main_runs(example, capsys):
    example.main()
    assert "pages live" in capsys.readouterr().out


def test_a_full_cache_is_reported(example):
    import torch
    model = example.Decoder()
    cache = model.new_cache(1, 2, 1, page_tokens=16)
    with pytest.raises(RuntimeError, match="full"):
        model(torch.arange(20, device="cuda"), [20], cache, 32)
