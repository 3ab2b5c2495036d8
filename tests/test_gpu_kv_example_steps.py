"""The example's decoding loop where its rows end at different steps, and what its cache holds after
any number of them: the next logits are those of a fresh cache that was filled with the same tokens,
as far as 8 bits allow.

Tolerances, relative to the norm of the logits.  One rounding of every stored value (half a step of a
block's scale) moves them by less than 0.03 (test_gpu_kv_example.py).  A block whose scale grew g
times has been rounded 1 + g times, independent errors that add in squares, in steps up to 1.3 times
as wide (the largest of 1024 or 2048 values).  g <= 4 for drafts (four rejected tokens can each raise
it): 0.03 sqrt(5) 1.3 for that cache and 0.03 for the fresh one, 0.12.  g <= 2 for a prompt cut twice
inside a block, with no value that is not there in the end: 0.03 sqrt(3) + 0.03, 0.09.  Cut at
blocks' ends: 0.06."""
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


def _prompts(*lengths):
    import torch
    gen = torch.Generator().manual_seed(5)
    return [torch.randint(0, 1000, (n,), generator=gen).tolist() for n in lengths]


def _next_logits(model, seqs, cache, longest):
    import torch
    return model(torch.tensor([s[-1] for s in seqs], device="cuda"), [1] * len(seqs), cache, longest)


def _fresh(model, seqs, page_tokens):
    import torch
    longest = max(map(len, seqs)) + 1
    cache = model.new_cache(len(seqs), -(-longest // page_tokens), len(seqs) * -(-longest // page_tokens),
                            page_tokens=page_tokens)
    model(torch.tensor(sum((s[:-1] for s in seqs), []), device="cuda"), [len(s) - 1 for s in seqs], cache, longest)
    return _next_logits(model, seqs, cache, longest)


@pytest.mark.parametrize("page_tokens", [16, 64])
@pytest.mark.parametrize("lengths,new,drafts", [((46, 10), 11, 4), ((47, 3), 12, 4), ((58, 1, 20), 5, 8)])
def test_a_row_that_ends_early_and_past_its_goal(example, page_tokens, lengths, new, drafts):
    """Row 0 takes all of its drafts and ends several tokens past its goal, the others take none."""
    model, prompts = example.Decoder(), _prompts(*lengths)
    plain, _, _ = example.generate(model, prompts, new + drafts, drafts=1, page_tokens=64)

    def draft(row, seq, n):
        said = (plain[row][len(seq):] + [0] * n)[:n]
        return said if row == 0 else [(t + 1) % 1000 for t in said]

    seqs, cache, hits = example.generate(model, prompts, new, drafts=drafts, draft=draft, page_tokens=page_tokens)
    assert all(len(p) + new <= len(s) <= len(p) + new + drafts for s, p in zip(seqs, prompts))
    assert all(s[:len(p)] == p for s, p in zip(seqs, prompts))
    assert cache.lens.tolist() == [len(s) - 1 for s in seqs]
    assert int((cache.refs > 0).sum()) == sum(-(-(len(s) - 1) // page_tokens) for s in seqs)


@pytest.mark.parametrize("lengths", [(1,), (1, 1, 1), (1, 30)])
def test_prompts_of_one_token(example, lengths):
    model, prompts = example.Decoder(), _prompts(*lengths)
    seqs, cache, _ = example.generate(model, prompts, 6, drafts=2, page_tokens=16)
    assert all(len(s) >= len(p) + 6 for s, p in zip(seqs, prompts))
    assert cache.lens.tolist() == [len(s) - 1 for s in seqs]


@pytest.mark.parametrize("new", [1, 2, 9, 24])
def test_after_rejected_drafts_the_cache_holds_the_same_tokens(example, new):
    import torch
    model, prompts = example.Decoder(), _prompts(2, 90, 31, 17)
    gen = torch.Generator().manual_seed(new)
    wrong = lambda row, seq, n: torch.randint(0, 1000, (n,), generator=gen).tolist()
    seqs, cache, _ = example.generate(model, prompts, new, drafts=4, draft=wrong, page_tokens=16)
    got = _next_logits(model, seqs, cache, 128)
    want = _fresh(model, seqs, 16)
    assert (got - want).norm() / want.norm() < 0.12


@pytest.mark.parametrize("cuts,most", [((5, 11), 0.09), ((16, 64), 0.06), ((1, 70), 0.09)])
def test_a_prompt_in_chunks(example, cuts, most):
    import torch
    model, prompts = example.Decoder(), _prompts(90, 81)
    cache = model.new_cache(2, 8, 16, page_tokens=16)
    for lo, hi in zip((0,) + cuts, cuts + (None,)):
        part = [p[:-1][lo:hi] for p in prompts]
        model(torch.tensor(sum(part, []), device="cuda"), [len(p) for p in part], cache, 128)
    got, want = _next_logits(model, prompts, cache, 128), _fresh(model, prompts, 16)
    assert (got - want).norm() / want.norm() < most
