"""Greedy speculative decoding of a few sequences with low-bit linear layers and the 8-bit KV cache.

A toy decoder (random weights: what it says means nothing, what it runs is the real path):
every layer's q, k, v and o projections are ``QuantLinear`` layers, keys and values go into a
``KVCache``, and the target's tokens come from ``spec_decode_verify``.  Each step

    reserve  room for the step's tokens (the last accepted one and its drafts), in every layer at once
    append   per layer: the new keys and values, quantised into the pages
    attend   per layer: every query over its own sequence's cache
    verify   the drafts against the target's logits
    truncate the rejected tokens leave the cache, their pages are free again

and at the end the surviving sequences are forked and the pool is compacted.

    python examples/cached_decode.py
"""
import sys
from pathlib import Path

import torch

if __name__ == "__main__":
    sys.path.insert(0, str(Path(__file__).resolve().parent.parent))

import bit_quantized_decode_unpack_gb300 as bqd
from bit_quantized_decode_unpack_gb300.quant_linear import QuantLinear


def random_linear(inp, out, fmt, gen):
    """A QuantLinear of random codes whose outputs keep their inputs' magnitude."""
    top = {"affine2": 4, "t5": 3}[fmt]
    codes = torch.randint(0, top, (out, inp), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.full((out, inp // 64), 1.2 / inp ** 0.5, dtype=torch.float16, device="cuda")
    return QuantLinear.from_packed(bqd.pack(codes, fmt, 64), scales, None, fmt, 64)


class Layer(torch.nn.Module):
    """One attention block; queries and keys are normalised per head."""

    def __init__(self, dim, heads, kv_heads, head_dim, gen):
        super().__init__()
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.q = random_linear(dim, heads * head_dim, "affine2", gen)
        self.k = random_linear(dim, kv_heads * head_dim, "affine2", gen)
        self.v = random_linear(dim, kv_heads * head_dim, "t5", gen)
        self.o = random_linear(heads * head_dim, dim, "t5", gen)

    def forward(self, x, cache, layer, base, starts, max_new, max_len):
        norm = lambda t: torch.nn.functional.rms_norm(t, (self.head_dim,))
        q = norm(self.q(x).view(-1, self.heads, self.head_dim))
        k = norm(self.k(x).view(-1, self.kv_heads, self.head_dim))
        v = self.v(x).view(-1, self.kv_heads, self.head_dim)
        cache.append(k, v, base, starts, layer=layer, max_new=max_new)
        out, _ = cache.attend(q, starts, layer=layer, max_new=max_new, max_len=max_len)
        return x + self.o(out.view(x.shape[0], -1))


class Decoder(torch.nn.Module):
    def __init__(self, layers=2, dim=512, heads=8, kv_heads=2, head_dim=64, vocab=1000, seed=0):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((vocab, dim), generator=gen, device="cuda").half()
        self.layers = torch.nn.ModuleList(Layer(dim, heads, kv_heads, head_dim, gen) for _ in range(layers))
        self.shape = (layers, kv_heads, head_dim)

    def new_cache(self, rows, row_pages, pages, **kw):
        layers, kv_heads, head_dim = self.shape
        return bqd.KVCache.empty(layers, pages, kv_heads, head_dim, rows, row_pages, **kw)

    def forward(self, tokens, counts, cache, max_len):
        """Logits of every token of a ragged batch: row r's next counts[r] tokens, in row order."""
        starts = torch.zeros(len(counts) + 1, dtype=torch.int32)
        starts[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
        starts = starts.cuda()
        base, status = cache.reserve(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        x = self.embed[tokens]
        for i, layer in enumerate(self.layers):
            x = layer(x, cache, i, base, starts, max(counts), max_len)
        if status.any():
            raise RuntimeError(f"the cache is full: {status.tolist()} (pages missing, rows too long)")
        return torch.nn.functional.rms_norm(x, (x.shape[1],)).float() @ self.embed.float().T


def generate(model, prompts, new_tokens, drafts=4, draft=None, **cache_kw):
    """Continues each prompt (a list of token ids) greedily by at least new_tokens tokens.

    ``draft(row, sequence, n)`` guesses n tokens (default: repeats the last one); every token taken is
    the model's own choice after those before it.  (A rejected guess leaves the cache, but may have
    raised its block's scale: two runs with other guesses agree as far as 8 bits do.)  A row leaves
    the batch with the step that reaches its goal.  Returns (sequences, cache, accepted drafts)."""
    draft = draft or (lambda row, seq, n: [seq[-1]] * n)
    rows, longest = len(prompts), max(map(len, prompts)) + new_tokens + drafts + 1
    pt = cache_kw.get("page_tokens", 64)
    cache = model.new_cache(rows, -(-longest // pt), rows * -(-longest // pt) + 1, **cache_kw)
    seqs = [list(p) for p in prompts]
    # the prompts, but for their last tokens: each step starts with the newest token of a sequence
    heads = [p[:-1] for p in prompts]
    if any(heads):
        model(torch.tensor(sum(heads, []), device="cuda"), [len(h) for h in heads], cache, longest)
    goal = [len(p) + new_tokens for p in prompts]
    hits = 0
    while live := [r for r in range(rows) if len(seqs[r]) < goal[r]]:
        guesses = [draft(r, seqs[r], drafts) for r in live]
        tokens = torch.tensor([[seqs[r][-1]] + g for r, g in zip(live, guesses)], device="cuda")
        counts = [1 + drafts if r in live else 0 for r in range(rows)]
        logits = model(tokens.view(-1), counts, cache, longest)
        accepted, following = bqd.spec_decode_verify(
            logits.view(len(live), 1 + drafts, -1), tokens[:, 1:].to(torch.int32).contiguous())
        for r, g, n, token in zip(live, guesses, accepted.tolist(), following.tolist()):
            seqs[r] += g[:n] + [token]
            hits += n
        # the cache holds every token but the newest of each sequence
        cache = cache.truncate(torch.tensor([len(s) - 1 for s in seqs], dtype=torch.int32, device="cuda"))
    return seqs, cache, hits


def main():
    model = Decoder()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (n,), generator=gen).tolist() for n in (7, 150, 33)]
    seqs, cache, hits = generate(model, prompts, 24, page_tokens=16)
    print(f"{sum(map(len, seqs))} tokens in the cache's rows, {hits} drafts accepted")
    for s, p in zip(seqs, prompts):
        print(" ", s[len(p):][:12], "...")
    # two beams of the first sequence, the second one freed, the pool made dense
    beams = cache.fork(torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda"))
    base, _ = beams.reserve()
    beams, moved = beams.compact()
    print(f"beams of {base.tolist()} tokens, {int((beams.refs > 0).sum())} pages live, {moved.item()} moved")


if __name__ == "__main__":
    main()
