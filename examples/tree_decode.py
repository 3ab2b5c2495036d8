"""Greedy speculative decoding with trees of drafts: low-bit linear layers, rotated queries and keys, the
8-bit KV cache.

A toy decoder (random weights: what it says means nothing, what it runs is the real path).  A step's
tokens are, for each sequence, the last token that the target chose (node 0) and drafts that hang below
it or below each other.  Each step

    reserve   room for the nodes, in every layer at once
    tree_mask which nodes each one sees, its depth and position
    rope      per layer: norm and rotation of queries and keys (QKNormRope)
    append    per layer: the new keys and values, quantised into the pages
    attend    per layer: every node over its sequence's cache, its own branch and nothing beside it
    verify    the path that the target's logits agree with (spec_tree_verify)
    accept    the path's tokens stay in the cache, the other branches leave it
    logprobs  what the chosen tokens' log probabilities are, with alternatives (token_logprobs)

    python examples/tree_decode.py
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
    """One attention block."""

    def __init__(self, dim, heads, kv_heads, head_dim, gen):
        super().__init__()
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.q = random_linear(dim, heads * head_dim, "affine2", gen)
        self.k = random_linear(dim, kv_heads * head_dim, "affine2", gen)
        self.v = random_linear(dim, kv_heads * head_dim, "t5", gen)
        self.o = random_linear(heads * head_dim, dim, "t5", gen)
        weights = [(1 + 0.2 * torch.randn(head_dim, generator=gen, device="cuda")).half() for _ in range(2)]
        self.rope = bqd.QKNormRope(head_dim, [10000.0 ** (-2 * j / head_dim) for j in range(head_dim // 2)],
                                   q_weight=weights[0], k_weight=weights[1])

    def forward(self, x, cache, layer, step):
        q, k = self.q(x).view(-1, self.heads, self.head_dim), self.k(x).view(-1, self.kv_heads, self.head_dim)
        q, k = self.rope(q, k, step["positions"], q_out=q, k_out=k)
        v = self.v(x).view(-1, self.kv_heads, self.head_dim)
        cache.append(k, v, step["base"], step["starts"], layer=layer, max_new=step["max_new"])
        out, _ = cache.attend(q, step["starts"], layer=layer, max_new=step["max_new"], max_len=step["max_len"],
                              mask=step["mask"], depth=step["depth"])
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

    def forward(self, tokens, counts, cache, max_len, parents=None):
        """(logits of every token of a ragged batch, starts): row r's next counts[r] tokens, in row order, one
        after the other, or the nodes of a tree where ``parents`` (the row's own indices) are given."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        starts = torch.zeros(len(counts) + 1, dtype=torch.int32)
        starts[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
        starts = starts.cuda()
        base, status = cache.reserve(i32(counts))
        step = {"base": base, "starts": starts, "max_new": max(counts), "max_len": max_len, "mask": None, "depth": None}
        tree = parents is not None
        words = -(-max(counts) // 64) if tree else 1
        chain = [i - 1 for n in counts for i in range(n)]
        mask, depth, step["positions"] = bqd.tree_mask(i32(parents if tree else chain), starts, words=words, base=base)
        if tree:
            step["mask"], step["depth"] = mask, depth
        x = self.embed[tokens]
        for i, layer in enumerate(self.layers):
            x = layer(x, cache, i, step)
        if status.any():
            raise RuntimeError(f"the cache is full: {status.tolist()} (pages missing, rows too long)")
        return torch.nn.functional.rms_norm(x, (x.shape[1],)).float() @ self.embed.float().T, starts


def guess(row, seq):
    """Drafts below the last token: (parents, tokens) of a small tree.  Here: the last token again, twice in
    a row, and the one before it."""
    return [0, 1, 0], [seq[-1], seq[-1], seq[-2] if len(seq) > 1 else 0]


def generate(model, prompts, new_tokens, draft=guess, depth=8, **cache_kw):
    """Continues each prompt (a list of token ids) greedily by at least new_tokens tokens.

    ``draft(row, sequence)`` returns (parents, tokens) of the drafted nodes 1, 2, ... below node 0, the
    sequence's last token; every token taken is the model's own choice after those before it.  Paths of
    ``depth`` nodes at most are taken in a step, and a row leaves the batch with the step that reaches its
    goal.  Returns (sequences, log probabilities of the new tokens, cache, accepted drafts, steps)."""
    rows, goal = len(prompts), [len(p) + new_tokens for p in prompts]
    pt, longest = cache_kw.get("page_tokens", 64), max(goal) + 64
    cache = model.new_cache(rows, -(-longest // pt), rows * -(-longest // pt) + 1, **cache_kw)
    seqs, logprobs = [list(p) for p in prompts], [[] for _ in prompts]
    heads = [p[:-1] for p in prompts]  # each step starts with the newest token of a sequence
    if any(heads):
        model(torch.tensor(sum(heads, []), device="cuda"), [len(h) for h in heads], cache, longest)
    hits = steps = 0
    while live := [r for r in range(rows) if len(seqs[r]) < goal[r]]:
        parents, nodes, counts = [], [], [0] * rows
        for r in live:
            p, t = draft(r, seqs[r])
            parents += [-1] + list(p)
            nodes += [seqs[r][-1]] + list(t)
            counts[r] = 1 + len(t)
        tokens = torch.tensor(nodes, dtype=torch.int32, device="cuda")
        logits, starts = model(tokens.long(), counts, cache, longest, parents)
        par = torch.tensor(parents, dtype=torch.int32, device="cuda")
        best = torch.empty_like(tokens)
        accepted, _, path = bqd.spec_tree_verify(logits, tokens, par, starts, max_path=depth, argmax_out=best)
        said = bqd.token_logprobs(logits, best, top=5)
        cache = cache.accept(path, starts)
        steps += 1
        lo = starts.tolist()
        for r in live:
            for node in path[r, :accepted[r] + 1].tolist():
                seqs[r].append(best[lo[r] + node].item())
                logprobs[r].append(said.logprob[lo[r] + node].item())
            hits += accepted[r].item()
    return seqs, logprobs, cache, hits, steps


def main():
    model = Decoder()
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 1000, (n,), generator=gen).tolist() for n in (7, 150, 33)]
    seqs, logprobs, cache, hits, steps = generate(model, prompts, 24, page_tokens=16)
    print(f"{sum(cache.lens.tolist())} tokens in the cache after {steps} steps, {hits} drafts accepted")
    for s, p, lp in zip(seqs, prompts, logprobs):
        print(" ", s[len(p):][:10], "mean log probability", round(sum(lp) / len(lp), 3))


if __name__ == "__main__":
    main()
