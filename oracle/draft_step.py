"""Float64 oracle of what a step with trees of drafts needs beside the cache (plain loops over NumPy
arrays): norm and rotation of heads, ancestor masks, attention under a mask, tree verification,
acceptance of a path, log probabilities.

Test infrastructure only, like the rest of this package.  Caches are those of ``kv_cache``.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .kv_cache import BLOCK, TOP, _f32, encode, fork, values
from .spec_verify import row_argmax

_PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


# ---- norm and rotation ---------------------------------------------------------------------------

def angle(position: int, inv_freq: float) -> float:
    """position * inv_freq modulo a turn, in radians, from exact fractions."""
    turns = Fraction(int(position)) * Fraction(float(inv_freq)) / (2 * _PI) % 1
    return float(turns * 2 * _PI)


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, norm=True, interleaved=False, amplitude=1.0):
    """(out, bound) of x [tokens, heads, D]; bound is what fp32 arithmetic may add up to before the
    output's rounding.

    A normalised value is off by at most (D / 2 + 12) 2^-24 of itself: a sum of D squares, its
    reciprocal root (2 units), two products.  Sines and cosines are off by 2^-25 half turns of
    argument, pi 2^-25, and 2 units: below 2^-21 together; the rotation adds two products and a sum."""
    x = np.asarray(x, np.float64)
    d = x.shape[2]
    y = x.copy()
    rel = 0.0
    if norm:
        y = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
        rel = (d / 2 + 12) * 2.0 ** -24
    out, bound = y.copy(), rel * np.abs(y)
    half = len(inv_freq)
    for t, p in enumerate(positions if half else []):
        for j, f in enumerate(inv_freq):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            th = angle(p, f)
            c, s = amplitude * np.cos(th), amplitude * np.sin(th)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, a] * s + y[t, :, b] * c
            e = abs(amplitude) * (np.abs(y[t, :, a]) + np.abs(y[t, :, b])) * (rel + 2.0 ** -21 + 2.0 ** -22)
            bound[t, :, a] = bound[t, :, b] = e
    return out, bound


# ---- trees -----------------------------------------------------------------------------------------

def tree_mask(parents, starts):
    """(ancestors and itself of each node, as a set of the row's indices; depth)."""
    parents = np.asarray(parents)
    seen, depth = [set() for _ in parents], np.zeros(len(parents), np.int64)
    for lo, hi in zip(starts[:-1], starts[1:]):
        for i in range(hi - lo):
            p = int(parents[lo + i])
            seen[lo + i] = {i} | (seen[lo + p] if 0 <= p < i else set())
            depth[lo + i] = len(seen[lo + i]) - 1
    return seen, depth


def mask_words(seen, words):
    """Sets of indices as int64 [tokens, words]."""
    out = np.zeros((len(seen), words), np.uint64)
    for i, s in enumerate(seen):
        for j in s:
            if j < 64 * words:
                out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def tree_verify(logits, drafted, parents, starts, max_path):
    """(accepted, next token, path, argmax)."""
    t = np.array([row_argmax(r) for r in logits], np.int64).reshape(-1)
    rows = len(starts) - 1
    accepted, nxt = np.zeros(rows, np.int64), np.full(rows, -1)
    path = np.full((rows, max_path), -1)
    for r in range(rows):
        lo, n = starts[r], starts[r + 1] - starts[r]
        at, k = 0, 0
        while n > 0 and k < max_path:
            path[r, k] = at
            k += 1
            nxt[r] = t[lo + at]
            kids = [i for i in range(at + 1, n) if parents[lo + i] == at and drafted[lo + i] == t[lo + at] and t[lo + at] >= 0]
            if not kids:
                break
            at = kids[0]
        accepted[r] = max(0, k - 1)
    return accepted, nxt, path, t


def masked_attend(cache, q, starts, seen, depth=None, layer=0, scale=None, window=0):
    """As ``kv_cache.attend`` under masks (``seen``: sets of the row's last tokens), with its bounds."""
    q = np.asarray(q, np.float64)
    tokens, hq, d = q.shape
    hk = cache["k"].shape[2]
    grp = hq // hk
    f = 1.0 / np.sqrt(d) if scale is None else float(scale)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lbound = np.full((tokens, hq), -np.inf), np.zeros((tokens, hq))
    for r in range(len(cache["lens"])):
        lo, hi = int(starts[r]), int(starts[r + 1])
        n, length = hi - lo, int(cache["lens"][r])
        before = length - n
        for h in range(hk):
            K, _ = values(cache, r, h, "k", layer)
            V, vs = values(cache, r, h, "v", layer)
            for i in range(n):
                at = [j for j in range(max(0, before))]
                if window:
                    p = before + max(0, min(int(depth[lo + i]), n - 1))
                    at = [j for j in at if j > p - window]
                at += [before + j for j in sorted(seen[lo + i]) if j < n and before + j >= 0]
                if not at:
                    continue
                k, v, sc = K[at], V[at], vs[at]
                for g in range(grp):
                    qv = q[lo + i, h * grp + g]
                    s = f * (k @ qv)
                    m = s.max()
                    w = np.exp(s - m)
                    z = w.sum()
                    e = 2.0 ** -20 * abs(f) * (np.abs(k) @ np.abs(qv) + np.abs(k).sum(axis=1) * np.abs(qv).max()).max() + 2.0 ** -20
                    e += 2.0 ** -22 * (np.abs(s).max() + 100)
                    out[lo + i, h * grp + g] = w @ v / z
                    bound[lo + i, h * grp + g] = (2.0 ** -11 + 4 * e) * (w @ np.abs(v)) / z + \
                        len(w) * 2.0 ** -25 * TOP[cache["fmt"]] * (w * sc).max() / z
                    lse[lo + i, h * grp + g] = m + np.log(z)
                    lbound[lo + i, h * grp + g] = 2 * e + 2.0 ** -20
    return out, lse, bound, lbound


def accept(cache, path, starts=None):
    """The new cache (its pools are shared, and changed in place)."""
    pt, fmt = cache["k"].shape[3], cache["fmt"]
    keep = []
    for r in range(len(cache["lens"])):
        length = int(cache["lens"][r])
        n = 1 if starts is None else int(starts[r + 1]) - int(starts[r])
        n = max(0, min(n, length))
        base, kept = length - n, []
        for p in path[r] if n else []:
            if p >= n or p <= (kept[-1] if kept else -1):
                break
            kept.append(int(p))
        keep.append(base + len(kept))
        place = lambda t: (int(cache["table"][r, t // pt]), t % pt // BLOCK, t % BLOCK)  # noqa: E731
        for b in range(base // BLOCK, -(-keep[r] // BLOCK)):
            here = range(b * BLOCK, min(keep[r], (b + 1) * BLOCK))
            src = [t if t < base else base + kept[t - base] for t in here]
            if not kept or all(s == t for s, t in zip(src, here)):
                continue
            page, sub, _ = place(b * BLOCK)
            for name in ("k", "v"):
                codes, scales = cache[name], cache[name + "s"]
                layers, _, heads = scales.shape[:3]
                for la in range(layers):
                    for h in range(heads):
                        got = []
                        for s in src:
                            pg, sb, at = place(s)
                            got.append((codes[la, pg, h, sb * BLOCK + at].copy(), float(scales[la, pg, h, sb])))
                        top = max(s for _, s in got)
                        inv = float(_f32(1.0 / top))
                        for t, (c, s) in zip(here, got):
                            codes[la, page, h, sub * BLOCK + t % BLOCK] = c if s == top else encode(_f32(_f32(c * s) * inv), fmt)
                        scales[la, page, h, sub] = top
    return fork(cache, list(range(len(keep))), keep)


# ---- log probabilities -------------------------------------------------------------------------------

def order(row):
    """Indices of a row's entries, the largest first, ties by index; NaN counts as -infinity."""
    r = np.where(np.isnan(row), -np.inf, np.asarray(row, np.float64))
    return r, np.lexsort((np.arange(len(r)), -r))


def token_logprobs(logits, tokens, top, threads=256):
    """dict of logprob, entropy, rank, top_ids, top_logprobs, and bounds of the three that are sums.

    Sums: each of a thread's terms is off by 2^-22 (the exponential) and |t| 2^-23 (its argument), and
    adding V / threads of them by 2^-24 each; l and s have one sign, so these are relative."""
    rows, v = logits.shape
    out = {"logprob": np.full(rows, -np.inf), "entropy": np.zeros(rows), "rank": np.full(rows, -1),
           "top_ids": np.full((rows, top), -1), "top_logprobs": np.full((rows, top), -np.inf)}
    bound = {"logprob": np.zeros(rows), "entropy": np.zeros(rows), "top_logprobs": np.zeros((rows, top))}
    for i in range(rows):
        r, by = order(logits[i])
        tok = int(tokens[i])
        if 0 <= tok < v:
            out["rank"][i] = int(np.flatnonzero(by == tok)[0])
        listed = [j for j in by[:top] if r[j] > -np.inf]
        out["top_ids"][i, :len(listed)] = listed
        m = r.max()
        if m == -np.inf:
            continue
        if m == np.inf:
            out["entropy"][i] = out["logprob"][i] = np.nan
            out["top_logprobs"][i, :len(listed)] = np.nan
            if not 0 <= tok < v:
                out["logprob"][i] = -np.inf
            continue
        d = (r - m)[r > -np.inf]
        e = np.exp(d)
        l, s = e.sum(), (e * -d).sum()
        out["entropy"][i] = np.log(l) + s / l
        rel = 2.0 ** -21 + (v / threads + 40) * 2.0 ** -24 + 2.0 ** -22 * s / l
        bound["entropy"][i] = rel * (1 + 2 * s / l) + 2.0 ** -21 * (np.log(l) + s / l) + 2.0 ** -22 * (e * d * d).sum() / l
        at = lambda x: (x - m - np.log(l), abs(x - m) * 2.0 ** -23 + rel + 2.0 ** -22 * np.log(l) + 2.0 ** -24 * abs(x - m - np.log(l)))  # noqa: E731
        if 0 <= tok < v and r[tok] > -np.inf:
            out["logprob"][i], bound["logprob"][i] = at(r[tok])
        for k, j in enumerate(listed):
            out["top_logprobs"][i, k], bound["top_logprobs"][i, k] = at(r[j])
    return out, bound
