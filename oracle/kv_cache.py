"""Float64 oracle of the paged 8-bit KV cache (plain loops over NumPy arrays).

Test infrastructure only, like the rest of this package: it shares no code with
the CUDA library.  A cache is a dict of NumPy arrays:

    k, v       codes as float64 values [layers, pages, heads, page_tokens, D]
    ks, vs     fp32 scales [layers, pages, heads, page_tokens / 16]
    table      int [rows, row_pages], lens int [rows], refs int [pages]

with "fmt" ("int8" or "e4m3").  Every rounding that the definition names is
carried out; everything else is float64.
"""
from __future__ import annotations

import copy

import numpy as np

BLOCK = 16
TOP = {"int8": 127.0, "e4m3": 448.0}
FLOOR = 2.0 ** -80


def e4m3_value(code: int) -> float:
    """Value of an e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F / 0xFF are NaN."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


E4M3 = np.array([e4m3_value(c) for c in range(256)])
_POS = E4M3[:127]  # 0 .. 448, ascending with the code


def _e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of |x| <= 448, ties to the even code."""
    a = np.abs(x)
    hi = np.searchsorted(_POS, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.copysign(_POS[pick], x)


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """fp32 quotients to code values: nearest even, clamped, NaN as 0."""
    top = TOP[fmt]
    x = np.where(np.isnan(x), 0.0, np.clip(x, -top, top)).astype(np.float64)
    return np.rint(x) if fmt == "int8" else _e4m3_round(x)


def decode_bytes(raw: np.ndarray, fmt: str) -> np.ndarray:
    """Stored bytes (uint8) to code values."""
    return raw.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[raw]


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def _spans(cache, starts):
    rows = len(cache["lens"])
    return [(r, r + 1) if starts is None else (int(starts[r]), int(starts[r + 1])) for r in range(rows)]


def append(cache, k, v, base, starts=None, layer=0):
    """Appends in place; k, v: [tokens, heads, D] of the values that the library gets."""
    pt, fmt = cache["k"].shape[3], cache["fmt"]
    top = TOP[fmt]
    for new, codes, scales in ((k, cache["k"][layer], cache["ks"][layer]), (v, cache["v"][layer], cache["vs"][layer])):
        new = np.asarray(new, np.float64)
        for r, (lo, hi) in enumerate(_spans(cache, starts)):
            b = int(base[r])
            if b < 0:
                continue
            at = b
            while at < b + hi - lo:  # one block at a time
                t0 = at // BLOCK * BLOCK
                end = min(t0 + BLOCK, b + hi - lo)
                page, sub = int(cache["table"][r, t0 // pt]), t0 % pt // BLOCK
                for h in range(new.shape[1]):
                    x = new[lo + at - b: lo + end - b, h]
                    fin = np.abs(x[np.isfinite(x)])
                    amax = max(fin.max() if fin.size else 0.0, FLOOR)
                    s0 = float(scales[page, h, sub]) if at > t0 else 0.0
                    s1 = max(s0, float(_f32(amax * float(_f32(1.0 / top)))))
                    inv = float(_f32(1.0 / s1))
                    rows = codes[page, h, t0 % pt: t0 % pt + BLOCK]
                    if s1 > s0:
                        old = rows[:at - t0]
                        rows[:at - t0] = encode(_f32(_f32(old * s0) * inv), fmt)
                        scales[page, h, sub] = s1
                    with np.errstate(invalid="ignore", over="ignore"):
                        rows[at - t0: end - t0] = encode(_f32(x * inv), fmt)
                at = end


def values(cache, row, head, which, layer=0):
    """Stored values [len, D] of one row and KV head, and their blocks' scales [len]."""
    pt, n = cache["k"].shape[3], int(cache["lens"][row])
    codes, scales = cache[which][layer], cache[which + "s"][layer]
    out, sc = np.zeros((n, codes.shape[-1])), np.zeros(n)
    for t in range(n):
        page = int(cache["table"][row, t // pt])
        sc[t] = float(scales[page, head, t % pt // BLOCK])
        out[t] = codes[page, head, t % pt] * sc[t]
    return out, sc


def attend(cache, q, starts=None, layer=0, scale=None, window=0):
    """(out, lse, bound): bound is what fp32 scores and fp16 weights may add up to, before
    the rounding of the output.  q: [tokens, q_heads, D] of the values that the library gets.

    A score's fp32 error is at most e = 2^-20 f sum_d |q_d K_d| (D <= 256 products summed in
    fp32, each sum off by no more than 2^-23 of the partial sums, and the loss of fp16's range
    in q, 2^-25 of its largest value a product), which scales a weight by at most 1 + 2e;
    a weight's fp16 rounding by 1 + 2^-11, with at least 2^-25 absolute of a weight near 1 for
    each of n keys with codes up to top."""
    q = np.asarray(q, np.float64)
    tokens, hq, d = q.shape
    hk = cache["k"].shape[2]
    grp = hq // hk
    f = 1.0 / np.sqrt(d) if scale is None else float(scale)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lbound = np.full((tokens, hq), -np.inf), np.zeros((tokens, hq))
    for r, (lo, hi) in enumerate(_spans(cache, starts)):
        n, length = hi - lo, int(cache["lens"][r])
        for h in range(hk):
            K, _ = values(cache, r, h, "k", layer)
            V, vs = values(cache, r, h, "v", layer)
            for i in range(n):
                p = length - n + i
                first = max(0, p + 1 - window) if window else 0
                if p < 0 or first > p:
                    continue
                for g in range(grp):
                    qv = q[lo + i, h * grp + g]
                    s = f * (K[first:p + 1] @ qv)
                    m = s.max()
                    w = np.exp(s - m)
                    Z = w.sum()
                    o = w @ V[first:p + 1] / Z
                    e = 2.0 ** -20 * abs(f) * (np.abs(K[first:p + 1]) @ np.abs(qv) +
                                              np.abs(K[first:p + 1]).sum(axis=1) * np.abs(qv).max()).max() + 2.0 ** -20
                    e += 2.0 ** -22 * (np.abs(s).max() + 100)
                    out[lo + i, h * grp + g] = o
                    bound[lo + i, h * grp + g] = (2.0 ** -11 + 4 * e) * (w @ np.abs(V[first:p + 1])) / Z + \
                        len(w) * 2.0 ** -25 * TOP[cache["fmt"]] * (w * vs[first:p + 1]).max() / Z
                    lse[lo + i, h * grp + g] = m + np.log(Z)
                    lbound[lo + i, h * grp + g] = 2 * e + 2.0 ** -20
    return out, lse, bound, lbound


# ---- pages ---------------------------------------------------------------------------------------

def _pages(n, pt):
    return -(-int(n) // pt)


def reserve(cache, counts):
    """(base, status); the cache changes in place where it succeeds."""
    pt, rows, width = cache["k"].shape[3], len(cache["lens"]), cache["table"].shape[1]
    lens, table, refs = cache["lens"], cache["table"], cache["refs"]
    ends = {}  # rows of the call that end inside a page, by page
    for r in range(rows):
        if counts[r] > 0 and lens[r] % pt:
            ends.setdefault(int(table[r, lens[r] // pt]), []).append(r)
    plan, total, over = [], 0, 0
    for r in range(rows):
        if counts[r] <= 0:
            continue
        if lens[r] + counts[r] > width * pt:
            over += 1
            continue
        copy_of = -1
        if lens[r] % pt:
            page = int(table[r, lens[r] // pt])
            if refs[page] > 1 and not (len(ends[page]) == refs[page] and ends[page][0] == r):
                copy_of = page
        fresh = _pages(lens[r] + counts[r], pt) - _pages(lens[r], pt)
        plan.append((r, copy_of, fresh))
        total += fresh + (copy_of >= 0)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    status = [max(0, total - len(free)), over]
    if status != [0, 0]:
        return np.full(rows, -1), status
    base = lens.copy()
    for r, copy_of, fresh in plan:
        if copy_of >= 0:
            page = free.pop(0)
            for name in ("k", "v", "ks", "vs"):
                cache[name][:, page] = cache[name][:, copy_of]
            table[r, lens[r] // pt] = page
            refs[page] = 1
            refs[copy_of] -= 1
        for j in range(fresh):
            page = free.pop(0)
            table[r, _pages(lens[r], pt) + j] = page
            refs[page] = 1
        lens[r] += counts[r]
    return base, status


def fork(cache, parents, keep=None):
    """The new cache (its pools are shared)."""
    pt, width = cache["k"].shape[3], cache["table"].shape[1]
    new = dict(cache)
    rows = len(parents)
    new["table"], new["lens"] = np.full((rows, width), -1, np.int64), np.zeros(rows, np.int64)
    refs = cache["refs"].copy()
    for r in range(len(cache["lens"])):
        for j in range(_pages(cache["lens"][r], pt)):
            refs[cache["table"][r, j]] -= 1
    for i, p in enumerate(parents):
        n = 0 if not 0 <= p < len(cache["lens"]) else int(cache["lens"][p])
        if keep is not None:
            n = max(0, min(n, int(keep[i])))
        new["lens"][i] = n
        for j in range(_pages(n, pt)):
            new["table"][i, j] = cache["table"][p, j]
            refs[new["table"][i, j]] += 1
    new["refs"] = refs
    return new


def compact(cache):
    """(new cache, pages moved); the pools change in place."""
    pt = cache["k"].shape[3]
    new = dict(cache)
    refs, to = cache["refs"].copy(), {}
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] == 0]
    for page in range(live, len(refs)):
        if refs[page] > 0:
            hole = holes.pop(0)
            to[page] = hole
            for name in ("k", "v", "ks", "vs"):
                cache[name][:, hole] = cache[name][:, page]
            refs[hole], refs[page] = refs[page], 0
    new["refs"], new["lens"] = refs, cache["lens"].copy()
    new["table"] = np.full_like(cache["table"], -1)
    for r in range(len(cache["lens"])):
        for j in range(_pages(cache["lens"][r], pt)):
            p = int(cache["table"][r, j])
            new["table"][r, j] = to.get(p, p)
    return new, len(to)


def clone(cache):
    return copy.deepcopy(cache)
