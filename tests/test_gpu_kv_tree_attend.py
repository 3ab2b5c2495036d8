"""Attention over the cache under masks (bqd_kv_attend_masked) against the float64 oracle, with the
tolerances of the causal attention's tests: the oracle's bound on fp32 scores and fp16 weights, and half a
unit in the last place of the output type.

Two kernels serve masked calls: the few-query one where the call is planned short (by the table's
capacity, where no length is given) or has few (query, head) rows, and one of 128-row tiles else.
``tiles`` asserts which one a case is here for: the tile kernel's scratch is over 16 MB, whatever the call."""
import numpy as np
import pytest

import oracle.draft_step as od
import oracle.kv_cache as okv
from _kv_util import BF16_HALF, F16_HALF, i32, random_cache, rounded, starts_of, to_library
from test_gpu_draft_trees import _parents

pytestmark = pytest.mark.gpu


LONG = 60000  # pages of a row's table: planned long


def _run(c, q, news, seen, words, depth, window, tiles=None, **kw):
    import torch
    lib = to_library(c)
    if tiles is not None:
        need = lib.attend_workspace(q.shape[1], sum(news), kw.get("max_new", max(news)), kw.get("max_len", 0), window, masked=True)
        assert (need > 1 << 24) == tiles
    kw.setdefault("max_new", max(news))
    mask = torch.from_numpy(od.mask_words(seen, words)).cuda()
    out, lse = lib.attend(q.cuda(), i32(starts_of(news)), mask=mask, depth=None if depth is None else i32(depth), window=window, **kw)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _compare(c, q, qd, news, dtype, seen, words=1, depth=None, window=0, layer=0, scale=None, **kw):
    got, glse = _run(c, q, news, seen, words, depth, window, layer=layer, scale=scale, **kw)
    seen = [{j for j in s if j < 64 * words} for s in seen]
    want, lse, bound, lbound = od.masked_attend(c, qd, starts_of(news), seen, depth, layer, scale, window)
    half = F16_HALF if dtype == "float16" else BF16_HALF
    tol = bound * (1 + half) + half * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
    some = lse > -np.inf
    np.testing.assert_array_equal(glse > -np.inf, some)
    assert np.all(np.abs(glse[some] - lse[some]) <= lbound[some] + 2.0 ** -22 * np.abs(lse[some]))
    assert np.all(got[~some] == 0)
    return got, glse


def _case(seed, lens, news, dtype, fmt, d, hk, grp, pt, **kw):
    rng = np.random.default_rng(seed)
    c = random_cache(rng, lens, heads=hk, d=d, pt=pt, fmt=fmt, **kw)
    q, qd = rounded(rng.standard_normal((sum(news), hk * grp, d)) * 1.5, dtype)
    seen, depth = od.tree_mask(_parents(rng, news), starts_of(news))
    return c, q, qd, seen, depth


SHAPES = [
    # dtype, fmt, D, kv heads, group, page, lens, news: few queries in clusters, then many
    ("float16", "int8", 128, 2, 6, 64, [40, 0, 5, 300], [8, 0, 5, 3]),
    ("bfloat16", "e4m3", 64, 1, 7, 32, [70, 6, 33], [6, 6, 5]),
    ("bfloat16", "int8", 256, 1, 4, 16, [100, 17, 16], [8, 1, 7]),
    ("float16", "e4m3", 128, 2, 1, 128, [260, 129, 48], [48, 2, 48]),
    ("float16", "int8", 128, 2, 6, 64, [701, 26, 90], [26, 26, 1]),
    ("bfloat16", "e4m3", 64, 1, 7, 32, [170, 64, 0], [64, 63, 0]),
    ("float16", "int8", 256, 1, 6, 16, [300, 61], [64, 61]),
    ("bfloat16", "int8", 128, 1, 16, 64, [500, 65], [40, 20]),
]


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens,news", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 30])
def test_trees(dtype, fmt, d, hk, grp, pt, lens, news, window):
    c, q, qd, seen, depth = _case(sum(lens) + d, lens, news, dtype, fmt, d, hk, grp, pt)
    _compare(c, q, qd, news, dtype, seen, depth=depth, window=window, tiles=False)


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens,news", SHAPES)
def test_trees_planned_long(dtype, fmt, d, hk, grp, pt, lens, news):
    """The tile kernel where the rows are more than the few-query kernel takes in two passes (one with heads of 128)."""
    rows = max(news) * grp
    c, q, qd, seen, depth = _case(sum(lens) + d, lens, news, dtype, fmt, d, hk, grp, pt, row_pages=LONG)
    _compare(c, q, qd, news, dtype, seen, depth=depth, tiles=rows > (32 if d == 64 else 16))


@pytest.mark.parametrize("d,fmt,dtype", [(64, "e4m3", "bfloat16"), (128, "int8", "float16"), (128, "e4m3", "bfloat16"), (256, "int8", "float16")])
@pytest.mark.parametrize("window", [1, 70, 900])
def test_a_window_over_tiles(d, fmt, dtype, window):
    """Enough rows and heads that even a window's keys are planned for the tile kernel; pairs, single tiles, an empty row."""
    lens, news = [1500, 64, 0, 700], [64, 60, 0, 33]
    c, q, qd, seen, depth = _case(d + window, lens, news, dtype, fmt, d, 12, 6, 64)
    _compare(c, q, qd, news, dtype, seen, depth=depth, window=window, tiles=window == 900 or None)


@pytest.mark.parametrize("grp,d", [(1, 64), (4, 128), (2, 256)])
@pytest.mark.parametrize("window,pages", [(0, None), (200, None), (0, LONG)])
def test_wide_masks(grp, d, window, pages):
    """More than 64 nodes, two to four words, bits that cross them and tiles."""
    news, lens = [150, 65, 200], [400, 65, 231]
    c, q, qd, seen, depth = _case(7, lens, news, "bfloat16", "int8", d, 1, grp, 32, row_pages=pages)
    _compare(c, q, qd, news, "bfloat16", seen, words=4, depth=depth, window=window)
    # tokens past the words are seen by none
    _compare(c, q, qd, news, "bfloat16", seen, words=2, depth=depth, window=window)


@pytest.mark.parametrize("n,grp", [(5, 3), (48, 1), (64, 6)])
@pytest.mark.parametrize("pages", [None, LONG])
def test_any_mask(n, grp, pages):
    """Bits of later tokens, rows without a bit, and bits past the row's tokens (not read); with and without a prefix."""
    rng = np.random.default_rng(n)
    news, lens = [n, n, n], [n + 77, n, n]
    c, q, qd, _, _ = _case(n, lens, news, "float16", "int8", 128, 1, grp, 64, row_pages=pages)
    seen = [set(rng.choice(n + 6, int(rng.integers(0, n)), replace=False).tolist()) for _ in range(3 * n)]
    seen[n:n + 2] = [set(), {n + 1}]
    for i in range(2 * n, 3 * n):
        seen[i] = set()             # a row that sees nothing at all
    _, lse = _compare(c, q, qd, news, "float16", seen)
    assert np.all(lse[2 * n:] == -np.inf) and np.all(lse[n:n + 2] == -np.inf)


@pytest.mark.parametrize("n,grp,d", [(8, 6, 128), (40, 3, 128), (8, 3, 256), (70, 7, 64)])
@pytest.mark.parametrize("pages", [None, 4000])
def test_a_causal_mask_gives_what_the_causal_call_gives(n, grp, d, pages):
    """Each within its bound of the exact value."""
    news, lens = [n, 3, n - 1], [900, 60, n - 1]
    c, q, qd, _, _ = _case(n, lens, news, "bfloat16", "int8", d, 2, grp, 64, row_pages=pages)
    got, lse = _compare(c, q, qd, news, "bfloat16", [set(range(i + 1)) for m in news for i in range(m)], words=2)
    out, want = to_library(c).attend(q.cuda(), i32(starts_of(news)), max_new=n)
    exact, _, bound, lbound = okv.attend(c, qd, starts_of(news))
    tol = 2 * (bound * (1 + BF16_HALF) + BF16_HALF * np.abs(exact))
    assert np.all(np.abs(got - out.double().cpu().numpy()) <= tol)
    assert np.all(np.abs(lse - want.double().cpu().numpy()) <= 2 * lbound + 2.0 ** -21 * np.abs(lse))


@pytest.mark.parametrize("n,grp,d,fmt", [(4, 4, 128, "int8"), (4, 7, 64, "e4m3"), (2, 6, 256, "int8")])
def test_equal_shares(n, grp, d, fmt):
    """Few queries planned long, so that shares cut the rows."""
    lens, news = [2600, 5, 0, 700, n, 1300], [n, 2, 0, 1, n, n - 1]
    c, q, qd, seen, depth = _case(d, lens, news, "float16", fmt, d, 4, grp, 64, row_pages=4000)
    lib = to_library(c)
    assert 0 < lib.attend_workspace(4 * grp, sum(news), n, masked=True) < 1 << 24
    _compare(c, q, qd, news, "float16", seen)


@pytest.mark.parametrize("n,grp,d,hk,fmt", [(4, 6, 128, 8, "int8"), (4, 6, 64, 8, "e4m3"), (4, 6, 256, 4, "int8")])
def test_equal_shares_with_a_window(n, grp, d, hk, fmt):
    rng = np.random.default_rng(d)
    lens = [int(1700 * u ** 2) for u in rng.random(24)]
    lens[:4] = [1700, 0, 899, 903]
    news = [n] + [int(x) for x in rng.integers(0, n + 1, 23)]
    lens = [max(a, b) for a, b in zip(lens, news)]
    c, q, qd, seen, depth = _case(d, lens, news, "bfloat16", fmt, d, hk, grp, 32, row_pages=600)
    assert 0 < to_library(c).attend_workspace(hk * grp, sum(news), n, 0, 900, masked=True) < 1 << 24
    _compare(c, q, qd, news, "bfloat16", seen, depth=depth, window=900)


@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (128, "int8"), (256, "int8")])
@pytest.mark.parametrize("hk", [1, 2])
def test_shares_of_tiles(d, fmt, hk):
    """Several CTAs share a tile's keys: rows of very different lengths, an empty one, pairs and single tiles.  The same
    bits every time; a plan that is shorter than the rows; and rows that a CTA does not add up."""
    lens, news = [2500, 0, 9, 1700], [64, 0, 9, 40]
    c, q, qd, seen, depth = _case(16, lens, news, "bfloat16", fmt, d, hk, 6, 64, row_pages=LONG)
    got, _ = _compare(c, q, qd, news, "bfloat16", seen, tiles=True)
    np.testing.assert_array_equal(got, _run(c, q, news, seen, 1, depth, 0)[0])
    _compare(c, q, qd, news, "bfloat16", seen, max_len=1000, tiles=None)


@pytest.mark.parametrize("d,grp", [(64, 11), (128, 7), (256, 6)])
def test_more_rows_than_a_cta_adds_up(d, grp):
    rng = np.random.default_rng(d)
    news = [int(n) for n in rng.integers(0, 4, 1030)]
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 40, 1030))]
    lens[5], news[1029] = 700, 3
    c, q, qd, seen, depth = _case(d, lens, news, "float16", "int8", d, 1, grp, 16, row_pages=4000)
    lib = to_library(c)
    assert lib.attend_workspace(grp, sum(news), 3, masked=True) == 0  # nothing is shared
    _compare(c, q, qd, news, "float16", seen, depth=depth)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 300])
def test_without_scratch(d, window):
    """The form that converts the codes in the kernel."""
    import ctypes
    import torch
    lens, news, hk, grp = [900, 64, 333], [64, 64, 17], 2, 6
    c, q, qd, seen, depth = _case(3, lens, news, "float16", "int8", d, hk, grp, 64, row_pages=LONG)
    lib = to_library(c)
    qg, starts = q.cuda(), i32(starts_of(news))
    out, lse = torch.empty_like(qg), torch.empty(q.shape[:2], device="cuda")
    mask, dep = torch.from_numpy(od.mask_words(seen, 1)).cuda(), i32(depth)
    st = lib._lib.bqd_kv_attend_masked(lib._ref, 0, qg.data_ptr(), hk * grp * d, d, 1, hk * grp, starts.data_ptr(), sum(news), 64, 0,
                                       ctypes.c_float(1 / np.sqrt(d)), window, mask.data_ptr(), 1, dep.data_ptr(), out.data_ptr(),
                                       lse.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want, _, bound, _ = od.masked_attend(c, qd, starts_of(news), seen, depth, window=window)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)


@pytest.mark.parametrize("n,most", [(40, 8), (100, 20), (30, 29)])
@pytest.mark.parametrize("window,pages", [(0, None), (50, None), (0, LONG)])
def test_more_nodes_than_the_bound(n, most, window, pages):
    """The later queries of a row are not computed; the others see what they saw."""
    news, lens = [n, 3], [300, 40]
    c, q, qd, seen, depth = _case(4, lens, news, "float16", "int8", 128, 1, 4, 64, row_pages=pages)
    full, _ = _run(c, q, news, seen, 2, depth, window)
    import torch
    lib = to_library(c)
    out = torch.full((sum(news), 4, 128), 7.0, dtype=torch.float16, device="cuda")
    lib.attend(q.cuda(), i32(starts_of(news)), mask=torch.from_numpy(od.mask_words(seen, 2)).cuda(), depth=i32(depth), window=window,
               max_new=most, out=out)
    out = out.double().cpu().numpy()
    assert np.all(out[most:n] == 7)
    want, _, bound, _ = od.masked_attend(c, qd, starts_of(news), seen, depth, window=window)
    done = list(range(most)) + list(range(n, n + 3))
    assert np.all(np.abs(out - want)[done] <= (bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)[done])


def test_wild_depths():
    """Depths outside [0, n) are cut to it."""
    news, lens = [6], [200]
    c, q, qd, seen, _ = _case(5, lens, news, "float16", "int8", 64, 1, 2, 32)
    depth = [-5, 2 ** 31 - 1, -2 ** 31, 3, 7, 0]
    _compare(c, q, qd, news, "float16", seen, depth=depth, window=60)
    news, lens = [60] * 3, [200, 60, 3000]
    c, q, qd, seen, _ = _case(5, lens, news, "float16", "int8", 64, 24, 4, 32)
    _compare(c, q, qd, news, "float16", seen, depth=depth * 30, window=600, tiles=True)


@pytest.mark.parametrize("n,grp", [(6, 6), (64, 6)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("pages", [None, LONG])
def test_what_lies_past_the_row_does_not_matter(n, grp, fmt, pages):
    """Stale codes, NaN bytes and NaN scales behind the row's end, on its last page and others."""
    import torch
    lens, news = [n + 39], [n]
    c, q, qd, seen, depth = _case(6, lens, news, "float16", fmt, 128, 1, grp, 64, row_pages=pages)
    want, _ = _run(c, q, news, seen, 1, None, 0)
    lib = to_library(c)
    page, used = int(c["table"][0, lens[0] // 64]), lens[0] % 64
    for t, s in ((lib.k, lib.k_scales), (lib.v, lib.v_scales)):
        t.view(torch.uint8)[:, page, :, used:] = 0x7F
        s[:, page, :, (used + 15) // 16:] = float("nan")
    mask = torch.full((n, 1), -1, dtype=torch.int64, device="cuda") & torch.from_numpy(od.mask_words(seen, 1)).cuda()
    out, _ = lib.attend(q.cuda(), i32([0, n]), mask=mask, max_new=n)
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)


def test_refusals():
    import torch
    lib = to_library(random_cache(np.random.default_rng(0), [20, 9], heads=2, d=64, pt=16))
    q, starts = torch.zeros((5, 4, 64), dtype=torch.float16, device="cuda"), i32([0, 3, 5])
    mask, depth = torch.ones((5, 1), dtype=torch.int64, device="cuda"), i32([0] * 5)
    lib.attend(q, starts, mask=mask, max_new=3)
    for kw in [dict(mask=mask.int()), dict(mask=mask[:4]), dict(mask=mask[:, 0]), dict(mask=mask.cpu()), dict(mask=mask[:, :0]),
               dict(mask=mask.expand(5, 17)), dict(mask=mask, depth=depth.long()), dict(mask=mask, depth=depth[:4]),
               dict(depth=depth), dict(mask=mask, window=5), dict(mask=mask.expand(5, 2))]:
        with pytest.raises(ValueError):
            lib.attend(q, starts, max_new=3, **kw)
    out, _ = lib.attend(q[:0], i32([0, 0, 0]), mask=mask[:0])
    assert out.shape == (0, 4, 64)


def test_the_names_of_the_entry_points_are_the_calls():
    import bit_quantized_decode_unpack_gb300 as bqd
    c, grp = random_cache(np.random.default_rng(3), [40, 3], heads=2, d=64, pt=16, row_pages=LONG // 16), 4
    lib = to_library(c)
    for args in [(2 * grp, 22, 20), (2 * grp, 22, 20, 900, 100), (2 * grp, 2, 1, 64)]:
        assert bqd.kv_attend_masked_workspace(lib, *args) == lib.attend_workspace(*args, masked=True)
        assert bqd.kv_attend_workspace(lib, *args) == lib.attend_workspace(*args)
    assert bqd.kv_attend_masked_workspace(lib, 2 * grp, 22, 20) != bqd.kv_attend_workspace(lib, 2 * grp, 22, 20)
