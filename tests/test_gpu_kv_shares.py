"""The few-query attention in equal shares (long plans: most decode calls of a server) over head sizes,
code formats, element types, windows, one and several queries a row; a row cut into more pieces than
the joining kernel holds at once; and more rows than a CTA adds up, which take clusters.  Each case
asserts that it is planned in the form it is here for.  Tolerances as in the other tests of attention."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import BF16_HALF, F16_HALF, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu


def _check(c, grp, news, dtype, window, seed, shares=True):
    d, heads = c["k"].shape[4], c["k"].shape[2]
    rows, most = len(c["lens"]), 1 if news is None else max(news)
    tokens = rows if news is None else sum(news)
    q, qd = rounded(np.random.default_rng(seed).standard_normal((tokens, heads * grp, d)) * 1.5, dtype)
    lib = to_library(c)
    assert (lib.attend_workspace(heads * grp, tokens, most, 0, window) > 0) == shares
    assert most * grp <= (32 if d == 256 else 48)  # the few-query form
    starts = None if news is None else starts_of(news)
    out, lse = lib.attend(q.cuda(), None if news is None else i32(starts), max_new=most, window=window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    want, wlse, bound, lbound = okv.attend(c, qd, starts, window=window)
    half = F16_HALF if dtype == "float16" else BF16_HALF
    tol = bound * (1 + half) + half * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(out - want) <= tol), float((np.abs(out - want) / tol).max())
    seen = wlse > -np.inf
    np.testing.assert_array_equal(lse > -np.inf, seen)
    assert np.all(np.abs(lse[seen] - wlse[seen]) <= lbound[seen] + 2.0 ** -22 * np.abs(wlse[seen]))
    assert np.all(out[~seen] == 0)


FORMS = [("float16", "int8", 128, 4, 6), ("bfloat16", "e4m3", 128, 3, 8), ("bfloat16", "int8", 64, 2, 7),
         ("float16", "e4m3", 64, 3, 3), ("float16", "e4m3", 256, 2, 6), ("bfloat16", "int8", 256, 1, 8)]


@pytest.mark.parametrize("dtype,fmt,d,heads,grp", FORMS)
@pytest.mark.parametrize("news", [None, [3, 1, 4, 0, 2, 2]])
def test_mixed_lengths(dtype, fmt, d, heads, grp, news):
    lens = [2600, 5, 0, 700, 17, 1300]
    c = random_cache(np.random.default_rng(d + heads), lens, heads=heads, d=d, pt=64, fmt=fmt, row_pages=4000)
    _check(c, grp, news, dtype, 0, d)


@pytest.mark.parametrize("dtype,fmt,d,heads,grp,rows", [
    ("float16", "int8", 128, 8, 6, 24), ("bfloat16", "e4m3", 64, 8, 6, 24), ("bfloat16", "e4m3", 256, 4, 6, 24)])
@pytest.mark.parametrize("most", [1, 4])
def test_a_window(dtype, fmt, d, heads, grp, rows, most):
    rng = np.random.default_rng(d)
    lens = [int(1700 * u ** 2) for u in rng.random(rows)]
    lens[:4] = [1700, 0, 899, 903]
    news = None if most == 1 else [int(n) for n in rng.integers(0, most + 1, rows)]
    if news:
        news[0] = most
    c = random_cache(rng, lens, heads=heads, d=d, pt=32, fmt=fmt, row_pages=600)
    _check(c, grp, news, dtype, 900, d)


@pytest.mark.parametrize("dtype,fmt,d,heads,grp", [("float16", "int8", 64, 10, 2), ("bfloat16", "e4m3", 256, 2, 24)])
def test_a_window_of_one(dtype, fmt, d, heads, grp):
    rng = np.random.default_rng(d)
    lens = [int(n) for n in rng.integers(0, 21, 1000)]
    c = random_cache(rng, lens, heads=heads, d=d, pt=16, fmt=fmt)
    _check(c, grp, None, dtype, 1, d)


@pytest.mark.parametrize("dtype,fmt,d,grp,news", [
    ("float16", "int8", 128, 6, None), ("bfloat16", "e4m3", 128, 5, [5, 2]), ("float16", "e4m3", 64, 4, [1, 3]),
    ("bfloat16", "int8", 256, 6, None)])
def test_a_row_in_many_pieces(dtype, fmt, d, grp, news):
    """A share has 32 tiles of 16 tokens at least: 9000 tokens are 18 pieces."""
    c = random_cache(np.random.default_rng(d), [9000, 40], heads=1, d=d, pt=128, fmt=fmt, row_pages=2000)
    _check(c, grp, news, dtype, 0, d)


@pytest.mark.parametrize("d,grp,news", [(128, 2, None), (64, 3, "some"), (256, 2, "some")])
def test_more_rows_than_a_cta_adds_up(d, grp, news):
    rng = np.random.default_rng(d)
    lens = [int(n) for n in rng.integers(0, 40, 1025)]
    lens[7], lens[1024] = 300, 39
    if news:
        news = [int(n) for n in rng.integers(0, 4, 1025)]
    c = random_cache(rng, lens, heads=1, d=d, pt=16, row_pages=4000)
    _check(c, grp, news, "float16", 0, d, shares=False)
