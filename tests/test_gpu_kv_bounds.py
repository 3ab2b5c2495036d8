"""bqd_kv_attend where a row has more queries than the call computes: max_new below a row's count,
or starts that go on past the tokens that are given.  The positions are those of the row's true
count (query i of n at lens - n + i), so what is computed equals the whole call's answer; the other
tokens' outputs stay as they are.  Tolerances as in the other tests of attention: the oracle's
bound and half a unit in the last place of the output."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import BF16_HALF, F16_HALF, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu


def _check(c, dtype, lens, news, max_new, tokens, window, seed, **kw):
    """Attends with the bounds and compares what they leave to compute with the oracle on everything."""
    import torch
    d, heads = c["k"].shape[4], c["k"].shape[2] * kw.pop("grp")
    starts = starts_of(news)
    q, qd = rounded(np.random.default_rng(seed).standard_normal((sum(news), heads, d)) * 1.5, dtype)
    want, lse, bound, lbound = okv.attend(c, qd, starts, window=window)
    out = torch.full((tokens, heads, d), 7.0, dtype=q.dtype, device="cuda")
    got_lse = torch.full((tokens, heads), 7.0, device="cuda")
    to_library(c).attend(q[:tokens].cuda(), i32(starts), max_new=max_new, window=window, out=out, lse=got_lse, **kw)
    out, got_lse = out.double().cpu().numpy(), got_lse.double().cpu().numpy()
    done = np.zeros(tokens, bool)
    for r in range(len(news)):
        done[starts[r]:min(starts[r] + min(news[r], max_new), tokens)] = True
    half = F16_HALF if dtype == "float16" else BF16_HALF
    err = np.abs(out - want[:tokens])[done]
    tol = (bound * (1 + half) + half * np.abs(want) + 2.0 ** -25)[:tokens][done]
    assert np.all(err <= tol), float((err / tol).max())
    seen = (lse[:tokens] > -np.inf) & done[:, None]
    assert np.all(got_lse[done[:, None] & ~seen] == -np.inf)
    assert np.all(np.abs(got_lse - lse[:tokens])[seen] <= (lbound[:tokens] + 2.0 ** -22 * np.abs(lse[:tokens]))[seen])
    assert np.all(out[~done] == 7) and np.all(got_lse[~done] == 7)


CASES = [
    # dtype, fmt, D, kv heads, group, page, lens, news, max_new, row_pages: the form that takes it
    ("float16", "int8", 64, 2, 2, 32, [20, 50], [4, 5], 3, None),                 # clusters, 8 columns
    ("bfloat16", "e4m3", 128, 1, 6, 64, [40, 0, 300, 7], [9, 0, 6, 7], 4, None),  # clusters, 16 columns
    ("float16", "int8", 256, 1, 6, 16, [100, 17], [9, 3], 5, None),
    ("float16", "int8", 64, 1, 4, 16, [900, 5, 33, 700, 64, 1], [6, 5, 4, 9, 2, 1], 3, 4000),  # shares
    ("float16", "int8", 128, 1, 6, 64, [90, 300], [30, 60], 20, None),            # one query tile
    ("bfloat16", "int8", 128, 2, 3, 64, [500, 210, 40], [400, 90, 40], 150, None),  # several
    ("float16", "e4m3", 64, 1, 7, 32, [200, 70], [180, 70], 100, None),
    ("float16", "int8", 256, 1, 4, 64, [330, 90], [200, 90], 70, None),
]


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens,news,max_new,row_pages", CASES)
@pytest.mark.parametrize("window", [0, 1, 40])
def test_max_new_below_a_rows_count(dtype, fmt, d, hk, grp, pt, lens, news, max_new, row_pages, window):
    c = random_cache(np.random.default_rng(d + max_new), lens, heads=hk, d=d, pt=pt, fmt=fmt, row_pages=row_pages)
    _check(c, dtype, lens, news, max_new, sum(news), window, max_new, grp=grp)


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens,news,max_new,row_pages", CASES)
@pytest.mark.parametrize("window", [0, 40])
def test_starts_past_the_tokens(dtype, fmt, d, hk, grp, pt, lens, news, max_new, row_pages, window):
    """The last row's later tokens (and some of the row before) are not in q."""
    c = random_cache(np.random.default_rng(d + max_new), lens, heads=hk, d=d, pt=pt, fmt=fmt, row_pages=row_pages)
    for tokens in (sum(news) - 1, sum(news[:-1]) - 1):
        _check(c, dtype, lens, news, max(news), tokens, window, tokens, grp=grp)


@pytest.mark.parametrize("max_new", [25, 64])
def test_few_computed_queries_far_behind(max_new):
    """Many keys and few computed queries, so that CTAs share the keys of a tile."""
    lens, news = [2500, 1700], [70, 90]
    c = random_cache(np.random.default_rng(3), lens, heads=1, d=128, pt=64)
    for window in (0, 900):
        _check(c, "bfloat16", lens, news, max_new, sum(news), window, max_new, grp=3)
