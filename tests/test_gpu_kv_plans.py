"""Many-query attention under plans that differ from the rows: windows far shorter than the table,
and tables too long to convert the codes ahead.  Against the oracle, with the tolerances of the
other tests of attention."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import BF16_HALF, F16_HALF, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu

MOST = 2 << 30


def _check(c, q, qd, news, dtype, window, **kw):
    lib, starts = to_library(c), starts_of(news)
    out, lse = lib.attend(q.cuda(), i32(starts), max_new=max(news), window=window, **kw)
    want, wlse, bound, lbound = okv.attend(c, qd, starts, window=window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    half = F16_HALF if dtype == "float16" else BF16_HALF
    tol = bound * (1 + half) + half * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(out - want) <= tol), float((np.abs(out - want) / tol).max())
    seen = wlse > -np.inf
    np.testing.assert_array_equal(lse > -np.inf, seen)
    assert np.all(np.abs(lse[seen] - wlse[seen]) <= lbound[seen] + 2.0 ** -22 * np.abs(wlse[seen]))
    return lib


@pytest.mark.parametrize("d,grp,fmt,dtype", [(64, 7, "e4m3", "bfloat16"), (128, 3, "int8", "float16"), (256, 2, "int8", "bfloat16")])
@pytest.mark.parametrize("window", [1, 100, 129, 700])
@pytest.mark.parametrize("max_len", [0, 1500, 300])
def test_a_window_far_shorter_than_the_table(d, grp, fmt, dtype, window, max_len):
    rng = np.random.default_rng(d + window)
    lens, news = [1500, 0, 331, 90], [260, 3, 331, 70]
    c = random_cache(rng, lens, heads=1, d=d, pt=64, fmt=fmt, row_pages=2048)
    q, qd = rounded(rng.standard_normal((sum(news), grp, d)), dtype)
    lib = _check(c, q, qd, news, dtype, window, max_len=max_len)
    # the codes are converted ahead, for the window and its queries alone
    step = 64 if d == 256 else 128
    need = lib.attend_workspace(grp, sum(news), max(news), max_len, window)
    assert 0 < need <= 4 * (min(max_len or 1 << 17, window + 331) // step + 2) * (2 * step * d * 2 + step // 2) + \
        16 * sum(news) * grp * (d * 4 + 8)


@pytest.mark.parametrize("d,dtype", [(64, "float16"), (128, "bfloat16"), (256, "float16")])
def test_a_table_too_long_to_convert_ahead(d, dtype):
    rng = np.random.default_rng(d)
    lens, news = [900, 130], [90, 100]
    c = random_cache(rng, lens, heads=8, d=d, pt=256, row_pages=4096)
    q, qd = rounded(rng.standard_normal((sum(news), 24, d)), dtype)
    lib = _check(c, q, qd, news, dtype, 0)
    assert 0 < lib.attend_workspace(24, sum(news), max(news)) <= 16 * sum(news) * 24 * (d * 4 + 8)
    _check(c, q, qd, news, dtype, 200)
