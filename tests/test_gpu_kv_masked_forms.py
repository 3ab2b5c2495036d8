"""The kernel of 128-row tiles under masks: calls without scratch, and plans over more rows than a warp, than the
threads of a CTA, and up to the most that a call plans."""
import ctypes

import numpy as np
import pytest

import oracle.draft_step as od
from _kv_util import F16_HALF, i32, random_cache, rounded, starts_of, to_library
from test_gpu_draft_trees import _parents
from test_gpu_kv_tree_attend import _compare, _run

pytestmark = pytest.mark.gpu

LARGE = 1 << 24  # the tile kernel's scratch is more than that


@pytest.mark.parametrize("fmt,d", [("int8", 64), ("e4m3", 128), ("int8", 256)])
@pytest.mark.parametrize("window", [0, 70, 900])
def test_tiles_without_scratch(fmt, d, window):
    """Enough rows and heads that the tile kernel is taken for a window's keys too; nothing is shared."""
    import torch
    lens, news, hk, grp = [1500, 64, 0, 700], [64, 60, 0, 33], 12, 6
    rng = np.random.default_rng(d + window)
    # (a window of 70 is planned for the few-query kernel at this size, and long rows do not change that)
    c = random_cache(rng, lens, heads=hk, d=d, pt=64, fmt=fmt)
    q, qd = rounded(rng.standard_normal((sum(news), hk * grp, d)) * 1.5, "float16")
    seen, depth = od.tree_mask(_parents(rng, news), starts_of(news))
    lib = to_library(c)
    need = lib.attend_workspace(hk * grp, sum(news), 64, 0, window, masked=True)
    assert window == 70 or need > LARGE
    qg, starts = q.cuda(), i32(starts_of(news))
    mask, dep = torch.from_numpy(od.mask_words(seen, 1)).cuda(), i32(depth)
    out, lse = torch.empty_like(qg), torch.empty(q.shape[:2], device="cuda")
    st = lib._lib.bqd_kv_attend_masked(lib._ref, 0, qg.data_ptr(), hk * grp * d, d, 1, hk * grp, starts.data_ptr(), sum(news), 64, 0,
                                       ctypes.c_float(1 / np.sqrt(d)), window, mask.data_ptr(), 1, dep.data_ptr(), out.data_ptr(),
                                       lse.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    want, wlse, bound, lbound = od.masked_attend(c, qd, starts_of(news), seen, depth, window=window)
    assert np.all(np.abs(got - want) <= bound * (1 + F16_HALF) + F16_HALF * np.abs(want) + 2.0 ** -25)
    some = wlse > -np.inf
    np.testing.assert_array_equal(glse > -np.inf, some)
    assert np.all(np.abs(glse[some] - wlse[some]) <= lbound[some] + 2.0 ** -22 * np.abs(wlse[some]))


@pytest.mark.parametrize("rows", [31, 33, 300, 512, 513, 600, 1024])
@pytest.mark.parametrize("d,grp,fmt", [(64, 11, "int8"), (128, 7, "e4m3"), (256, 6, "int8")])
def test_plans_over_many_rows(rows, d, grp, fmt):
    """Rows of a few tokens among some of thousands, whose keys are shared, and rows without nodes; the same bits again."""
    rng = np.random.default_rng(rows + d)
    news = [int(n) for n in rng.integers(0, 4, rows)]
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 40, rows))]
    for at, n in ((0, 1700), (rows // 2, 2600), (rows - 1, 700)):
        lens[at], news[at] = n, 3
    lens[1], news[1] = 2000, 0
    c = random_cache(rng, lens, heads=1, d=d, pt=16, fmt=fmt, row_pages=12000)
    q, qd = rounded(rng.standard_normal((sum(news), grp, d)) * 1.5, "float16")
    seen, depth = od.tree_mask(_parents(rng, news), starts_of(news))
    got, _ = _compare(c, q, qd, news, "float16", seen, depth=depth, tiles=True)
    np.testing.assert_array_equal(got, _run(c, q, news, seen, 1, None, 0)[0])


@pytest.mark.parametrize("rows,n,grp", [(40, 64, 6), (600, 43, 6)])
def test_plans_over_many_rows_of_several_tiles(rows, n, grp):
    """Pairs and single tiles in one plan, most rows idle."""
    rng = np.random.default_rng(rows)
    news, lens = [0] * rows, [int(x) for x in rng.integers(0, 30, rows)]
    for at, m, length in ((0, n, 900), (3, 1, 40), (rows // 2 + 1, n, 2100), (rows - 2, n // 2, 300), (rows - 1, n - 1, n - 1)):
        news[at], lens[at] = m, length
    c = random_cache(rng, lens, heads=2, d=128, pt=32, row_pages=6000)
    q, qd = rounded(rng.standard_normal((sum(news), 2 * grp, 128)) * 1.5, "bfloat16")
    seen, depth = od.tree_mask(_parents(rng, news), starts_of(news))
    got, _ = _compare(c, q, qd, news, "bfloat16", seen, depth=depth, tiles=True)
    np.testing.assert_array_equal(got, _run(c, q, news, seen, 1, None, 0)[0])
