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


def _planned(rows, seed, top):
    """A cache of `rows` rows with a few nodes each, planned long, and its oracle's numbers."""
    rng = np.random.default_rng(seed)
    news = [int(n) for n in rng.integers(0, 9, rows)]
    lens = [n + int(top * u ** 6) for n, u in zip(news, rng.random(rows))]
    return rng, news, lens


@pytest.mark.parametrize("rows", [12, 40])
def test_a_captured_call_follows_lengths_and_trees(rows):
    """The plan is made on the device: a graph is replayed over other lengths, counts and masks, on another stream."""
    import torch
    _, news, lens = _planned(rows, 0, 3000)
    most = 8 * rows
    c = random_cache(np.random.default_rng(1), [3008] * rows, heads=2, d=128, pt=64, row_pages=6000)
    lib = to_library(c)
    q, qd = rounded(np.random.default_rng(2).standard_normal((most, 12, 128)) * 1.5, "float16")
    qg, starts = q.cuda(), i32([0] * (rows + 1))
    mask = torch.zeros((most, 1), dtype=torch.int64, device="cuda")
    out, lse = torch.empty_like(qg), torch.empty((most, 12), device="cuda")
    assert lib.attend_workspace(12, most, 8, masked=True) > LARGE
    lib.attend(qg, starts, mask=mask, max_new=8, out=out, lse=lse)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        lib.attend(qg, starts, mask=mask, max_new=8, out=out, lse=lse)
    for seed in (3, 4, 5):
        rng, news, lens = _planned(rows, seed, 3000)
        seen, _ = od.tree_mask(_parents(rng, news), starts_of(news))
        out.fill_(7)
        lib.lens.copy_(i32(lens))
        starts.copy_(i32(starts_of(news)))
        mask[:sum(news)] = torch.from_numpy(od.mask_words(seen, 1)).cuda()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.current_stream().wait_stream(stream)
        c["lens"] = np.array(lens)
        want, wlse, bound, _ = od.masked_attend(c, qd[:sum(news)], starts_of(news), seen)
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got[:sum(news)] - want) <= bound * (1 + F16_HALF) + F16_HALF * np.abs(want) + 2.0 ** -25)
        np.testing.assert_array_equal(lse[:sum(news)].cpu().numpy() > -np.inf, wlse > -np.inf)
        assert np.all(got[sum(news):] == 7)


def test_planned_calls_on_two_streams_at_once():
    """Each call has its own scratch, and with it its own plan."""
    import torch
    cases = []
    for rows, seed in ((40, 6), (90, 7)):
        rng, news, lens = _planned(rows, seed, 2000)
        c = random_cache(rng, lens, heads=2, d=128, pt=64, row_pages=6000)
        lib = to_library(c)
        q = torch.from_numpy(rng.standard_normal((sum(news), 12, 128))).half().cuda()
        seen, _ = od.tree_mask(_parents(rng, news), starts_of(news))
        mask, starts = torch.from_numpy(od.mask_words(seen, 1)).cuda(), i32(starts_of(news))
        assert lib.attend_workspace(12, sum(news), 8, masked=True) > LARGE
        cases.append((lib, q, starts, mask, lib.attend(q, starts, mask=mask, max_new=8)[0], torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(20):
        for lib, q, starts, mask, _, stream, got in cases:
            with torch.cuda.stream(stream):
                got.append(lib.attend(q, starts, mask=mask, max_new=8)[0])
    torch.cuda.synchronize()
    for _, _, _, _, want, _, got in cases:
        assert all(torch.equal(want, g) for g in got)
