"""bqd_kv_accept against the oracle: the tables, counts, codes and scales are equal, bit for bit."""
import numpy as np
import pytest

import oracle.draft_step as od
import oracle.kv_cache as okv
from _kv_util import assert_same, i32, random_cache, starts_of, to_library

pytestmark = pytest.mark.gpu


def _run(c, path, starts):
    lib = to_library(c)
    new = lib.accept(i32(path), None if starts is None else i32(starts))
    want = od.accept(c, path, starts)
    assert_same(new, want)
    return new


def _paths(rng, news, width):
    """Rising paths of random lengths, padded with -1."""
    out = np.full((len(news), width), -1)
    for r, n in enumerate(news):
        k = int(rng.integers(0, min(n, width) + 1))
        out[r, :k] = np.sort(rng.choice(n, k, replace=False)) if k else []
    return out


@pytest.mark.parametrize("d,heads,pt,fmt,layers", [(64, 3, 16, "int8", 1), (128, 2, 64, "e4m3", 3), (256, 1, 32, "int8", 2),
                                                  (128, 1, 128, "int8", 1), (64, 1, 256, "e4m3", 2), (256, 2, 16, "e4m3", 1)])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_paths(d, heads, pt, fmt, layers, seed):
    rng = np.random.default_rng(d + pt + seed)
    news = [int(n) for n in rng.integers(0, 70, 7)] + [1, 40, 64]
    lens = [n + int(rng.integers(0, 90)) for n in news]
    lens[2], news[3] = news[2], 0
    c = random_cache(rng, lens, heads=heads, d=d, pt=pt, fmt=fmt, layers=layers)
    _run(c, _paths(rng, news, 70), starts_of(news))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scales_far_apart(fmt):
    rng = np.random.default_rng(5)
    c = random_cache(rng, [100, 64], heads=2, d=64, pt=16, fmt=fmt, spread=8.0)
    _run(c, _paths(rng, [80, 60], 80), [0, 80, 140])


def test_paths_that_end_early():
    rng = np.random.default_rng(6)
    lens = [50, 50, 50, 50, 50, 50, 0, 9]
    c = random_cache(rng, lens, heads=1, d=64, pt=16)
    path = [[0, 5, 5, 6, 7], [3, 2, 9, 10, 11], [-1, 3, 4, 5, 6], [7, 30, 40, 41, 42], [0, 1, 2, 3, 2 ** 31 - 1], [39, 40, 1, 2, 3],
            [0, 1, 2, 3, 4], [0, 2, 4, 6, 8]]
    new = _run(c, path, starts_of([40, 40, 40, 40, 40, 40, 3, 12]))
    assert new.lens.tolist() == [12, 11, 10, 12, 14, 11, 0, 5]


@pytest.mark.parametrize("width", [1, 33, 100])
def test_the_whole_row_and_one_node(width):
    rng = np.random.default_rng(width)
    c = random_cache(rng, [100, 100, 100], heads=1, d=128, pt=32)
    path = np.full((3, width), -1)
    path[0] = np.arange(width)
    path[1] = np.arange(width) + (100 - width)
    path[2, 0] = 99
    _run(c, path, starts_of([100, 100, 100]))


def test_one_token_for_each_row():
    rng = np.random.default_rng(7)
    c = random_cache(rng, [17, 1, 0, 33], heads=1, d=64, pt=16)
    new = _run(c, [[0], [-1], [0], [-1]], None)
    assert new.lens.tolist() == [17, 0, 0, 32]


def test_shared_pages_lose_one_reference_and_other_rows_keep_theirs():
    """Two rows that share a prefix; the nodes are on pages of their own."""
    rng = np.random.default_rng(8)
    c = random_cache(rng, [40, 12], heads=2, d=64, pt=16, spare=12, row_pages=8)
    c = okv.fork(c, [0, 0, 1])
    lib = to_library(c)
    counts = [20, 33, 4]
    base, status = lib.reserve(i32(counts))
    assert okv.reserve(c, counts)[1] == [0, 0] and status.tolist() == [0, 0]
    new = lib.accept(i32([[0, 9, 19], [0, 20, 32], [1, 3, -1]]), i32(starts_of(counts)))
    assert_same(new, od.accept(c, [[0, 9, 19], [0, 20, 32], [1, 3, -1]], starts_of(counts)))
    assert new.lens.tolist() == [43, 43, 14]


def test_wild_pages_and_lengths():
    """Ids outside the pool are read as page 0 and not written; lengths are cut to the table."""
    import torch
    rng = np.random.default_rng(9)
    c = random_cache(rng, [60, 60], heads=1, d=64, pt=16)
    lib = to_library(c)
    lib.table[0, 2] = 10 ** 6
    lib.table[0, 3] = -5
    lib.lens[1] = 10 ** 9
    before = lib.k.clone()
    new = lib.accept(i32([[0, 30, 39], [-1, 0, 0]]), i32([0, 40, 43]))
    torch.cuda.synchronize()
    assert new.lens[0] == 23 and new.lens[1] == lib.row_pages * 16 - 3
    assert sorted((before != lib.k).flatten(1).any(dim=0).nonzero().shape)  # (it ended, and wrote inside the pool alone)


def test_refusals_and_the_given_output():
    rng = np.random.default_rng(10)
    lib = to_library(random_cache(rng, [30, 20], heads=1, d=64, pt=16))
    path, starts = i32([[0, 2], [1, -1]]), i32([0, 4, 7])
    for args in [(path.long(), starts), (path[:1], starts), (path[0], starts), (path[:, :0], starts), (path, starts.long()),
                 (path, starts[:2]), (path.cpu(), starts)]:
        with pytest.raises(ValueError):
            lib.accept(*args)
    with pytest.raises(ValueError):
        lib.accept(path, starts, out=lib)
    out = lib.fork(i32([0, 1]))
    again = to_library(random_cache(np.random.default_rng(10), [30, 20], heads=1, d=64, pt=16))
    got = lib.accept(path, starts, out=out)
    want = again.accept(path, starts)
    assert got is out and got.lens.tolist() == want.lens.tolist() == [28, 18] and got.refs.tolist() == want.refs.tolist()
