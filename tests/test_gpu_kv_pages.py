"""Page operations against the oracle's sequential rules, bit for bit."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import assert_same, i32, random_cache, to_library

pytestmark = pytest.mark.gpu


def _random_state(seed, rows=13, pt=32, layers=2, fmt="int8", spare=30, longest=200, d=64):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest, rows)
    lens[rng.integers(0, rows)] = 0
    return rng, random_cache(rng, lens.tolist(), heads=2, d=d, pt=pt, layers=layers, fmt=fmt, spare=spare,
                             row_pages=longest // pt + 3)


@pytest.mark.parametrize("seed", range(6))
def test_a_life_of_a_cache(seed):
    """Forks, reservations, cuts and compactions in turn."""
    pt = [16, 32, 64, 128, 256, 16][seed]
    rng, c = _random_state(seed, pt=pt, fmt="e4m3" if seed % 2 else "int8", spare=200)
    lib = to_library(c)
    for step in range(8):
        rows = len(c["lens"])
        what = rng.integers(0, 4)
        if what == 0:
            parents = rng.integers(-1, rows + 1, int(rng.integers(1, 24)))
            keep = rng.integers(0, 220, len(parents)) if rng.random() < 0.7 else None
            c = okv.fork(c, parents, keep)
            lib = lib.fork(i32(parents), None if keep is None else i32(keep))
        elif what == 1:
            counts = rng.integers(0, 3, rows) * rng.integers(0, 20, rows)
            base, status = okv.reserve(c, counts)
            got, st = lib.reserve(i32(counts))
            np.testing.assert_array_equal(got.cpu().numpy(), base)
            assert st.tolist() == status
        elif what == 2:
            keep = rng.integers(0, 220, rows)
            c = okv.fork(c, range(rows), keep)
            lib = lib.truncate(i32(keep))
        else:
            c, moved = okv.compact(c)
            lib, m = lib.compact()
            assert m.item() == moved
        assert_same(lib, c)


def test_beams_share_then_copy():
    """Children of one parent: the last page is copied for all but one."""
    rng, c = _random_state(20, rows=3, pt=16, spare=40)
    c["lens"][:] = [37, 16, 5]
    c = random_cache(rng, [37, 16, 5], heads=2, d=64, pt=16, layers=2, spare=40, row_pages=12)
    lib = to_library(c)
    parents = [0, 0, 0, 1, 1, 2, 2, 0]
    c, lib = okv.fork(c, parents), lib.fork(i32(parents))
    assert_same(lib, c)
    base, _ = okv.reserve(c, [1] * 8)
    got, status = lib.reserve()          # the default: one token each
    np.testing.assert_array_equal(got.cpu().numpy(), base)
    assert status.tolist() == [0, 0]
    assert_same(lib, c)
    last = lib.table.cpu().numpy()[[0, 1, 2, 7], 2]
    assert len(set(last.tolist())) == 4


def test_rows_left_out_keep_the_shared_page():
    c = random_cache(np.random.default_rng(21), [20], heads=1, d=64, pt=16, spare=9, row_pages=3)
    lib = to_library(c)
    c, lib = okv.fork(c, [0, 0, 0]), lib.fork(i32([0, 0, 0]))
    for counts in ([0, 2, 2], [1, 0, 0], [0, 12, 0]):
        base, st = okv.reserve(c, counts)
        got, status = lib.reserve(i32(counts))
        np.testing.assert_array_equal(got.cpu().numpy(), base)
        assert_same(lib, c)


def test_pins_of_the_caller_count():
    """A page that the caller holds a reference to is neither written to nor freed."""
    c = random_cache(np.random.default_rng(22), [20, 30], heads=1, d=64, pt=16, spare=5, row_pages=4)
    c["refs"][c["table"][0, 1]] += 1
    lib = to_library(c)
    okv.reserve(c, [1, 1])
    lib.reserve()
    assert_same(lib, c)
    c, lib = okv.fork(c, [-1, -1]), lib.fork(i32([-1, -1]))
    assert c["refs"].sum() == 1
    assert_same(lib, c)
    c, moved = okv.compact(c)
    lib, _ = lib.compact()
    assert c["refs"][0] == 1
    assert_same(lib, c)


def test_failed_reservations_change_nothing():
    c = random_cache(np.random.default_rng(23), [16, 3, 40], heads=1, d=64, pt=16, spare=2, row_pages=4)
    lib = to_library(c)
    for counts, status in (([1, 14, 25], [0, 1]), ([17, 14, 9], [2, 0]), ([0, 100, 0], [0, 1]), ([2 ** 31 - 1, 0, 0], [0, 1])):
        base, st = okv.reserve(c, counts)
        got, s = lib.reserve(i32(counts))
        assert s.tolist() == st == status
        assert torch_all(got == -1)
        assert_same(lib, c)
    # negative counts are none
    got, s = lib.reserve(i32([-5, 0, 0]))
    assert s.tolist() == [0, 0]
    assert_same(lib, c)


def torch_all(t):
    return bool(t.all().item())


@pytest.mark.parametrize("rows", [1, 1025, 4096])
def test_many_rows(rows):
    rng = np.random.default_rng(rows)
    c = random_cache(rng, [int(x) for x in rng.integers(0, 40, rows)], heads=1, d=64, pt=16, layers=1, spare=3 * rows,
                     row_pages=5)
    lib = to_library(c)
    parents = rng.integers(0, rows, rows)
    c, lib = okv.fork(c, parents), lib.fork(i32(parents))
    counts = rng.integers(0, 30, rows)
    base, st = okv.reserve(c, counts)
    got, s = lib.reserve(i32(counts))
    assert s.tolist() == st == [0, 0]
    np.testing.assert_array_equal(got.cpu().numpy(), base)
    assert_same(lib, c)
    c, _ = okv.compact(c)
    lib, _ = lib.compact()
    assert_same(lib, c)


def test_large_pool_scan():
    """More pages than one pass of the scan covers (4096), free ones only at the end."""
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    lib = KVCache.empty(1, 10001, 1, 64, 3, 40, page_tokens=16)
    lib.refs[:9990] = 1
    base, st = lib.reserve(i32([100, 0, 17]))
    assert st.tolist() == [0, 0] and base.tolist() == [0, 0, 0]
    assert lib.table[0, :7].tolist() == list(range(9990, 9997)) and lib.table[2, :2].tolist() == [9997, 9998]
    assert lib.lens.tolist() == [100, 0, 17]
    lib.refs[:9990:3] = 0
    new, moved = lib.compact()
    live = int((lib.refs > 0).sum())
    assert moved.item() == int((lib.refs[live:] > 0).sum()) and torch.all(new.refs[live:] == 0)
    assert int((new.refs > 0).sum()) == live


def test_copy_pages():
    c = random_cache(np.random.default_rng(24), [64] * 6, heads=3, d=256, pt=32, layers=3)
    lib = to_library(c)
    src, dst = [0, 3, 5, -1, 10 ** 7, 2], [1, 4, 2, 6, 7, 10 ** 7]
    lib.copy_pages(i32(src), i32(dst))
    for a, b in zip(src[:3], dst[:3]):
        for n in ("k", "v", "ks", "vs"):
            c[n][:, b] = c[n][:, a]
    assert_same(lib, c)
    lib.copy_pages(i32([]), i32([]))


def test_given_siblings_are_reused():
    c = random_cache(np.random.default_rng(25), [30, 10], heads=1, d=64, pt=16)
    lib = to_library(c)
    other = lib.fork(i32([0, 1]))
    third = lib.fork(i32([1, 0]), out=other)
    assert third is other
    assert_same(third, okv.fork(c, [1, 0]))
    with pytest.raises(ValueError):
        lib.fork(i32([0, 1, 1]), out=other)
    with pytest.raises(ValueError):
        lib.compact(out=lib)
