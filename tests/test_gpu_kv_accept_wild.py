"""Acceptance with ids outside the pool in the table: what is read and written, over the whole pools."""
import copy

import numpy as np
import pytest

import oracle.draft_step as od
import oracle.kv_cache as okv
from _kv_util import code_bytes, i32, random_cache, raw, to_library

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,d,layers", [("int8", 64, 2), ("e4m3", 128, 1), ("int8", 256, 1)])
def test_blocks_on_wild_pages_are_read_as_page_0_and_not_written(fmt, d, layers):
    """Tokens 20 .. 59 are nodes, 24 stay: they fill block 1 (a valid page) and block 2 (an id outside the pool), and
    come from these, from a valid page and from another wild id."""
    rng = np.random.default_rng(d)
    c = random_cache(rng, [64, 40], heads=2, d=d, pt=16, fmt=fmt, layers=layers, spread=1.0)
    c["lens"][0] = 60
    pages = c["k"].shape[1]
    path = np.full((2, 24), -1)
    path[0] = [0, 2, 3, 5, 7, 8, 11, 12, 13, 14, 15, 16, 18, 20, 21, 24, 27, 28, 29, 30, 33, 35, 37, 39]
    path[1, :2] = [0, 1]
    starts = [0, 40, 43]
    # the expected pools: a copy of page 0 stands for each wild id, and what it becomes is left out
    want = copy.deepcopy(c)
    for name in ("k", "v", "ks", "vs"):
        want[name] = np.concatenate([want[name]] + [want[name][:, :1]] * 2, axis=1)
    want["refs"] = np.concatenate([want["refs"], [0, 0]])
    want["table"][0, 2], want["table"][0, 3] = pages, pages + 1
    od.accept(want, path, starts)
    lib = to_library(c)
    lib.table[0, 2], lib.table[0, 3] = 10 ** 6, -5
    new = lib.accept(i32(path), i32(starts))
    assert new.lens.tolist() == [44, 39]
    for name in ("k", "v"):
        got, left = raw(getattr(lib, name)), code_bytes(c[name], fmt)
        np.testing.assert_array_equal(okv.decode_bytes(got, fmt), want[name][:, :pages])
        np.testing.assert_array_equal(getattr(lib, name + "_scales").cpu().numpy(), want[name + "s"][:, :pages])
        pages_changed = np.flatnonzero((got != left).any(axis=(0, 2, 3, 4)))
        assert pages_changed.tolist() == [c["table"][0, 1]]
    assert new.table[0, 1:3].tolist() == [c["table"][0, 1], 10 ** 6]
