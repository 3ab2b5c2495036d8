"""Rows with fewer tokens than their tree has nodes: how attention under masks and acceptance number them."""
import numpy as np
import pytest

import oracle.draft_step as od
from _kv_util import F16_HALF, assert_same, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,n", [(9, 12), (1, 2), (16, 40), (0, 3)])
@pytest.mark.parametrize("pages", [None, 60000])
def test_attention_counts_from_the_rows_end_and_acceptance_from_its_start(length, n, pages):
    import torch
    rng = np.random.default_rng(length + n)
    news, lens = [n, 5], [length, 30]
    c = random_cache(rng, lens, heads=1, d=64, pt=16, row_pages=pages)
    lib = to_library(c)
    # node i sees itself alone: the last `length` nodes see token i - (n - length), the others nothing
    seen = [{i} for m in news for i in range(m)]
    q, qd = rounded(rng.standard_normal((sum(news), 2, 64)), "float16")
    out, lse = lib.attend(q.cuda(), i32(starts_of(news)), mask=torch.from_numpy(od.mask_words(seen, 1)).cuda(), max_new=max(news))
    want, wlse, bound, lbound = od.masked_attend(c, qd, starts_of(news), seen)
    np.testing.assert_array_equal(wlse[:n, 0] > -np.inf, np.arange(n) >= n - length)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    np.testing.assert_array_equal(lse > -np.inf, wlse > -np.inf)
    some = wlse > -np.inf
    assert np.all(np.abs(lse[some] - wlse[some]) <= lbound[some] + 2.0 ** -22 * np.abs(wlse[some]))
    assert np.all(np.abs(out - want) <= bound * (1 + F16_HALF) + F16_HALF * np.abs(want) + 2.0 ** -25)
    # acceptance: node j is token j, up to the row's last one
    path = np.full((2, n), -1)
    path[0, :(n + 1) // 2] = np.arange(0, n, 2)
    path[1, :2] = [0, 3]
    new = lib.accept(i32(path), i32(starts_of(news)))
    assert new.lens.tolist() == [len(range(0, length, 2)), 27]
    assert_same(new, od.accept(c, path, starts_of(news)))
