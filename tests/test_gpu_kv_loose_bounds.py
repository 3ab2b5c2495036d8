"""Bounds of a row's new tokens that are far above the tokens given: the same answer as a tight one."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import assert_same, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu


def test_append_of_very_many_rows_with_a_loose_bound():
    """65535 rows of a wide table, a few of them with tokens: no more blocks are launched than the
    tokens can touch."""
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    rows, heads, d, pt = 65535, 64, 64, 256
    lib = KVCache.empty(1, 4, heads, d, rows, 256, page_tokens=pt)
    lib.k.view(torch.uint8).fill_(3)
    before = lib.k.clone()
    rng = np.random.default_rng(1)
    counts = np.zeros(rows, np.int64)
    counts[[0, 40000, 65534]] = [3, 2, 1]
    base = np.zeros(rows, np.int32)
    for page, r in enumerate((0, 40000, 65534)):
        lib.table[r, 0] = page
    k, kd = rounded(rng.standard_normal((6, heads, d)), "float16")
    c = random_cache(rng, [3, 2, 1], heads=heads, d=d, pt=pt)
    for page in range(3):
        c["table"][page, 0] = page
    okv.append(c, kd, kd, [0, 0, 0], starts_of([3, 2, 1]))
    lib.append(k.cuda(), k.cuda(), i32(base), i32(starts_of(counts)), max_new=1 << 30)
    got = lib.k.cpu().numpy().astype(np.float64)
    for page, n in enumerate((3, 2, 1)):
        np.testing.assert_array_equal(got[0, page, :, :n], c["k"][0, page, :, :n])
        np.testing.assert_array_equal(lib.k_scales[0, page, :, 0].cpu().numpy(), c["ks"][0, page, :, 0])
        assert torch.equal(lib.k[0, page, :, 16:], before[0, page, :, 16:])
    assert torch.equal(lib.k[0, 3], before[0, 3])


@pytest.mark.parametrize("bound", [None, 7, 1000, 1 << 30])
def test_append_and_attend(bound):
    """The verification of drafts without a bound, or with one that says nothing."""
    rng = np.random.default_rng(2)
    lens, news = [40, 0, 300, 64], [5, 0, 7, 3]
    total = [a + b for a, b in zip(lens, news)]
    c = random_cache(rng, total, heads=2, d=128, pt=64)
    k, kd = rounded(rng.standard_normal((15, 2, 128)), "float16")
    q, qd = rounded(rng.standard_normal((15, 12, 128)), "float16")
    lib, starts = to_library(c), i32(starts_of(news))
    lib.append(k.cuda(), k.cuda(), i32(lens), starts, max_new=bound)
    okv.append(c, kd, kd, lens, starts_of(news))
    assert_same(lib, c)
    out, _ = lib.attend(q.cuda(), starts, max_new=bound)
    want, _, tol, _ = okv.attend(c, qd, starts_of(news))
    tol = tol * 1.001 + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
