"""Pins of the KV cache's oracle: the e4m3 table against its bit fields and
torch's conversion, the append rule on cases worked out by hand, attention
against a direct softmax, and the invariants of the page operations."""
import numpy as np
import pytest
import torch

import oracle.kv_cache as okv
from _kv_util import code_bytes, random_cache, starts_of


def test_e4m3_table():
    v = okv.E4M3
    assert v[0x7E] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)


def test_e4m3_rounding_matches_torch():
    rng = np.random.default_rng(0)
    mids = (okv.E4M3[:126] + okv.E4M3[1:127]) / 2
    x = np.concatenate([mids, -mids, okv.E4M3[:127], rng.standard_normal(4000) * 100, rng.standard_normal(4000) * 0.01])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(okv.encode(x, "e4m3"), want)
    np.testing.assert_array_equal(okv.decode_bytes(code_bytes(want, "e4m3"), "e4m3"), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_by_hand(fmt):
    top = okv.TOP[fmt]
    c = random_cache(np.random.default_rng(1), [3], heads=1, d=64, pt=16, fmt=fmt)
    page = c["table"][0, 0]
    # three tokens in an empty block: the largest magnitude is the top code
    x = np.zeros((3, 1, 64))
    x[1, 0, 5] = -2.0
    x[2, 0, 6] = 1.0
    okv.append(c, x, x, [0], np.array([0, 3]))
    s = np.float32(2.0 * np.float32(1 / top))
    assert c["ks"][0, page, 0, 0] == s
    assert c["k"][0, page, 0, 1, 5] == -top and abs(c["k"][0, page, 0, 2, 6] - top / 2) <= 0.5
    # a larger token: the scale doubles, the earlier codes halve (ties to even)
    c["lens"][0] = 4
    y = np.zeros((1, 1, 64))
    y[0, 0, 0] = 4.0
    okv.append(c, y, y, [3], np.array([0, 1]))
    assert c["ks"][0, page, 0, 0] == np.float32(4.0 * np.float32(1 / top))
    assert c["k"][0, page, 0, 1, 5] == okv.encode(np.array([-top / 2]), fmt)[0]
    # a smaller one leaves them
    before = c["k"].copy()
    okv.append(c, y * 0.25, y * 0.25, [4], np.array([0, 1]))
    np.testing.assert_array_equal(before[0, page, 0, :4], c["k"][0, page, 0, :4])
    # infinities saturate, NaN is 0, and neither sets the scale
    z = np.zeros((1, 1, 64))
    z[0, 0, :4] = [np.inf, -np.inf, np.nan, 1.0]
    okv.append(c, z, z, [0], np.array([0, 1]))
    np.testing.assert_array_equal(c["k"][0, page, 0, 0, :4], [top, -top, 0, top])


def test_append_error_is_half_a_step():
    rng = np.random.default_rng(2)
    c = random_cache(rng, [40], heads=2, d=64, pt=16)
    x = rng.standard_normal((40, 2, 64))
    okv.append(c, x, x, [0], np.array([0, 40]))
    for h in range(2):
        got, s = okv.values(c, 0, h, "k")
        assert np.all(np.abs(got - x[:, h]) <= 0.5 * s[:, None] * (1 + 1e-5))


def test_attend_against_a_direct_softmax():
    rng = np.random.default_rng(3)
    c = random_cache(rng, [21, 0, 5], heads=2, d=64, pt=16)
    news = [3, 2, 7]
    q = rng.standard_normal((12, 4, 64))
    out, lse, _, _ = okv.attend(c, q, starts_of(news), window=4)
    for h in range(4):
        K, V = okv.values(c, 0, h // 2, "k")[0], okv.values(c, 0, h // 2, "v")[0]
        s = torch.from_numpy(K[16:20] @ q[1, h] / 8)  # query 1 of row 0 is at position 19
        np.testing.assert_allclose(out[1, h], torch.softmax(s, 0).numpy() @ V[16:20], rtol=1e-12)
        np.testing.assert_allclose(lse[1, h], torch.logsumexp(s, 0).item(), rtol=1e-12)
    # row 1 is empty; row 2 has more queries than keys: its first two see nothing
    for t in (3, 4, 5, 6):
        assert np.all(out[t] == 0) and np.all(lse[t] == -np.inf)
    assert np.all(np.isfinite(lse[7:]))


def _check_refs(c, pt):
    want = np.zeros(len(c["refs"]), np.int64)
    for r, n in enumerate(c["lens"]):
        for j in range(-(-int(n) // pt)):
            want[c["table"][r, j]] += 1
    np.testing.assert_array_equal(c["refs"], want)


def test_pages_keep_their_counts():
    rng = np.random.default_rng(4)
    pt = 16
    c = random_cache(rng, [5, 32, 17, 0], heads=1, d=64, pt=pt, spare=40, row_pages=6)
    kept = [okv.values(c, r, 0, "k")[0] for r in range(4)]
    f = okv.fork(c, [0, 0, 1, 2, 2, 2, 3, -1, 9], [9, 3, 20, 17, 17, 16, 4, 4, 4])
    _check_refs(f, pt)
    assert f["lens"].tolist() == [5, 3, 20, 17, 17, 16, 0, 0, 0]
    base, status = okv.reserve(f, [1, 1, 0, 2, 2, 2, 1, 0, 0])
    assert status == [0, 0]
    _check_refs(f, pt)
    np.testing.assert_array_equal(base, [5, 3, 20, 17, 17, 16, 0, 0, 0])
    assert len({int(f["table"][r, 0]) for r in (0, 1)}) == 2     # the shared page was copied once
    f["lens"][:] = base
    for r, p in ((0, 0), (1, 0), (2, 1), (3, 2), (4, 2), (5, 2)):
        np.testing.assert_array_equal(okv.values(f, r, 0, "k")[0], kept[p][:base[r]])
    g, moved = okv.compact(okv.fork(f, list(range(9))))
    assert np.all(g["refs"][(g["refs"] > 0).sum():] == 0)
    for r in range(9):
        np.testing.assert_array_equal(okv.values(g, r, 0, "k")[0][:base[r]], kept[[0, 0, 1, 2, 2, 2, 3, 3, 3][r]][:base[r]])


def test_reserve_refuses_as_a_whole():
    c = random_cache(np.random.default_rng(5), [16, 3], heads=1, d=64, pt=16, spare=1, row_pages=2)
    before = okv.clone(c)
    assert okv.reserve(c, [1, 14])[1] == [1, 0]
    assert okv.reserve(c, [17, 1])[1] == [0, 1]
    for n in ("table", "lens", "refs"):
        np.testing.assert_array_equal(before[n], c[n])
