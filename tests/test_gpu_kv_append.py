"""bqd_kv_append against the oracle: codes and scales bit for bit."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import assert_same, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, fmt, D, heads, page, lens before, new tokens
    ("float16", "int8", 128, 2, 64, [0, 1, 15, 16, 17, 63, 64, 100], [1] * 8),
    ("bfloat16", "e4m3", 128, 3, 16, [0, 7, 31], [1, 1, 1]),
    ("float16", "e4m3", 64, 1, 32, [5, 0, 40, 0], [3, 0, 60, 33]),
    ("bfloat16", "int8", 256, 2, 128, [130, 3], [1, 200]),
    ("float16", "int8", 64, 5, 256, [250], [300]),
    ("bfloat16", "int8", 128, 8, 16, [0], [1]),
    ("float16", "e4m3", 256, 1, 64, [9, 0, 33], [17, 1, 0]),
]


def _setup(rng, dtype, fmt, d, heads, pt, lens, news, magnitude=1.0):
    total = [a + b for a, b in zip(lens, news)]
    c = random_cache(rng, total, heads=heads, d=d, pt=pt, fmt=fmt)
    shape = (sum(news), heads, d)
    k, kd = rounded(rng.standard_normal(shape) * magnitude, dtype)
    v, vd = rounded(rng.standard_normal(shape) * magnitude * 0.3, dtype)
    return c, k, kd, v, vd


@pytest.mark.parametrize("dtype,fmt,d,heads,pt,lens,news", CASES)
@pytest.mark.parametrize("magnitude", [1.0, 30.0, 1e-4])
def test_matches_the_oracle(dtype, fmt, d, heads, pt, lens, news, magnitude):
    rng = np.random.default_rng(len(lens) * d + heads)
    c, k, kd, v, vd = _setup(rng, dtype, fmt, d, heads, pt, lens, news, magnitude)
    lib = to_library(c)
    starts = None if set(news) == {1} else starts_of(news)
    st = None if starts is None else i32(starts)
    for _ in range(2):  # appending the same tokens again changes nothing
        lib.append(k.cuda(), v.cuda(), i32(lens), st, max_new=max(news))
        if _ == 0:
            okv.append(c, kd, vd, lens, starts)
        assert_same(lib, c)


def test_one_token_at_a_time_matches_and_stays_close():
    rng = np.random.default_rng(9)
    n, d = 50, 128
    c, k, kd, v, vd = _setup(rng, "float16", "int8", d, 2, 16, [0], [n], 1.0)
    grow = (1 + np.arange(n) / 5.0)[:, None, None]  # every token raises the scale
    k, kd = rounded(kd * grow, "float16")
    lib = to_library(c)
    for t in range(n):
        okv.append(c, kd[t:t + 1], vd[t:t + 1], [t], np.array([0, 1]))
        lib.append(k[t:t + 1].cuda(), v[t:t + 1].cuda(), i32([t]))
    assert_same(lib, c)
    got, s = okv.values(c, 0, 0, "k")
    # each of up to 15 growths rounds a code once more, by half a step of a scale that only grew
    assert np.all(np.abs(got - kd[:, 0]) <= 8 * s[:, None])


def test_strided_views_and_unaligned_bases():
    import torch
    rng = np.random.default_rng(10)
    lens, news = [3, 20], [9, 30]
    c, k, kd, v, vd = _setup(rng, "float16", "int8", 64, 2, 32, lens, news)
    t = sum(news)
    for token, offset in ((2 * 2 * 64 + 8, 0), (2 * 2 * 64 + 3, 0), (2 * 2 * 64 + 8, 1)):
        buf = torch.full((t * token + 64,), 777.0, dtype=torch.float16, device="cuda")
        kk = buf[offset:].as_strided((t, 2, 64), (token, 64, 1))
        vv = buf[offset + 128:].as_strided((t, 2, 64), (token, 64, 1))
        kk.copy_(k), vv.copy_(v)
        want = okv.clone(c)
        okv.append(want, kd, vd, lens, starts_of(news))
        lib = to_library(c)
        lib.append(kk, vv, i32(lens), i32(starts_of(news)))
        assert_same(lib, want)
    # heads and tokens swapped in memory, one value broadcast over the tokens
    kk = k.cuda().permute(1, 0, 2).contiguous().permute(1, 0, 2)
    vv = v.cuda()[:1].expand(t, 2, 64)
    want = okv.clone(c)
    okv.append(want, kd, np.broadcast_to(vd[:1], vd.shape), lens, starts_of(news))
    lib = to_library(c)
    lib.append(kk, vv, i32(lens), i32(starts_of(news)))
    assert_same(lib, want)


@pytest.mark.parametrize("dtype,fmt", [("float16", "int8"), ("bfloat16", "e4m3"), ("float16", "e4m3"), ("bfloat16", "int8")])
def test_extreme_values(dtype, fmt):
    rng = np.random.default_rng(11)
    c, k, kd, v, vd = _setup(rng, dtype, fmt, 64, 2, 16, [4], [40])
    big = 65504.0 if dtype == "float16" else 3.0e38
    x = kd.copy()
    x[0, 0, :6] = [np.inf, -np.inf, np.nan, big, -big, 0]
    x[13, 1, :] = np.nan          # a token of NaN
    x[12:28, 0, :] = 0            # a block of zeros
    x[30, 1, 3] = 6e-8            # subnormal in fp16
    x[36:, 1] = np.inf
    k, kd = rounded(x, dtype)
    v, vd = rounded(np.zeros_like(vd), dtype)
    lib = to_library(c)
    lib.append(k.cuda(), v.cuda(), i32([4]), i32([0, 40]))
    okv.append(c, kd, vd, [4], np.array([0, 40]))
    assert_same(lib, c)


def test_skipped_rows_layers_and_bounds():
    import torch
    rng = np.random.default_rng(12)
    c = random_cache(rng, [20, 20, 20], heads=2, d=64, pt=16, layers=3, row_pages=2)
    k, kd = rounded(rng.standard_normal((24, 2, 64)), "float16")
    starts = np.array([0, 8, 16, 24], np.int32)
    want = okv.clone(c)
    okv.append(want, kd, kd, [12, -1, 12], np.array([0, 8, 16, 24]), layer=1)
    # row 2's tokens 12 .. 19 stand; row 0 keeps max_new = 8
    lib = to_library(c)
    lib.append(k.cuda(), k.cuda(), i32([12, -1, 12]), i32(starts), layer=1, max_new=8)
    assert_same(lib, want)
    # past the table's capacity (32 tokens): the tokens that fit are stored
    want = okv.clone(c)
    okv.append(want, kd[:2], kd[:2], [30, -1, -1], np.array([0, 2, 2, 2]))
    lib = to_library(c)
    lib.append(k.cuda(), k.cuda(), i32([30, 32, 1 << 30]), i32(starts))
    # only row 0 fits two tokens
    assert_same(lib, want)
    # an id outside the pool is skipped
    lib = to_library(c)
    lib.table[0, 0] = 10 ** 6
    lib.table[1, 0] = -1
    before = lib.k.clone()
    lib.append(k.cuda()[:3], k.cuda()[:3], i32([0, 0, -1]))
    torch.cuda.synchronize()
    assert torch.equal(before, lib.k)
    # nothing to do
    lib.append(k.cuda()[:0], k.cuda()[:0], i32([0, 0, 0]), i32([0, 0, 0, 0]))
