"""bqd_kv_attend against the float64 oracle.

Tolerance of each output: the oracle's bound on fp32 scores and fp16 weights
plus half a unit in the last place of the output type (2^-11 or 2^-8 of the
value, 2^-25 absolute for fp16's subnormals)."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import BF16_HALF, F16_HALF, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu


def _run(c, q, news=None, **kw):
    lib = to_library(c)
    starts = None if news is None else i32(starts_of(news))
    if news is not None:
        kw.setdefault("max_new", max(news))
    out, lse = lib.attend(q.cuda(), starts, **kw)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _compare(c, q, qd, news, dtype, layer=0, scale=None, window=0, **kw):
    got, glse = _run(c, q, news, layer=layer, scale=scale, window=window, **kw)
    want, lse, bound, lbound = okv.attend(c, qd, None if news is None else starts_of(news), layer, scale, window)
    half = F16_HALF if dtype == "float16" else BF16_HALF
    tol = bound * (1 + half) + half * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())
    seen = lse > -np.inf
    np.testing.assert_array_equal(glse > -np.inf, seen)
    assert np.all(np.abs(glse[seen] - lse[seen]) <= lbound[seen] + 2.0 ** -22 * np.abs(lse[seen]))
    assert np.all(got[~seen] == 0)
    return got, glse


DECODE = [
    # dtype, fmt, D, kv heads, group, page, lens
    ("float16", "int8", 128, 2, 6, 64, [1, 15, 16, 17, 64, 65, 700]),
    ("bfloat16", "int8", 128, 1, 1, 16, [0, 1, 2, 33]),
    ("float16", "e4m3", 64, 2, 7, 32, [129, 0, 5]),
    ("bfloat16", "e4m3", 256, 2, 6, 128, [300, 1, 127]),
    ("float16", "int8", 256, 1, 16, 256, [513, 40]),
    ("bfloat16", "int8", 64, 3, 8, 64, [2000]),
    ("float16", "int8", 128, 1, 33, 64, [90, 31]),
]


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens", DECODE)
@pytest.mark.parametrize("window", [0, 1, 50])
def test_one_token_for_each_row(dtype, fmt, d, hk, grp, pt, lens, window):
    rng = np.random.default_rng(d + grp)
    c = random_cache(rng, lens, heads=hk, d=d, pt=pt, fmt=fmt)
    q, qd = rounded(rng.standard_normal((len(lens), hk * grp, d)) * 1.5, dtype)
    _compare(c, q, qd, None, dtype, window=window)


RAGGED = [
    ("float16", "int8", 128, 2, 6, 64, [40, 0, 5, 300], [5, 0, 5, 3]),
    ("bfloat16", "e4m3", 64, 1, 7, 32, [70, 33], [70, 17]),
    ("bfloat16", "int8", 256, 1, 6, 16, [100, 17], [9, 1]),
    ("float16", "int8", 128, 1, 4, 64, [3, 2], [8, 2]),          # more queries than keys
    ("float16", "e4m3", 128, 2, 5, 128, [260, 129, 1], [130, 129, 1]),
    ("bfloat16", "int8", 128, 1, 6, 64, [400, 150], [150, 150]),
]


@pytest.mark.parametrize("dtype,fmt,d,hk,grp,pt,lens,news", RAGGED)
@pytest.mark.parametrize("window", [0, 1, 37])
def test_several_tokens_for_each_row(dtype, fmt, d, hk, grp, pt, lens, news, window):
    rng = np.random.default_rng(sum(lens))
    c = random_cache(rng, lens, heads=hk, d=d, pt=pt, fmt=fmt)
    q, qd = rounded(rng.standard_normal((sum(news), hk * grp, d)) * 1.5, dtype)
    _compare(c, q, qd, news, dtype, window=window)


@pytest.mark.parametrize("max_len", [0, 1, 40, 5000])
@pytest.mark.parametrize("news", [[1, 1], [6, 3], [200, 64]])
def test_any_hint_of_the_length_gives_the_same_answer(max_len, news):
    rng = np.random.default_rng(3)
    c = random_cache(rng, [900, 64], heads=1, d=128, pt=64, row_pages=64)
    q, qd = rounded(rng.standard_normal((sum(news), 6, 128)), "float16")
    _compare(c, q, qd, news, "float16", max_len=max_len)


@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (128, "int8"), (256, "int8")])
@pytest.mark.parametrize("window", [0, 900])
def test_few_queries_far_behind_in_a_long_row(d, fmt, window):
    """A chunk of queries whose tiles' keys several CTAs share, beside an empty row, a short one and
    queries before the first key."""
    rng = np.random.default_rng(16)
    lens, news = [2500, 0, 9, 1700], [40, 30, 33, 64]
    c = random_cache(rng, lens, heads=1, d=d, pt=64, fmt=fmt)
    q, qd = rounded(rng.standard_normal((sum(news), 3, d)), "bfloat16")
    _compare(c, q, qd, news, "bfloat16", window=window)
    got = _run(c, q, news, window=window)
    again = _run(c, q, news, window=window, max_len=1000)  # the first row is longer than planned
    want, _, bound, _ = okv.attend(c, qd, starts_of(news), 0, None, window)
    assert np.all(np.abs(again[0] - want) <= bound * 1.01 + BF16_HALF * np.abs(want) + 2.0 ** -25)
    np.testing.assert_array_equal(got[0], _run(c, q, news, window=window)[0])


@pytest.mark.parametrize("heads", [1, 4])
@pytest.mark.parametrize("grp,news", [(4, [1] * 6), (6, [3, 1, 4, 0, 2, 2])])
def test_shares_of_mixed_lengths(heads, grp, news):
    """Rows of very different lengths, so that the equal shares cut units at every place, and rows
    shorter than what a unit costs."""
    rng = np.random.default_rng(17)
    lens = [2600, 5, 0, 700, 17, 1300]
    c = random_cache(rng, lens, heads=heads, d=64, pt=16, row_pages=4000)  # planned long: shares
    q, qd = rounded(rng.standard_normal((sum(news), heads * grp, 64)), "float16")
    _compare(c, q, qd, None if set(news) == {1} else news, "float16")


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_scales_far_apart(dtype, n):
    """Blocks whose V (and K) scales differ by many orders of magnitude, zero blocks among them."""
    rng = np.random.default_rng(4)
    c = random_cache(rng, [400], heads=2, d=64, pt=16, spread=0.0)
    shape = c["vs"].shape
    c["vs"] = (c["vs"] * 10.0 ** rng.uniform(-20, 3, shape)).astype(np.float32)
    c["ks"] = (c["ks"] * 10.0 ** rng.uniform(-6, 0, shape)).astype(np.float32)
    for b in range(0, 25, 5):  # what an appended block of zeros holds
        page = c["table"][0, b]
        c["v"][0, page], c["vs"][0, page] = 0, np.float32(2.0 ** -80 / 127)
        c["k"][0, page], c["ks"][0, page] = 0, np.float32(2.0 ** -80 / 127)
    q, qd = rounded(rng.standard_normal((n, 6, 64)), dtype)
    _compare(c, q, qd, [n], dtype)
    # every stored value zero
    c["v"][:] = 0
    c["vs"][:] = np.float32(2.0 ** -80 / 127)
    got, _ = _run(c, q, [n])
    assert np.all(got == 0)


@pytest.mark.parametrize("n", [1, 130])
def test_sharp_scores_growing_along_the_row(n):
    """Scores that keep rising, so that every tile replaces the running reference."""
    rng = np.random.default_rng(5)
    c = random_cache(rng, [640], heads=1, d=64, pt=64, spread=0.0)
    ramp = (np.arange(640 // 16) + 1.0) / 10
    for b in range(40):
        page = c["table"][0, b // 4]
        c["ks"][0, page, 0, b % 4] = ramp[b]
    c["k"] = np.abs(c["k"])
    q, qd = rounded(np.abs(rng.standard_normal((n, 3, 64))), "float16")
    _compare(c, q, qd, [n], "float16")


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("magnitude", [1e-6, 1e4, 3e37, 1e-38])
def test_queries_of_any_magnitude(n, magnitude):
    rng = np.random.default_rng(6)
    dtype = "bfloat16" if not 1e-7 < magnitude < 6e4 else "float16"
    c = random_cache(rng, [200], heads=1, d=128, pt=64)
    x = rng.standard_normal((n, 6, 128)).clip(-3, 3) * magnitude
    x[:, 1] = 0
    q, qd = rounded(x, dtype)
    _compare(c, q, qd, [n], dtype, scale=float(0.1 / magnitude) if magnitude > 1e-30 else 1e30)


@pytest.mark.parametrize("n", [1, 140])
def test_infinities_and_nan_in_queries_stay_in_their_rows(n):
    rng = np.random.default_rng(7)
    c = random_cache(rng, [300], heads=2, d=64, pt=32)
    x = rng.standard_normal((n, 8, 64))
    q, qd = rounded(x, "float16")
    clean, _ = _run(c, q, [n])
    x[n // 2, 3, 7] = np.nan
    x[n - 1, 6, 1] = np.inf
    q, qd = rounded(x, "float16")
    got, _ = _run(c, q, [n])
    hit = np.zeros((n, 8), bool)
    hit[n // 2, 3] = hit[n - 1, 6] = True
    assert np.all(np.isnan(got[n // 2, 3]))
    np.testing.assert_array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("n", [1, 20, 150])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_what_lies_past_the_row_is_not_read(n, fmt):
    """Stale codes (e4m3 NaN among them), NaN scales and wild page ids past a row's end change nothing."""
    import torch
    rng = np.random.default_rng(8)
    c = random_cache(rng, [165], heads=1, d=128, pt=64, fmt=fmt)
    q, _ = rounded(rng.standard_normal((n, 6, 128)), "float16")
    clean, lse = _run(c, q, [n])
    lib = to_library(c)
    kept = np.zeros(len(c["refs"]), bool)
    kept[c["table"][0, :3]] = True
    for t in (lib.k_scales, lib.v_scales):
        t[0, torch.from_numpy(~kept).cuda()] = float("nan")
        t[0, int(c["table"][0, 2]), 0, 3] = float("nan")       # the last page's last block: tokens 176 .. 191
    for t in (lib.k, lib.v):
        b = t.view(torch.uint8)
        b[0, torch.from_numpy(~kept).cuda()] = 0x7F
        b[0, int(c["table"][0, 2]), 0, 165 - 128:] = 0x7F       # within the last block too
    lib.table[0, 3:] = 12345678
    out, lse2 = lib.attend(q.cuda(), i32([0, n]), max_new=n)
    np.testing.assert_array_equal(out.double().cpu().numpy(), clean)
    np.testing.assert_array_equal(lse2.double().cpu().numpy(), lse)


@pytest.mark.parametrize("n", [1, 9, 160])
def test_strides_of_queries(n):
    import torch
    rng = np.random.default_rng(9)
    c = random_cache(rng, [222], heads=2, d=64, pt=64)
    q, qd = rounded(rng.standard_normal((n, 6, 64)), "bfloat16")
    clean, lse = _run(c, q, [n])
    for token, head, offset in ((6 * 64 + 128, 64, 0), (6 * 64 + 1, 64, 0), (6 * 72, 72, 8), (6 * 65, 65, 3)):
        buf = torch.full((n * token + 600,), 9e4, dtype=torch.bfloat16, device="cuda")
        view = buf[offset:].as_strided((n, 6, 64), (token, head, 1))
        view.copy_(q)
        out, lse2 = to_library(c).attend(view, i32([0, n]), max_new=n)
        np.testing.assert_array_equal(out.double().cpu().numpy(), clean)
        np.testing.assert_array_equal(lse2.double().cpu().numpy(), lse)


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(10)
    c = random_cache(rng, [3000, 17, 900], heads=2, d=128, pt=64)
    for news in ([1, 1, 1], [40, 2, 300]):
        q, _ = rounded(rng.standard_normal((sum(news), 12, 128)), "bfloat16")
        a = _run(c, q, news)
        for _ in range(3):
            b = _run(c, q, news)
            np.testing.assert_array_equal(a[0], b[0])
            np.testing.assert_array_equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 9, 150])
def test_a_scale_of_zero_is_a_mean(n):
    rng = np.random.default_rng(15)
    c = random_cache(rng, [210, n], heads=1, d=64, pt=32)
    q, qd = rounded(rng.standard_normal((2 * n, 2, 64)), "float16")
    _compare(c, q, qd, [n, n], "float16", scale=0.0, window=100)


def test_layers_scale_given_outputs_and_untouched_rows():
    import torch
    rng = np.random.default_rng(11)
    c = random_cache(rng, [50, 20], heads=2, d=64, pt=32, layers=3)
    q, qd = rounded(rng.standard_normal((9, 4, 64)), "float16")
    _compare(c, q, qd, [4, 5], "float16", layer=2, scale=-0.3)
    lib = to_library(c)
    out = torch.full((9, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((9, 4), 5.0, device="cuda")
    # queries 0 and 7, 8 belong to no row; a row computes max_new of its queries
    lib.attend(q.cuda(), i32([1, 3, 7]), max_new=3, out=out, lse=lse)
    untouched = [0, 6, 7, 8]
    assert torch.all(out[untouched] == 5) and torch.all(lse[untouched] == 5) and torch.all(out[1:6] != 5)


def test_another_stream_and_shared_pages():
    import torch
    rng = np.random.default_rng(12)
    c = random_cache(rng, [500, 80], heads=2, d=128, pt=64)
    c["table"][1] = c["table"][0, :c["table"].shape[1]]
    c["lens"][1] = 321
    q, qd = rounded(rng.standard_normal((2, 8, 128)), "float16")
    want, _ = _compare(c, q, qd, None, "float16")
    lib, qq = to_library(c), q.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [lib.attend(qq, stream=s)[0] for _ in range(8)]
    with torch.cuda.stream(s):
        outs.append(lib.attend(qq)[0])
    s.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.double().cpu().numpy(), want)


def test_in_a_cuda_graph():
    import torch
    rng = np.random.default_rng(13)
    c = random_cache(rng, [130, 60], heads=1, d=128, pt=64)
    lib = to_library(c)
    q = torch.zeros((2, 6, 128), dtype=torch.float16, device="cuda")
    lib.attend(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = lib.attend(q)
    for seed in range(3):
        x, _ = rounded(np.random.default_rng(seed).standard_normal((2, 6, 128)), "float16")
        q.copy_(x)
        lib.lens.copy_(i32([130 - seed, 60]))
        graph.replay()
        want, _ = lib.attend(q)
        assert torch.equal(out, want)


@pytest.mark.parametrize("n", [1, 130])
def test_pool_beyond_32_bit_offsets(n):
    """Pages whose codes lie past 4 GB of the pool: append, then attend."""
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    rng = np.random.default_rng(14)
    d, heads, pt, pages = 128, 8, 256, 20000
    lib = KVCache.empty(1, pages, heads, d, 1, 4, page_tokens=pt)
    assert lib.k.numel() > 2 ** 32
    high = [19999, 16500, 16385]
    lib.table[0, :3] = i32(high)
    lib.refs[i32(high).long()] = 1
    length = 600
    lib.lens[0] = length
    c = random_cache(rng, [length], heads=heads, d=d, pt=pt)
    k, kd = rounded(rng.standard_normal((length, heads, d)), "float16")
    v, vd = rounded(rng.standard_normal((length, heads, d)), "float16")
    okv.append(c, kd, vd, [0], np.array([0, length]))
    lib.append(k.cuda(), v.cuda(), i32([0]), i32([0, length]))
    for j, page in enumerate(high[:2]):
        got = lib.k[0, page].cpu().numpy().astype(np.float64)
        np.testing.assert_array_equal(got, c["k"][0, c["table"][0, j]])
    q, qd = rounded(rng.standard_normal((n, heads, d)), "float16")
    out, _ = lib.attend(q.cuda(), i32([0, n]), max_new=n)
    want, _, bound, _ = okv.attend(c, qd, np.array([0, n]))
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)
