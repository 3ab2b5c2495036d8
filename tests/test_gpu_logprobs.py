"""bqd_token_logprobs against the float64 oracle: ids and ranks equal, sums within the oracle's bound
(which counts the exponentials' and the additions' roundings)."""
import numpy as np
import pytest

import bit_quantized_decode_unpack_gb300 as bqd
import oracle.draft_step as od
from _kv_util import i32

pytestmark = pytest.mark.gpu
FP32_MAX = 3.4028235e38
DTYPES = ["float16", "bfloat16", "float32"]


def _check(x, tokens, top, **kw):
    """x: a CUDA tensor [rows, V]."""
    r = bqd.token_logprobs(x, i32(tokens), top, **kw)
    want, bound = od.token_logprobs(x.double().cpu().numpy(), tokens, top)
    np.testing.assert_array_equal(r.top_ids.cpu().numpy(), want["top_ids"])
    np.testing.assert_array_equal(r.rank.cpu().numpy(), want["rank"])
    for name, b in bound.items():
        got, w = getattr(r, name).double().cpu().numpy(), want[name]
        w = np.where(w < -FP32_MAX, -np.inf, w)  # beyond fp32, as a difference of its two ends is
        np.testing.assert_array_equal(np.isnan(got), np.isnan(w), err_msg=name)
        np.testing.assert_array_equal(got == -np.inf, w == -np.inf, err_msg=name)
        fine = np.isfinite(w)
        err = np.abs(got[fine] - w[fine])
        assert np.all(err <= b[fine] + 1e-9), (name, float((err / (b[fine] + 1e-9)).max()))
    return r


def _logits(rng, rows, v, dtype, spread=2.5):
    import torch
    return torch.from_numpy((rng.standard_normal((rows, v)) * spread).astype(np.float32)).cuda().to(getattr(torch, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,v,top", [(1, 1, 1), (3, 7, 5), (5, 1000, 20), (2, 4099, 32), (40, 513, 3), (1, 100003, 32),
                                        (700, 3001, 5), (9, 50257, 0), (2, 33, 32)])
def test_shapes(rows, v, top, dtype):
    rng = np.random.default_rng(rows + v)
    tokens = rng.integers(0, v, rows)
    x = _logits(rng, rows, v, dtype)
    tokens[0] = int(x[0].float().argmax())
    _check(x, tokens, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("first", [0, 1, 3, 5])
def test_rows_apart_and_off_alignment(first, dtype):
    rng = np.random.default_rng(first)
    x = _logits(rng, 6, 2011, dtype)[:, first:first + 2000 - first]
    assert not x.is_contiguous()
    _check(x, rng.integers(0, x.shape[1], 6), 20)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [40, 3000, 70001])
def test_masked_values(v, dtype):
    """Rows masked by -infinity, NaN or the type's lowest value, with few, one or none left."""
    import torch
    rng = np.random.default_rng(v)
    x = _logits(rng, 12, v, dtype)
    low = torch.finfo(x.dtype).min
    at = sorted(rng.choice(v, 3, replace=False).tolist())
    for r, fill in enumerate([-np.inf, np.nan, low]):
        for k, kept in enumerate([at, at[1:2], []]):
            row = x[3 * r + k]
            some = row[kept].clone()
            row[:] = fill
            row[kept] = some
    x[9, ::2] = -np.inf
    x[10, ::3] = float("nan")
    x[11, at[0]] = low
    tokens = [at[0], at[1], 0, at[2], at[1], v - 1, at[0], at[0], 5, 1, 3, at[0]]
    r = _check(x, tokens, min(20, v))
    assert r.entropy[2] == 0 and r.entropy[5] == 0 and abs(r.entropy[8].item() - np.log(v)) < 1e-3
    assert r.top_ids[8].tolist() == list(range(min(20, v)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties(dtype):
    """Constant rows, two values, many copies of the largest: the lowest indices win."""
    import torch
    x = torch.zeros((6, 30000), dtype=getattr(torch, dtype), device="cuda")
    x[1] = -7.5
    x[2, 12345:] = 1
    x[3, ::1000] = 2
    x[4, 29990:] = torch.arange(10, device="cuda")
    x[5] = (torch.arange(30000, device="cuda") % 5).to(x.dtype)
    for top in (1, 7, 32):
        _check(x, [0, 29999, 12345, 5000, 29990, 4], top)
    zeros = torch.zeros((1, 600), dtype=x.dtype, device="cuda")
    zeros[0, ::2] = -0.0
    assert _check(zeros, [599], 8).top_ids[0].tolist() == list(range(8))


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_in_order(dtype):
    """Rising and falling rows, and the largest values side by side or far apart: no order of arrival matters."""
    import torch
    rng = np.random.default_rng(1)
    v = 40000
    up = np.sort(rng.standard_normal(v) * 3)
    x = torch.from_numpy(np.stack([up, up[::-1], np.roll(up, 777), rng.permutation(up)]).astype(np.float32)).cuda().to(getattr(torch, dtype))
    _check(x, [v - 1, 0, 776, 11], 32)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_more_candidates_than_the_list_holds(dtype):
    """Large values in the places of few threads only: 4 lanes take every 256th vector."""
    import torch
    e = 4 if dtype == "float32" else 8
    v = 256 * e * 800
    rng = np.random.default_rng(2)
    x = _logits(rng, 1, v, dtype, 0.1)
    big = torch.from_numpy(rng.permutation(800 * 3 * e).astype(np.float32)).cuda() / (800 * 3 * e) + 50
    x.view(800, 256, e)[:, 10:13] = big.view(800, 3, e).to(x.dtype)
    many = x.expand(400, v)  # one CTA a row
    r = bqd.token_logprobs(many.contiguous()[:400], i32([10 * e] * 400), 32)
    want, _ = od.token_logprobs(x.double().cpu().numpy(), [10 * e], 32)
    assert (r.top_ids.cpu().numpy() == want["top_ids"]).all() and (r.rank.cpu().numpy() == want["rank"]).all()
    _check(x, [10 * e], 32)


def test_large_values_and_infinity():
    import torch
    rng = np.random.default_rng(3)
    x = _logits(rng, 6, 5000, "float32")
    x[0] *= 1e30
    x[1, 7] = 3.3e38
    x[2] = -3.4e38
    x[2, 9] = 3.4e38
    x[3, 1234] = float("inf")
    x[4, :] = float("inf")
    x[5, 100] = 80.0
    r = _check(x, [3, 7, 9, 1234, 0, 100], 4)
    assert r.logprob[1] == 0 and r.entropy[1] == 0 and r.logprob[5] == 0
    assert torch.isnan(r.logprob[3]) and r.top_ids[3, 0] == 1234 and r.rank[3] == 0


def test_tokens_outside_the_vocabulary_and_none():
    rng = np.random.default_rng(4)
    x = _logits(rng, 4, 300, "float16")
    _check(x, [-1, 300, 2 ** 31 - 1, 299], 3)
    r = bqd.token_logprobs(x, None, 2)
    full = bqd.token_logprobs(x, i32([1, 2, 3, 4]), 2)
    assert r.logprob is None and r.rank is None
    assert r.entropy.tolist() == full.entropy.tolist() and r.top_ids.tolist() == full.top_ids.tolist()


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_same_answer_every_time_and_for_any_number_of_rows(dtype):
    import torch
    rng = np.random.default_rng(5)
    x = _logits(rng, 400, 20011, dtype)
    tok = i32(rng.integers(0, 20011, 400))
    a, b = bqd.token_logprobs(x, tok, 20), bqd.token_logprobs(x, tok, 20)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    one = bqd.token_logprobs(x[5:6], tok[5:6], 20)  # shared by CTAs of a cluster
    assert torch.equal(one.top_ids[0], a.top_ids[5]) and one.rank[0] == a.rank[5]
    assert abs((one.logprob[0] - a.logprob[5]).item()) < 1e-5


def test_refusals():
    import torch
    x = torch.zeros((3, 50), dtype=torch.float16, device="cuda")
    tok = i32([0, 1, 2])
    for args, kw in [((x.double(), tok), {}), ((x[0], tok), {}), ((x, tok.long()), {}), ((x, tok[:2]), {}), ((x, tok.cpu()), {}),
                     ((x, tok, 33), {}), ((x, tok, -1), {}), ((x.t(), tok), {}), ((x[:, :0], tok), {}),
                     ((x[:1].expand(3, 50), tok), {})]:
        with pytest.raises(ValueError):
            bqd.token_logprobs(*args, **kw)
    r = bqd.token_logprobs(x[:0], tok[:0], 4)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 4)


def test_ties_at_the_end_of_the_longest_row():
    """The last indices of the largest V: positions behind the row pass 2^31 in the ordered search for ties."""
    import torch
    v = 2 ** 31 - 1024
    x = torch.full((1, v), -1.0, dtype=torch.bfloat16, device="cuda")
    x[0, v - 2000:] = 1.0
    r = bqd.token_logprobs(x, i32([v - 1]), 32)
    assert r.top_ids[0].tolist() == list(range(v - 2000, v - 1968)) and r.rank.tolist() == [1999]
    assert bool((r.top_logprobs == r.logprob).all())
