"""bqd_qk_norm_rope against the float64 oracle.

Tolerance of a value: the oracle's bound on fp32 arithmetic plus half a unit in the last place of the
output type (2^-11 or 2^-8 of the value, 2^-25 absolute for fp16's subnormals)."""
import numpy as np
import pytest

import bit_quantized_decode_unpack_gb300 as bqd
import oracle.draft_step as od
from _kv_util import BF16_HALF, F16_HALF, i32, rounded

pytestmark = pytest.mark.gpu

THETA = lambda rot, base=10000.0: [base ** (-2.0 * j / rot) for j in range(rot // 2)]  # noqa: E731


def _inputs(rng, tokens, heads, kv_heads, d, dtype):
    """Views of one fused buffer [tokens, heads + 2 kv_heads, d], and their values."""
    t, v = rounded(rng.standard_normal((tokens, heads + 2 * kv_heads, d)) * rng.uniform(0.2, 5, (1, heads + 2 * kv_heads, 1)), dtype)
    return t.cuda(), v


def _check(got, x, positions, freq, dtype, weight, **kw):
    want, bound = od.norm_rope(x, positions, freq, weight, **kw)
    half = F16_HALF if dtype == "float16" else BF16_HALF
    tol = bound * (1 + half) + half * np.abs(want) + 2.0 ** -25
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())


def _run(tokens, heads, kv_heads, d, rot, dtype, wtype, interleaved, first, seed, amplitude=1.0, norm=True, split=True):
    import torch
    rng = np.random.default_rng(seed)
    buf, v = _inputs(rng, tokens, heads, kv_heads, d, dtype)
    w = [None, None]
    if wtype:
        w = [rounded(1 + 0.3 * rng.standard_normal(d), wtype) for _ in range(2)]
    freq = THETA(rot) if rot else []
    pos = (first + np.arange(tokens)).astype(np.int64)
    plan = bqd.QKNormRope(d, freq, q_weight=w[0] and w[0][0].cuda(), k_weight=w[1] and w[1][0].cuda(), eps=1e-5, norm=norm,
                          interleaved=interleaved, amplitude=amplitude)
    q, k = plan(buf[:, :heads], buf[:, heads:heads + kv_heads], i32(pos) if rot else None)
    assert q.shape == (tokens, heads, d) and k.shape == (tokens, kv_heads, d) and q.dtype == buf.dtype
    kw = dict(eps=1e-5, norm=norm, interleaved=interleaved, amplitude=amplitude)
    _check(q, v[:, :heads], pos, freq, dtype, w[0] and w[0][1], **kw)
    _check(k, v[:, heads:heads + kv_heads], pos, freq, dtype, w[1] and w[1][1], **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wtype", [("float16", "float16"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float16", None)])
@pytest.mark.parametrize("tokens,heads,kv_heads,d,rot", [
    (1, 6, 1, 128, 128), (3, 7, 2, 64, 64), (5, 3, 3, 256, 64), (2, 1, 1, 64, 16), (17, 12, 2, 128, 32), (4, 5, 2, 256, 256),
    (2, 9, 4, 128, 112)])
def test_shapes(tokens, heads, kv_heads, d, rot, dtype, wtype, interleaved):
    _run(tokens, heads, kv_heads, d, rot, dtype, wtype, interleaved, 100, tokens + heads)


@pytest.mark.parametrize("first", [0, -3, 131072, 2 ** 31 - 4, -(2 ** 31)])
def test_far_positions(first):
    _run(4, 2, 1, 128, 128, "float16", None, False, first, 5)
    _run(4, 2, 1, 64, 32, "bfloat16", "bfloat16", True, first, 6)


@pytest.mark.parametrize("norm,rot", [(False, 128), (True, 0), (False, 0)])
def test_without_a_norm_or_a_rotation(norm, rot):
    _run(6, 3, 2, 128, rot, "bfloat16", None, False, 9, 7, norm=norm)


def test_amplitude():
    _run(5, 3, 1, 128, 64, "float16", "float32", False, 77, 8, amplitude=1.3)


@pytest.mark.parametrize("tokens", [1000, 5000])
def test_many_tokens(tokens):
    """One warp takes several head groups of a token, or all of them."""
    _run(tokens, 14, 3, 64, 64, "bfloat16", "bfloat16", False, 3, 9)


@pytest.mark.parametrize("layout", ["odd base", "odd stride", "heads first"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_strides(layout, dtype):
    import torch
    rng = np.random.default_rng(10)
    d, tokens, heads = 64, 7, 5
    if layout == "odd base":
        t, v = rounded(rng.standard_normal(tokens * heads * d + 3), dtype)
        q, qv = (x[3:].reshape(tokens, heads, d) for x in (t.cuda(), v))
    elif layout == "odd stride":
        t, v = rounded(rng.standard_normal((tokens, heads, d + 1)), dtype)
        q, qv = t.cuda()[:, :, :d], v[:, :, :d]
    else:
        t, v = rounded(rng.standard_normal((heads, tokens, d)), dtype)
        q, qv = t.cuda().transpose(0, 1), v.transpose(1, 0, 2)
    pos = np.arange(tokens) * 11
    plan = bqd.QKNormRope(d, THETA(d))
    want = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device="cuda")
    out, none = plan(q, None, i32(pos), q_out=want)
    assert out.data_ptr() == want.data_ptr() and none is None
    _check(out, qv, pos, THETA(d), dtype, None)


def test_in_place_and_what_lies_between():
    import torch
    rng = np.random.default_rng(11)
    buf, v = _inputs(rng, 9, 4, 2, 128, "float16")
    plan = bqd.QKNormRope(128, THETA(64))
    q, k = plan(buf[:, :4], buf[:, 4:6], i32(np.arange(9)))
    before = buf.clone()
    plan(buf[:, :4], buf[:, 4:6], i32(np.arange(9)), q_out=buf[:, :4], k_out=buf[:, 4:6])
    assert torch.equal(buf[:, :4], q) and torch.equal(buf[:, 4:6], k) and torch.equal(buf[:, 6:], before[:, 6:])


def test_one_head_for_all_tokens():
    """A broadcast input: strides of 0."""
    import torch
    rng = np.random.default_rng(12)
    t, v = rounded(rng.standard_normal((1, 1, 64)), "float16")
    plan = bqd.QKNormRope(64, THETA(64))
    q, _ = plan(t.cuda().expand(6, 3, 64), None, i32(np.arange(6)))
    _check(q, np.broadcast_to(v, (6, 3, 64)), np.arange(6), THETA(64), "float16", None)
    with pytest.raises(bqd.BqdError):
        plan(q, None, i32(np.arange(6)), q_out=torch.empty((1, 1, 64), dtype=torch.float16, device="cuda").expand(6, 3, 64))


def test_zeros_infinities_and_nan():
    import torch
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 0
    x[1, 0, 5] = float("nan")
    x[2, 0, 5] = float("inf")
    q, _ = bqd.QKNormRope(64, THETA(32))(x, None, i32(np.arange(4)))
    assert torch.all(q[0, 0] == 0) and torch.isnan(q[1, 0]).all() and torch.isnan(q[2, 0, 5])
    assert torch.isfinite(q[:, 1]).all() and torch.isfinite(q[3]).all()


def test_refusals():
    import torch
    plan = bqd.QKNormRope(64, THETA(64), q_weight=torch.ones(64, dtype=torch.float16, device="cuda"))
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    pos = i32([0, 1, 2])
    plan(x, x, pos)
    for args, kw in [((x.float(), x, pos), {}), ((x.bfloat16(), None, pos), {}), ((x, x.bfloat16(), pos), {}), ((x, x[:2], pos), {}),
                     ((x[:, :, :32], None, pos), {}), ((x[0], None, pos), {}), ((x, x, pos.long()), {}), ((x, x, pos[:2]), {}),
                     ((x, x, None), {}), ((x.cpu(), None, pos), {}), ((x, None, pos.cpu()), {}), ((x, None, pos), {"k_out": x}),
                     ((x, x, pos), {"q_out": x[:, :1]}), ((x, x, pos), {"k_out": x[:2]}),
                     ((x.transpose(1, 2).contiguous().transpose(1, 2), None, pos), {})]:
        with pytest.raises(ValueError):
            plan(*args, **kw)
    ones = torch.ones(64, device="cuda")
    for kw in (dict(q_weight=ones[:32]), dict(q_weight=ones.double()), dict(q_weight=ones, k_weight=ones.half()),
               dict(q_weight=ones, norm=False)):
        with pytest.raises(ValueError):
            bqd.QKNormRope(64, THETA(64), **kw)
    q, k = plan(x[:0], x[:0], pos[:0])
    assert q.shape == (0, 2, 64) and k.shape == (0, 2, 64)
    a, _ = bqd.qk_norm_rope(x, None, pos, THETA(64))
    assert a.shape == x.shape


def test_a_plan_of_one_call_on_another_stream_is_read_before_its_memory_is_used_again():
    """qk_norm_rope's own plan is gone when the call returns, the kernel perhaps not begun."""
    import torch
    rng = np.random.default_rng(5)
    buf, v = _inputs(rng, 9, 3, 1, 128, "float16")
    pos, freq, side = np.arange(1000, 1009), THETA(128), torch.cuda.Stream()
    at = i32(pos)
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        q, _ = bqd.qk_norm_rope(buf[:, :3], None, at, freq, stream=side)
        torch.empty(64, dtype=torch.int64, device="cuda").fill_(0x3333333333333333)  # of the size that the plan's have
        side.synchronize()
        _check(q, v[:, :3], pos, freq, "float16", None)
