"""The oracle of a step with trees of drafts against closed forms and other formulations."""
import numpy as np
import pytest

import oracle.draft_step as od
import oracle.kv_cache as okv
from _kv_util import random_cache, starts_of


def test_rotation_by_quarter_turns_and_unit_norm():
    x = np.arange(1, 65, dtype=float).reshape(1, 1, 64)
    quarter = [np.pi / 2] * 32
    y, _ = od.norm_rope(x, [1], quarter, norm=False)
    np.testing.assert_allclose(y[0, 0, :32], -x[0, 0, 32:], atol=1e-9)
    np.testing.assert_allclose(y[0, 0, 32:], x[0, 0, :32], atol=1e-9)
    y, _ = od.norm_rope(x, [3], quarter, norm=False, interleaved=True, amplitude=2.0)
    np.testing.assert_allclose(y[0, 0, 0::2], 2 * x[0, 0, 1::2], atol=1e-9)
    np.testing.assert_allclose(y[0, 0, 1::2], -2 * x[0, 0, 0::2], atol=1e-9)
    y, _ = od.norm_rope(x, [0], [], weight=np.full(64, 3.0), eps=0.0)
    assert np.isclose(np.sqrt((y ** 2).mean()), 3.0)


def test_angles_of_far_positions():
    """Modulo a turn, against the sum of the angles of a position's powers of two."""
    for p in (1, 2 ** 20 + 12345, 2 ** 31 - 1, -(2 ** 31)):
        for f in (1.0, 0.01, 1e-6):
            z = np.prod([np.exp(1j * od.angle(2 ** b, f)) for b in range(32) if abs(p) >> b & 1])
            assert abs((z if p > 0 else z.conjugate()) - np.exp(1j * od.angle(p, f))) < 1e-13
            assert abs(np.exp(1j * od.angle(p, f)) - np.exp(1j * p * f)) < abs(p) * 2.0 ** -50


def test_masks_of_a_chain_and_a_star():
    seen, depth = od.tree_mask([-1, 0, 1, 2, -1, 0, 0, 5, 9], [0, 4, 9])
    assert seen[:4] == [{0}, {0, 1}, {0, 1, 2}, {0, 1, 2, 3}] and depth[:4].tolist() == [0, 1, 2, 3]
    assert seen[4:] == [{0}, {0, 1}, {0, 2}, {3}, {4}]  # a parent outside [0, i) makes a root
    assert od.mask_words([{0, 63}, {64, 70}], 2).tolist() == [[1 - 2 ** 63, 0], [0, 65]]


def test_a_chain_is_the_verification_of_a_sequence():
    import oracle
    rng = np.random.default_rng(0)
    logits = rng.standard_normal((6, 5, 40))
    draft = rng.integers(0, 40, (6, 4))
    t = logits.argmax(axis=2)
    for b in range(6):
        draft[b, :b % 5] = t[b, :b % 5]
    want = oracle.spec_decode_verify(logits, draft)
    nodes = np.concatenate([np.zeros((6, 1), int), draft], axis=1)  # node 0: the token before the drafts
    got = od.tree_verify(logits.reshape(30, 40), nodes.ravel(), np.tile(np.arange(-1, 4), 6), np.arange(0, 31, 5), 5)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[3].reshape(6, 5), want[2])
    for b in range(6):
        assert got[2][b].tolist() == list(range(want[0][b] + 1)) + [-1] * (4 - want[0][b])


@pytest.mark.parametrize("window", [0, 5])
def test_a_causal_mask_is_the_causal_attention(window):
    rng = np.random.default_rng(1)
    c = random_cache(rng, [20, 3, 0], heads=1, d=64, pt=16)
    news = [6, 3, 0]
    q = rng.standard_normal((9, 2, 64))
    seen = [{j for j in range(i + 1) if not window or j > i - window} for n in news for i in range(n)]
    depth = [i for n in news for i in range(n)]
    want = okv.attend(c, q, starts_of(news), window=window)
    got = od.masked_attend(c, q, starts_of(news), seen, depth, window=window)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=1e-12)


def test_accepting_a_prefix_is_truncation():
    rng = np.random.default_rng(2)
    c = random_cache(rng, [40, 17, 5], heads=2, d=64, pt=16, layers=2)
    ref = okv.fork(okv.clone(c), [0, 1, 2], [33, 17, 1])
    got = od.accept(okv.clone(c), [[0, 1, 2, -1], [0, -1, -1, -1], [-1, 0, 1, 2]], [0, 10, 11, 15])
    for name in ref:
        np.testing.assert_array_equal(got[name], ref[name])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_accepted_tokens_keep_their_values(fmt):
    """To half a step of the larger scale; exactly where the scale stays."""
    rng = np.random.default_rng(3)
    c = random_cache(rng, [70], heads=1, d=64, pt=16, fmt=fmt)
    old = okv.clone(c)
    path = [0, 3, 4, 20, 38, -1]
    new = od.accept(c, [path], [0, 40])
    assert new["lens"][0] == 35
    src = list(range(30)) + [30 + p for p in path[:5]]
    for name in ("k", "v"):
        was, s0 = okv.values(old, 0, 0, name)
        now, s1 = okv.values(new, 0, 0, name)
        assert np.all(s1 >= s0[src])
        step = 0.5 * s1[:, None] if fmt == "int8" else np.maximum(np.abs(was[src]) / 16, 2.0 ** -10 * s1[:, None])
        assert np.all(np.abs(now - was[src]) <= step * 1.001)
        same = s1 == s0[src]
        assert same.any() and np.array_equal(now[same], was[src][same])


def test_log_probabilities():
    logits = np.log(np.array([[0.5, 0.25, 0.125, 0.125], [0.0, 1.0, 0.0, 0.0]]) + 0.0, where=[[True] * 4, [False, True, False, False]],
                    out=np.full((2, 4), -np.inf)) + 3.0
    got, _ = od.token_logprobs(logits, [3, 0], 3)
    assert np.allclose(got["logprob"], [np.log(0.125), -np.inf]) and np.allclose(got["entropy"], [1.75 * np.log(2), 0])
    assert got["rank"].tolist() == [3, 1] and got["top_ids"].tolist() == [[0, 1, 2], [1, -1, -1]]
    x = np.random.default_rng(4).standard_normal((3, 50))
    got, _ = od.token_logprobs(x, [0, 60, 7], 5)
    p = np.exp(x) / np.exp(x).sum(axis=1, keepdims=True)
    np.testing.assert_allclose(got["entropy"], -(p * np.log(p)).sum(axis=1))
    np.testing.assert_allclose(got["top_logprobs"], -np.sort(-np.log(p), axis=1)[:, :5])
    assert got["rank"][1] == -1 and got["logprob"][1] == -np.inf
