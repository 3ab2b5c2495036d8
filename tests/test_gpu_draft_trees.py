"""Ancestor masks and greedy tree verification against the oracle (whole numbers: equal)."""
import numpy as np
import pytest

import bit_quantized_decode_unpack_gb300 as bqd
import oracle.draft_step as od
from _kv_util import i32, starts_of

pytestmark = pytest.mark.gpu


def random_tree(rng, n, late=0.5):
    """Parents of n nodes: node 0 a root, others below any earlier node."""
    return [-1] + [int(i * (1 - (1 - late) * rng.random())) if rng.random() < 0.7 else int(rng.integers(0, i)) for i in range(1, n)]


def _parents(rng, news):
    return [min(p, i - 1) for n in news for i, p in enumerate(random_tree(rng, n) if n else [])]


@pytest.mark.parametrize("news,words", [([1], 1), ([26, 0, 64, 3], 1), ([130, 7, 65], 3), ([1000, 1], 16), ([200], 1), ([0, 0], 2)])
def test_masks(news, words):
    import torch
    rng = np.random.default_rng(sum(news))
    parents, starts, base = _parents(rng, news), starts_of(news), rng.integers(0, 5000, len(news))
    mask, depth, positions = bqd.tree_mask(i32(parents), i32(starts), words=words, base=i32(base))
    seen, want = od.tree_mask(parents, starts)
    assert mask.dtype == torch.int64
    np.testing.assert_array_equal(mask.cpu().numpy(), od.mask_words(seen, words))
    np.testing.assert_array_equal(depth.cpu().numpy(), want)
    np.testing.assert_array_equal(positions.cpu().numpy(), np.repeat(base, news) + want)


def test_masks_of_a_chain_and_of_wild_parents():
    chain = list(range(-1, 1023))
    mask, depth, none = bqd.tree_mask(i32(chain), i32([0, 1024]), words=16)
    assert none is None and depth.tolist() == list(range(1024))
    np.testing.assert_array_equal(mask.cpu().numpy(), od.mask_words([set(range(i + 1)) for i in range(1024)], 16))
    wild = [5, 7, -2 ** 31, 2 ** 31 - 1, 3, 5, 0, 7]
    mask, depth, _ = bqd.tree_mask(i32(wild), i32([0, 8]))
    seen, want = od.tree_mask(wild, [0, 8])
    np.testing.assert_array_equal(mask.cpu().numpy(), od.mask_words(seen, 1))
    assert depth.tolist() == want.tolist()


@pytest.mark.parametrize("given", ["mask", "depth", "positions"])
def test_masks_of_deep_trees_without_the_other_outputs(given):
    """Walks that leave their group of 128 nodes, each output by itself: nothing may be read from one that is not there."""
    import ctypes
    import torch
    rng = np.random.default_rng(11)
    news = [700, 1, 129, 1024]
    parents = _parents(rng, news)
    parents[-1024:] = [-1] + [i - 1 - (i % 7 == 0 and i > 9) * int(rng.integers(0, 9)) for i in range(1, 1024)]
    starts, base = starts_of(news), rng.integers(-50, 5000, len(news))
    seen, want = od.tree_mask(parents, starts)
    n, p, s, b = len(parents), i32(parents), i32(starts), i32(base)
    out = torch.full((n, 16) if given == "mask" else (n,), -9, dtype=torch.int64 if given == "mask" else torch.int32, device="cuda")
    at = {k: out.data_ptr() if k == given else None for k in ("mask", "depth", "positions")}
    assert bqd.load().bqd_tree_mask(p.data_ptr(), s.data_ptr(), len(news), n, 16, b.data_ptr(), at["mask"], at["depth"],
                                    at["positions"], torch.cuda.current_stream().cuda_stream) == 0
    right = {"mask": lambda: od.mask_words(seen, 16), "depth": lambda: want, "positions": lambda: np.repeat(base, news) + want}
    np.testing.assert_array_equal(out.cpu().numpy(), right[given]())


def test_a_chain_of_many_nodes_takes_time_by_its_length():
    """200000 nodes in one row: 1563 groups of 128 steps, not 2e10 steps."""
    n = 200_000
    mask, depth, pos = bqd.tree_mask(i32(range(-1, n - 1)), i32([0, n]), words=2, base=i32([7]))
    np.testing.assert_array_equal(depth.cpu().numpy(), np.arange(n))
    np.testing.assert_array_equal(pos.cpu().numpy(), np.arange(n) + 7)
    i = np.arange(n)[:, None] - 64 * np.arange(2)[None]  # bits 0 .. i of each word
    want = np.where(i < 0, 0, np.where(i >= 63, -1, (1 << np.clip(i + 1, 0, 63)) - 1)).astype(np.int64)
    np.testing.assert_array_equal(mask.cpu().numpy(), want)


def test_nodes_of_no_row_stay_as_they_are():
    import torch
    mask = torch.full((9, 1), 77, dtype=torch.int64, device="cuda")
    depth, pos = i32([-7] * 9), i32([-8] * 9)
    bqd.tree_mask(i32([-1, 0, 0, -1, 0, 1, 2, 3, 4]), i32([2, 3, 5]), base=i32([10, 20]), mask=mask, depth=depth, positions=pos)
    assert mask.flatten().tolist() == [77, 77, 1, 1, 3, 77, 77, 77, 77]
    assert depth.tolist() == [-7, -7, 0, 0, 1, -7, -7, -7, -7] and pos.tolist() == [-8, -8, 10, 20, 21, -8, -8, -8, -8]
    # starts outside the tokens are cut to them
    bqd.tree_mask(i32([-1, 0, 0]), i32([-5, 2, 2000]), depth=depth[:3], mask=mask[:3])
    assert depth[:3].tolist() == [0, 1, 0]


def _verify(x, drafted, parents, starts, max_path):
    import torch
    best = torch.full((len(parents),), -7, dtype=torch.int32, device="cuda")
    acc, nxt, path = bqd.spec_tree_verify(x, i32(drafted), i32(parents), i32(starts), max_path=max_path, argmax_out=best)
    wa, wn, wp, wt = od.tree_verify(x.double().cpu().numpy(), drafted, parents, starts, max_path)
    np.testing.assert_array_equal(best.cpu().numpy(), wt)
    np.testing.assert_array_equal(path.cpu().numpy(), wp)
    np.testing.assert_array_equal(acc.cpu().numpy(), wa)
    np.testing.assert_array_equal(nxt.cpu().numpy(), wn)
    return wa


def _case(rng, news, v, dtype):
    """Logits whose argmax agrees with a child of most nodes."""
    import torch
    parents, starts = _parents(rng, news), starts_of(news)
    x = rng.standard_normal((sum(news), v)).astype(np.float32)
    drafted = rng.integers(0, v, sum(news))
    for lo, hi in zip(starts[:-1], starts[1:]):
        for i in range(hi - lo):
            kids = [j for j in range(hi - lo) if parents[lo + j] == i]
            if kids and rng.random() < 0.85:
                x[lo + i, drafted[lo + rng.choice(kids)]] = 9.0
    return torch.from_numpy(x).cuda().to(getattr(torch, dtype)), drafted, parents, starts


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("news,v,max_path", [([1], 1, 1), ([26], 20011, 26), ([0, 5, 64, 1], 517, 64), ([70, 33, 100], 1001, 9),
                                             ([300], 64, 300), ([8] * 60, 3001, 2)])
def test_verification(news, v, max_path, dtype):
    rng = np.random.default_rng(sum(news) + v)
    acc = _verify(*_case(rng, news, v, dtype), max_path)
    if max(news) > 20 and max_path > 8:
        assert acc.max() >= 2


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_ties_nan_infinities_and_twins(dtype):
    import torch
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((12, 900)).astype(np.float32)).cuda().to(getattr(torch, dtype))
    parents = [-1, 0, 0, 1, 2, 4, -1, 0, 1, 2, 9, 1]
    drafted = [0, 5, 5, 7, 8, 9, 0, -1, 3, 899, 0, 900]
    x[0, [5, 300, 899]] = 40            # a tie: 5, and of the twins 1 and 2 the lower
    x[1, [0, 7]] = float("inf")         # two infinities: 0
    x[2] = float("nan")
    x[3] = -np.inf                      # all -infinity: 0
    x[4] = -np.inf
    x[4, :5] = float("nan")             # the first that is no NaN: 5
    x[5, 1::2] = float("nan")
    x[6] = float("nan")                 # node 0 of the second row: -1 matches no draft of -1
    x[7, 899] = 50
    x[8, 0] = 50
    x[9] = 0.0
    x[9, ::2] = -0.0                    # equal zeros: 0
    _verify(x, drafted, parents, [0, 6, 12], 6)


@pytest.mark.parametrize("first", [1, 3, 7])
@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_rows_apart_and_off_alignment(first, dtype):
    rng = np.random.default_rng(first)
    x, drafted, parents, starts = _case(rng, [9, 4], 1200, dtype)
    _verify(x[:, first:], [max(0, t - first) for t in drafted], parents, starts, 9)


def test_full_vocabulary():
    rng = np.random.default_rng(9)
    _verify(*_case(rng, [26, 13, 64], 151936, "bfloat16"), 16)


def test_refusals():
    import torch
    x, z = torch.zeros((4, 10), device="cuda"), i32([0, 0, 0, 0])
    s = i32([0, 4])
    bqd.spec_tree_verify(x, z, i32([-1, 0, 1, 2]), s, max_path=4)
    for args, kw in [((x[:3], z, z, s), {}), ((x.double(), z, z, s), {}), ((x, z.long(), z, s), {}), ((x, z, z[:3], s), {}),
                     ((x, z, z, s.long()), {}), ((x, z, z, s[:0]), {}), ((x, z, z, s), {"max_path": 0}),
                     ((x, z, z, s), {"path": i32([[0, 0]])}), ((x, z, z, s), {"accepted": z}), ((x, z.cpu(), z, s), {}),
                     ((x.t(), z, z, s), {})]:
        with pytest.raises(ValueError):
            bqd.spec_tree_verify(*args, **dict({"max_path": 4}, **kw))
    for args, kw in [((z.long(), s), {}), ((z, s.long()), {}), ((z, s), {"words": 0}), ((z, s), {"words": 17}),
                     ((z, s), {"positions": z}), ((z, s), {"base": z}), ((z, s), {"mask": torch.zeros((4, 2), device="cuda").long()}),
                     ((z, s), {"depth": z[:3]})]:
        with pytest.raises(ValueError):
            bqd.tree_mask(*args, **kw)
    acc, nxt, path = bqd.spec_tree_verify(x[:0], z[:0], z[:0], i32([0, 0, 0]), max_path=2)
    assert acc.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and path.tolist() == [[-1, -1], [-1, -1]]
    acc, _, _ = bqd.spec_tree_verify(x[:0], z[:0], z[:0], i32([0]), max_path=2)
    assert acc.shape == (0,)
