"""Time of ancestor masks over the length of a chain."""
import pytest

import bit_quantized_decode_unpack_gb300 as bqd
from _kv_util import i32

pytestmark = pytest.mark.gpu


def _ms(n):
    import torch
    parents, starts = i32(range(-1, n - 1)), i32([0, n])
    mask, depth, _ = bqd.tree_mask(parents, starts, words=2)
    best = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(3):
            bqd.tree_mask(parents, starts, words=2, mask=mask, depth=depth)
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b) / 3)
    return min(best)


def test_a_chains_time_grows_with_its_length():
    """Four times the nodes take four times the steps; walks to the root would take sixteen times as many."""
    short, long = _ms(50_000), _ms(200_000)
    assert long < 8 * short, (short, long)
