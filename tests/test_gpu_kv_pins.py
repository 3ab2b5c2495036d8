"""Pages that the caller holds by counts of its own in refs: compaction moves them like any live page,
and says where to."""
import numpy as np
import pytest

import oracle.kv_cache as okv
from _kv_util import assert_same, random_cache, to_library

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pinned", [[], [40], [3, 17, 40, 41]])
def test_a_pinned_page_can_be_followed(pinned):
    import torch
    rng = np.random.default_rng(len(pinned))
    c = random_cache(rng, [300, 0, 90, 41], heads=2, d=64, pt=16, spare=20)
    pages = len(c["refs"])
    free = [p for p in range(pages) if c["refs"][p] == 0]
    held = [p for p in pinned if p in free] + free[-1:]
    for p in held:
        c["refs"][p] = 1                     # no row lists it
    shared = int(c["table"][0, 2])
    c["refs"][shared] += 1                   # a row lists it too
    held.append(shared)
    lib = to_library(c)
    before = lib.k.clone()
    work = torch.full((2 * pages,), -7, dtype=torch.int32, device="cuda")
    new, moved = lib.compact(work=work)
    ref, n = okv.compact(c)
    assert moved.tolist() == [n] and n > 0
    assert_same(new, ref)
    place = work[pages:].tolist()
    live = sum(r > 0 for r in ref["refs"])
    for p in held:
        assert place[p] < live and ref["refs"][place[p]] > 0
        assert torch.equal(new.k[:, place[p]], before[:, p])
    assert sorted(place[int(p)] for p in np.flatnonzero(c["refs"])) == list(range(live))
    again, moved = new.compact()
    assert moved.tolist() == [0]
    assert_same(again, ref)


def test_work_of_another_size_is_refused():
    import torch
    lib = to_library(random_cache(np.random.default_rng(0), [30], heads=1, d=64, pt=16))
    for bad in (torch.empty(2 * lib.pages + 1, dtype=torch.int32, device="cuda"),
                torch.empty(2 * lib.pages, dtype=torch.int64, device="cuda"), torch.empty(2 * lib.pages, dtype=torch.int32)):
        with pytest.raises(ValueError):
            lib.compact(work=bad)
