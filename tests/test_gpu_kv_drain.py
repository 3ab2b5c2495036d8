"""Waits of the many-query attention kernel that run out at any point of a call.  With limits from
one nanosecond to a tenth of a millisecond some roles of some CTAs give up while the products of
others are in flight; every CTA lets what it issued finish before it frees its TMEM and leaves.  A
call whose waits all came through has the right answer; another is reported by bqd_device_status;
and the calls after it are clean."""
import numpy as np
import pytest

import oracle.kv_cache as okv
import bit_quantized_decode_unpack_gb300 as bqd
from _kv_util import F16_HALF, i32, random_cache, rounded, starts_of, to_library

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 7


@pytest.mark.parametrize("d,grp,lens,news,max_len", [
    (128, 6, [900, 400], [300, 200], 0),     # several query tiles: converted once
    (64, 6, [900, 400], [300, 200], 500),    # the first row is longer than planned
    (128, 6, [2500, 900], [30, 40], 0),      # one query tile, CTAs share its keys
    (64, 4, [700], [20], 0),                 # one tile of 128 rows
    (256, 4, [900, 130], [200, 40], 0),
])
def test_waits_that_run_out_anywhere(d, grp, lens, news, max_len):
    rng = np.random.default_rng(d + len(lens))
    c = random_cache(rng, lens, heads=2, d=d, pt=64)
    q, qd = rounded(rng.standard_normal((sum(news), 2 * grp, d)), "float16")
    lib, qq, starts = to_library(c), q.cuda(), i32(starts_of(news))
    want, _, bound, _ = okv.attend(c, qd, starts_of(news))
    tol = bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25

    def call():
        out, _ = lib.attend(qq, starts, max_new=max(news), max_len=max_len)
        status = bqd.device_status()
        return status, np.all(np.abs(out.double().cpu().numpy() - want) <= tol)

    assert call() == (OK, True)
    statuses = []
    for limit in (1, 300, 1000, 2000, 4000, 7000, 12000, 19000, 25000, 50000, 100000):
        for _ in range(3):
            bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, limit)
            try:
                status, right = call()
            finally:
                bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, 0)
            assert status == TIMEOUT or (status == OK and right)
            statuses.append(status)
            assert call() == (OK, True)
    assert statuses[0] == TIMEOUT
