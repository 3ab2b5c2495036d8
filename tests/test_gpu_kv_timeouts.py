"""Failure detection without a GPU fault: the many-query attention kernel bounds
its waits.  With a limit of 1 ns the first wait for work in flight runs out; the
CTA stops, lets what it issued finish, frees its TMEM, and bqd_device_status
reports it.  The next call is clean."""
import numpy as np
import pytest

import oracle.kv_cache as okv
import bit_quantized_decode_unpack_gb300 as bqd
from _kv_util import F16_HALF, i32, random_cache, rounded, to_library

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(64, 300), (128, 300), (128, 40), (256, 90)])
def test_expired_wait_is_reported_and_the_next_call_is_clean(d, n):
    rng = np.random.default_rng(d)
    c = random_cache(rng, [700], heads=1, d=d, pt=64)
    q, qd = rounded(rng.standard_normal((n, 4, d)), "float16")
    lib, qq, starts = to_library(c), q.cuda(), i32([0, n])
    assert bqd.device_status() == 0
    bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, 1)
    try:
        for _ in range(3):
            lib.attend(qq, starts, max_new=n)
        assert bqd.device_status() == 7
    finally:
        bqd.set_option(bqd.OPT_WAIT_LIMIT_NS, 0)
    out, _ = lib.attend(qq, starts, max_new=n)
    assert bqd.device_status() == 0
    want, _, bound, _ = okv.attend(c, qd, np.array([0, n]))
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound * 1.001 + F16_HALF * np.abs(want) + 2.0 ** -25)
