"""The masked entry point by its own name: a call without a mask is refused, as the C function does."""
import pytest

import bit_quantized_decode_unpack_gb300 as bqd


class Cache:
    """Records what the function hands on."""

    def attend(self, *args, **kw):
        return args, kw


def test_a_call_without_a_mask_is_refused():
    with pytest.raises(ValueError):
        bqd.kv_attend_masked(Cache(), "q", "starts", max_new=3)
    with pytest.raises(ValueError):
        bqd.kv_attend_masked(Cache(), "q", mask=None)


def test_everything_else_is_handed_on():
    args, kw = bqd.kv_attend_masked(Cache(), "q", "starts", mask="m", depth="d", layer=2, window=9, max_new=3, out="o", lse="l")
    assert args == ("q", "starts")
    assert kw == dict(mask="m", depth="d", layer=2, window=9, max_new=3, out="o", lse="l")
    args, kw = bqd.kv_attend_masked(Cache(), "q", mask="m")
    assert args == ("q", None) and kw["mask"] == "m"
