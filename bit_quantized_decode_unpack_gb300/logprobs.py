"""Log probabilities of given tokens, with entropy, rank and the most likely alternatives."""
from __future__ import annotations

import ctypes
from typing import Any, NamedTuple

from . import _check
from . import drafts as _drafts
from . import kv_cache as _kv

MAX_TOP = 32


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; None where there were no tokens."""
    logprob: Any        # fp32 [rows]
    entropy: Any        # fp32 [rows]
    rank: Any           # int32 [rows]
    top_ids: Any        # int32 [rows, top]
    top_logprobs: Any   # fp32 [rows, top]


def declare(lib):
    """Argument types of the entry point."""
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.bqd_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp]
    lib.bqd_token_logprobs.restype = i32


def token_logprobs(logits, tokens=None, top: int = 0, *, stream=None) -> TokenLogprobs:
    """Log probabilities under softmax(logits), in one pass over them (bqd_token_logprobs).

    logits fp16, bf16 or fp32 [rows, V] (rows may be apart); tokens int32 [rows].  logprob and rank
    (0: the most likely) are those of ``tokens`` (an id outside [0, V): -infinity and -1), entropy is
    in nats, and the ``top`` most likely tokens come in order, ties by the lower id.  Values of
    -infinity or NaN have probability 0 and are not listed (ids of -1 end a short list)."""
    torch = _drafts._bind()
    kind, rows, v, stride = _drafts._logits(logits)
    dev = logits.device
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be in [0, {MAX_TOP}], got {top}")
    if tokens is not None:
        _kv._dense(tokens, "tokens", torch.int32, (rows,), dev)
    on = _drafts._here(dev, stream)
    if on is not None:
        with on:
            return token_logprobs(logits, tokens, top)
    f32, i32, empty = torch.float32, torch.int32, torch.empty
    entropy = empty(rows, dtype=f32, device=dev)
    logprob = rank = None
    if tokens is not None:
        logprob, rank = empty(rows, dtype=f32, device=dev), empty(rows, dtype=i32, device=dev)
    ids, lps = empty((rows, top), dtype=i32, device=dev), empty((rows, top), dtype=f32, device=dev)
    at = _drafts._at
    _check("bqd_token_logprobs", _drafts._lib.bqd_token_logprobs(
        logits.data_ptr(), kind, stride, rows, v, at(tokens), top, at(logprob), entropy.data_ptr(), at(rank), ids.data_ptr(),
        lps.data_ptr(), _kv._raw_stream(dev.index)))
    return TokenLogprobs(logprob, entropy, rank, ids, lps)
