"""How many steps a call of attention or its gradient may have: the host's count
of one sequence of all rows against the definition, tile by tile, around the
limit (needs no GPU)."""

import numpy as np
import pytest

from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t

MOST = 2 ** 31 - 2
P = 0x10000  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


def of_queries(n, nk, tok, causal, cost):
    last = np.minimum((np.arange(-(-n // tok), dtype=np.int64) + 1) * tok, n) - 1  # a tile's last token
    sees = np.maximum(0, last + 1 - n + nk) if causal else np.full_like(last, nk)
    return int((np.maximum(1, -(-sees // 128)) + cost).sum())


def of_keys(n, nk, tok, causal, cost):
    first = np.arange(-(-nk // 128), dtype=np.int64) * 128  # a tile's first key
    unseen = np.maximum(0, first - nk + n) // tok if causal else 0 * first  # by tiles of queries
    return int((np.maximum(1, -(-n // tok) - unseen) + cost).sum())


def steps(n, nk, heads, kv, causal, gradient):
    tok = 128 // (heads // kv)
    if gradient:
        return kv * max(of_queries(n, nk, tok, causal, 2), of_keys(n, nk, tok, causal, 2))
    return kv * of_queries(n, nk, 2 * tok, causal, 4)


def taken(lib, n, nk, heads, kv, causal, gradient):
    """Whether the call gets as far as the handle."""
    q, k = (P, heads * 8, 8), (P, kv * 8, 8)
    shape = (None, 1, n, nk, heads, kv, 8, None, None, None, causal, 1.0)
    if gradient:
        status = lib.tpo_attention_bwd(*shape, *q, *q, *k, *k, *q, P, *q, *k, *k, None)
    else:
        status = lib.tpo_attention(*shape, *q, *k, *k, *q, None, None)
    assert status == (t.TPO_ERR_INVALID_ARG if "handle" in t.tpo_last_error() else t.TPO_ERR_UNSUPPORTED)
    assert status == t.TPO_ERR_INVALID_ARG or "2^31" in t.tpo_last_error()
    return status == t.TPO_ERR_INVALID_ARG


SHAPES = {  # n -> (n, nk), heads, key heads
    "as many keys": (lambda n: (n, n), 1, 1), "of three heads": (lambda n: (n, n), 6, 2),
    "behind others": (lambda n: (n, n + 70001), 10, 2), "a few queries": (lambda n: (777, n), 1 << 14, 1 << 14),
    "more queries": (lambda n: (n + 12345, n), 4, 4), "few keys": (lambda n: (n, 300), 511 * 128, 511),
    "no keys": (lambda n: (n, 0), 2046 * 32, 2046), "no queries": (lambda n: (0, n), 1 << 12, 1 << 12),
}


@pytest.mark.parametrize("gradient", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both ways"])
@pytest.mark.parametrize("name", SHAPES)
def test_what_is_taken(lib, name, causal, gradient):
    shape, heads, kv = SHAPES[name]
    count = lambda n: steps(*shape(n), heads, kv, causal, gradient)  # noqa: E731
    # the limit by bisection, then sizes on either side of it
    lo, hi = 0, 1 << 20
    while count(hi) <= MOST and hi < 1 << 28:
        hi *= 2
    if count(hi) <= MOST:  # a forward call without queries
        assert taken(lib, *shape(hi), heads, kv, causal, gradient)
        return
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if count(mid) <= MOST else (lo, mid)
    sizes = sorted({max(0, lo + d) for d in (-4096, -257, -129, -128, -2, -1, 0, 1, 2, 127, 128, 256, 257, 4096)})
    verdicts = [taken(lib, *shape(n), heads, kv, causal, gradient) for n in sizes]
    assert verdicts == [count(n) <= MOST for n in sizes]
    assert True in verdicts and False in verdicts


@pytest.mark.parametrize("gradient", [False, True], ids=["forward", "gradient"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both ways"])
def test_small_counts(lib, causal, gradient):
    """Counts of short sequences, read off by the most key heads that are taken."""
    for n, nk, group in ((1, 1, 1), (2, 1000, 1), (1000, 3, 1), (700, 700, 3), (129, 1, 128), (5, 130, 128), (0, 900, 1)):
        one = steps(n, nk, group, 1, causal, gradient)
        most = 65535 // group
        if one * most > MOST:
            kv = MOST // one
            assert taken(lib, n, nk, group * kv, kv, causal, gradient)
            assert not taken(lib, n, nk, group * (kv + 1), kv + 1, causal, gradient)
        else:
            assert taken(lib, n, nk, group * most, most, causal, gradient)
