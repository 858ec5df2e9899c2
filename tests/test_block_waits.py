"""The bound of the block operators' device-side waits: the option, and calls
whose waits run out."""

import pytest

from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


@pytest.mark.parametrize("value,word", [(0, "wait_timeout_ms"), (-1, "wait_timeout_ms"), (600001, "wait_timeout_ms"),
                                        (1, "handle"), (600000, "handle")])
def test_option_range(lib, value, word):
    assert lib.tpo_block_set_opt(None, b"wait_timeout_ms", value) == t.TPO_ERR_INVALID_ARG
    assert word in t.tpo_last_error()


@pytest.mark.gpu
def test_option_round_trip(cuda_ok, lib):
    b = t.tpo_block_create(0)
    try:
        assert t.tpo_block_get_opt(b, "wait_timeout_ms") == 2000
        t.tpo_block_set_opt(b, "wait_timeout_ms", 50)
        assert t.tpo_block_get_opt(b, "wait_timeout_ms") == 50
        assert t.tpo_block_get_opt(b, "path") == 0 and t.tpo_block_get_opt(b, "split") == 0
    finally:
        t.tpo_block_destroy(b)
