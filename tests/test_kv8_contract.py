"""Host-side contract of the 8-bit cache operators beside test_kv8_refusals: nothing is
launched here."""
import ctypes as C

import pytest

import bloom_decoder_token_gb300 as bg


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return bg.lib()


def test_wait_bound(lib):
    f = lib.bloom_op_attn_decode_kv8_wait_us
    assert f(-1) == 1 and f(-2 ** 31) == 1 and lib.bloom_last_error()
    assert f(5) == 0 and f(0) == 0
