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


X = C.c_void_p(16)       # never dereferenced: refused before a launch


def strides(*v):
    return (C.c_int64 * 3)(*v)


# (batch, heads, T, d, strides of rows, tokens, heads) whose elements share places
SHARED = [
    (2, 2, 4, 64, (64, 64, 64)),
    (1, 2, 4, 64, (0, 64, 64)),              # token 1 of head 0 on token 0 of head 1
    (1, 4, 4, 64, (0, 128, 64)),             # heads run into the next token
    (1, 2, 4, 64, (0, 64, 192)),             # tokens run into the next head
    (3, 1, 4, 128, (256, 128, 0)),           # tokens run into the next row
    (2, 2, 4, 64, (440, 128, 64)),           # eight elements short of a row
    (2, 2, 64, 64, (2 ** 62, 2 ** 62, 64)),  # and spans past 64 bits
]


@pytest.mark.parametrize("B,n,T,d,st", SHARED)
def test_read_back_outputs_that_share_places(lib, B, n, T, d, st):
    """Every stride is d at least, and two elements lie at one place all the same."""
    c = bg.KV8C(16, 16, 16, 16, 0, B, n, 128, d)
    dense = strides(T * n * d, n * d, d)
    for k, v in ((strides(*st), dense), (dense, strides(*st))):
        assert lib.bloom_op_kv8_read(C.byref(c), X, k, X, v, T, X, None, None, None) == 1
        assert b"strides" in lib.bloom_last_error()


def places(B, n, T, st):
    return [b * st[0] + t * st[1] + h * st[2] for b in range(B) for t in range(T) for h in range(n)]


def test_shared_places_are_what_the_cases_say():
    for B, n, T, d, st in SHARED:
        p = sorted(places(B, n, T, st))
        assert min(b - a for a, b in zip(p, p[1:])) < d
