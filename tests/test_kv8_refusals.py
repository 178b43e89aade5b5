"""What the 8-bit cache operators and the log probabilities refuse, on the host:
nothing is launched, so no GPU is needed; and the plain forms' own closed cases."""
import ctypes as C

import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import kv8_plain as plain

X = C.c_void_p(16)       # never dereferenced: every call here is refused before a launch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return bg.lib()


def desc(**kw):
    f = dict(k=16, v=16, k_scale=16, v_scale=16, codes=0, batch=2, n_kv=2, max_seq=64, d=64)
    f.update(kw)
    return bg.KV8C(*[f[n] for n, _ in bg.KV8C._fields_])


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
              (dict(k=24), 1), (dict(v=17), 1), (dict(codes=2), 1), (dict(codes=-1), 1), (dict(d=96), 2),
              (dict(d=0), 2), (dict(batch=0), 1), (dict(n_kv=0), 1), (dict(max_seq=0), 1),
              (dict(batch=70000), 1), (dict(max_seq=2 ** 30 + 1), 1)]
ST = (C.c_int64 * 3)(64 * 2 * 4, 128, 64)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):
    c = desc(**kw)
    assert lib.bloom_op_kv8_write(C.byref(c), X, ST, X, ST, 4, X, None, None, None, None) == status
    assert lib.bloom_op_kv8_read(C.byref(c), X, ST, X, ST, 4, X, None, None, None) == status
    assert lib.bloom_op_attn_decode_kv8(C.byref(c), X, X, X, X, 1, 2, X, X, 1 << 30, None, None) == status
    assert lib.bloom_op_attn_decode_kv8_workspace(C.byref(c), 1, 2) == 0
    assert lib.bloom_last_error()


def test_null_cache(lib):
    assert lib.bloom_op_kv8_write(None, X, ST, X, ST, 4, X, None, None, None, None) == 1
    assert lib.bloom_op_kv8_read(None, X, ST, X, ST, 4, X, None, None, None) == 1
    assert lib.bloom_op_attn_decode_kv8(None, X, X, X, X, 1, 2, X, X, 0, None, None) == 1


def test_write_and_read_refusals(lib):
    c = C.byref(desc())
    w, r = lib.bloom_op_kv8_write, lib.bloom_op_kv8_read
    odd = (C.c_int64 * 3)(512, 128, 60)
    neg = (C.c_int64 * 3)(512, -128, 64)
    off = C.c_void_p(24)
    for k, ks, v, vs, T, start in [(None, ST, X, ST, 4, X), (X, None, X, ST, 4, X), (X, ST, None, ST, 4, X),
                                   (X, ST, X, None, 4, X), (X, ST, X, ST, 4, None), (off, ST, X, ST, 4, X),
                                   (X, ST, off, ST, 4, X), (X, odd, X, ST, 4, X), (X, ST, X, odd, 4, X),
                                   (X, neg, X, ST, 4, X), (X, ST, X, ST, -1, X), (X, ST, X, ST, 65, X)]:
        assert w(c, k, ks, v, vs, T, start, None, None, None, None) == 1
        assert r(c, k, ks, v, vs, T, start, None, None, None) == 1
    # outputs that would lie on one another; sources may
    for bad in [(0, 128, 64), (512, 0, 64), (512, 128, 0), (512, 32, 64)]:
        assert r(c, X, (C.c_int64 * 3)(*bad), X, ST, 4, X, None, None, None) == 1
        assert r(c, X, ST, X, (C.c_int64 * 3)(*bad), 4, X, None, None, None) == 1
    # nothing to do is no error, whatever the pointers
    assert w(c, None, None, None, None, 0, None, None, None, None, None) == 0
    assert r(c, None, None, None, None, 0, None, None, None, None) == 0
    big = desc(batch=65535, n_kv=65535, max_seq=1 << 20)
    assert w(C.byref(big), X, ST, X, ST, 4, X, None, None, None, None) == 1


def test_attention_refusals(lib):
    c = C.byref(desc())
    f = lib.bloom_op_attn_decode_kv8
    big = 1 << 30
    assert f(c, None, X, X, X, 1, 2, X, X, big, None, None) == 1
    assert f(c, X, None, X, X, 1, 2, X, X, big, None, None) == 1
    assert f(c, X, X, X, None, 1, 2, X, X, big, None, None) == 1
    assert f(c, X, X, X, X, 1, 2, None, X, big, None, None) == 1
    assert f(c, C.c_void_p(18), X, X, X, 1, 2, X, X, big, None, None) == 1
    assert f(c, X, X, X, X, 1, 2, C.c_void_p(18), X, big, None, None) == 1
    assert f(c, X, X, X, X, 1, 2, X, C.c_void_p(24), big, None, None) == 1
    assert f(c, X, X, X, X, 1, 3, X, X, big, None, None) == 1       # heads not a multiple
    assert f(c, X, X, X, X, 1, 0, X, X, big, None, None) == 1
    assert f(c, X, X, X, X, 0, 2, X, X, big, None, None) == 1
    assert f(c, X, X, X, X, 33, 2, X, X, big, None, None) == 2
    huge = desc(batch=1 << 12, n_kv=16, max_seq=1 << 15)       # 2^31 slots
    assert f(C.byref(huge), X, X, X, X, 1, 16, X, X, big, None, None) == 2
    c = C.byref(desc(max_seq=1000))                            # rows that may be cut need a workspace
    need = lib.bloom_op_attn_decode_kv8_workspace(c, 1, 2)
    assert need > 0
    if need:
        assert f(c, X, X, X, X, 1, 2, X, None, 0, None, None) == 1
        assert f(c, X, X, X, X, 1, 2, X, X, need - 1, None, None) == 1


def test_logprobs_refusals(lib):
    f = lib.bloom_op_logprobs
    ok = dict(z=X, B=1, V=8, ld=8, tok=X, J=1, lp=X, ent=X, top=1, ids=X, lps=X)
    for kw in [dict(z=None), dict(B=-1), dict(B=65536), dict(V=0), dict(ld=7), dict(J=-1), dict(tok=None),
               dict(lp=None), dict(top=-1), dict(top=33), dict(ids=None), dict(lps=None)]:
        a = dict(ok, **kw)
        assert f(a["z"], a["B"], a["V"], a["ld"], a["tok"], a["J"], a["lp"], a["ent"], a["top"], a["ids"],
                 a["lps"], None) == 1, kw
    assert f(None, 0, 8, 8, None, 0, None, None, 0, None, None, None) == 0   # no rows


def cpu_cache(**kw):
    a = dict(batch=2, n_kv=2, max_seq=40, d=64, device="cpu")
    a.update(kw)
    return bg.KV8.empty(**a)


def refused(f):
    with pytest.raises(bg.BloomError) as e:
        f()
    assert e.value.status in (1, 2)


def test_python_checks(lib):
    kv = cpu_cache()
    assert kv.k_scale.shape == (2, 2, 2) and cpu_cache(codes=torch.float8_e4m3fn).k.dtype is torch.float8_e4m3fn
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    st = torch.zeros(2, dtype=torch.int32)
    i32 = torch.int32
    # host tensors are refused
    refused(lambda: bg.op_kv8_write(kv, x, x, st))
    refused(lambda: bg.op_kv8_read(kv, st, 3))
    refused(lambda: bg.op_attn_decode_kv8(x, kv, torch.zeros(2, 40, dtype=i32), None, st))
    refused(lambda: bg.op_logprobs(torch.zeros(2, 8)))
    # types, shapes and strides, before the device is looked at
    refused(lambda: bg.op_kv8_write(kv, x.float(), x, st))
    refused(lambda: bg.op_kv8_write(kv, x[0], x, st))
    refused(lambda: bg.op_kv8_write(kv, x[:, :2], x, st))
    refused(lambda: bg.op_kv8_write(kv, x, x.transpose(2, 3).contiguous().transpose(2, 3), st))
    refused(lambda: bg.op_kv8_read(kv, st, -1))
    refused(lambda: bg.op_attn_decode_kv8(x[0, 0], kv, torch.zeros(2, 40, dtype=i32), None, st))
    refused(lambda: bg.op_attn_decode_kv8(x.transpose(1, 2), kv, torch.zeros(2, 40, dtype=i32), None, st))
    refused(lambda: bg.op_logprobs(torch.zeros(2, 8, dtype=torch.bfloat16)))
    refused(lambda: bg.op_logprobs(torch.zeros(8)))
    refused(lambda: bg.op_logprobs(torch.zeros(8, 2).t()))
    refused(lambda: bg.op_logprobs(torch.zeros(2, 8), top=33))
    refused(lambda: bg.op_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)))
    refused(lambda: bg.op_logprobs(torch.zeros(2, 8), torch.zeros(3, 1, dtype=i32)))
    for bad in [kv._replace(k=kv.k.float()), kv._replace(k=kv.k[0]), kv._replace(v=kv.v[:, :, :39]),
                kv._replace(v=kv.v.to(torch.float8_e4m3fn)), kv._replace(k_scale=kv.k_scale[:, :, :1]),
                kv._replace(v_scale=kv.v_scale.double()), kv._replace(k=kv.k.transpose(1, 2))]:
        refused(lambda: bad.c())


# ------------------------------------------------- the plain forms' own closed cases
def test_plain_rounding_is_the_types():
    y = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.05, 0.05, 20001)])
    t = torch.from_numpy(y).float()
    assert np.array_equal(plain.round_codes(t.double().numpy(), torch.float8_e4m3fn),
                          t.to(torch.float8_e4m3fn).double().numpy())


def test_plain_scale_bounds():
    for codes, top in plain.LARGEST.items():
        for amax in [1e-45, 1e-38, 0.3, 1.0, top, np.nextafter(top, 999), 3e38]:
            s = plain.scale_of(amax, codes)
            assert amax <= top * s and (s == 2.0 ** -126 or amax > top * s / 2)


def test_plain_logprobs_closed_forms():
    lp, ent, ids, top = plain.logprobs(np.zeros((1, 4)), np.array([[2, -1, 4]]), 3)
    assert np.allclose(lp[0, 0], -np.log(4)) and lp[0, 1] == 0 and np.isnan(lp[0, 2])
    assert np.allclose(ent, np.log(4)) and ids.tolist() == [[0, 1, 2]]
    lp, ent, ids, top = plain.logprobs(np.full((1, 3), -np.inf), np.array([[1]]), 2)
    assert lp[0, 0] == -np.inf and ent[0] == 0 and ids.tolist() == [[-1, -1]]
