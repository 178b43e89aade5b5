"""What the 4-bit weights' operators and filtered sampling refuse, on the host: nothing is
launched, so no GPU is needed; and the plain forms' own closed cases."""
import ctypes as C

import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import sample_plain
import w4_plain as plain

X = C.c_void_p(16)       # never dereferenced: every call here is refused before a launch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return bg.lib()


def desc(**kw):
    f = dict(tiles=16, n=48, k=512, group=64)
    f.update(kw)
    return C.byref(bg.W4C(*[f[n] for n, _ in bg.W4C._fields_]))


BAD_WEIGHTS = [(dict(tiles=None), 1), (dict(tiles=24), 1), (dict(group=0), 2), (dict(group=16), 2), (dict(group=-64), 2),
               (dict(group=256), 2), (dict(n=0), 1), (dict(n=-1), 1), (dict(k=0), 1), (dict(k=-8), 1), (dict(k=12), 2),
               (dict(n=2 ** 30 + 1), 1), (dict(k=2 ** 24 + 8), 1)]


@pytest.mark.parametrize("kw,status", BAD_WEIGHTS)
def test_bad_weights(lib, kw, status):
    w = desc(**kw)
    assert lib.bloom_op_w4_quantize(X, 1 << 25, w, None) == status
    assert lib.bloom_op_w4_read(w, X, 1 << 25, None) == status
    for M in (0, 1, 9):
        assert lib.bloom_op_linear_w4(w, X, 1 << 25, M, None, 0, X, 1 << 31, 0, X, 1 << 40, None, None) == status
        assert lib.bloom_op_linear_w4_workspace(w, M) == 0
    assert lib.bloom_last_error()


def test_null_weights(lib):
    assert lib.bloom_op_w4_quantize(X, 512, None, None) == 1
    assert lib.bloom_op_w4_read(None, X, 512, None) == 1
    assert lib.bloom_op_linear_w4(None, X, 512, 1, None, 0, X, 48, 0, None, 0, None, None) == 1


def test_bytes(lib):
    f = lib.bloom_w4_bytes
    assert f(16, 256, 32) == 2048 + 256 and f(16, 256, 64) == 2048 + 128 and f(16, 256, 128) == 2048 + 64
    assert f(17, 264, 64) == 4 * f(16, 256, 64) and f(1, 8, 64) == f(16, 256, 64)
    assert f(2 ** 30, 2 ** 24, 128) == 2 ** 26 * 2 ** 16 * 2112
    for bad in [(0, 8, 64), (-1, 8, 64), (16, 0, 64), (16, 12, 64), (16, 8, 16), (16, 8, 0), (2 ** 30 + 1, 8, 64),
                (16, 2 ** 24 + 8, 64)]:
        assert f(*bad) == 0


def test_quantize_and_read_refusals(lib):
    for p, ld in [(None, 512), (C.c_void_p(18), 512), (C.c_void_p(24), 512), (X, 511), (X, 504), (X, 516), (X, 0), (X, -512)]:
        assert lib.bloom_op_w4_quantize(p, ld, desc(), None) == 1
        assert lib.bloom_op_w4_read(desc(), p, ld, None) == 1


def test_linear_refusals(lib):
    f, big = lib.bloom_op_linear_w4, 1 << 40
    ok = dict(x=X, ldx=512, M=12, bias=None, epi=0, y=X, ldy=48, f32=0, ws=X, wn=big, flag=None)
    odd = C.c_void_p
    for kw in [dict(x=None), dict(x=odd(24)), dict(ldx=504), dict(ldx=516), dict(ldx=-512), dict(M=-1), dict(M=2 ** 20 + 1),
               dict(bias=odd(17)), dict(epi=-1), dict(epi=3), dict(y=None), dict(y=odd(17)), dict(y=odd(18), f32=1),
               dict(ldy=47), dict(ldy=-48), dict(flag=odd(18)), dict(ws=None), dict(ws=odd(24)), dict(wn=0),
               dict(wn=lib.bloom_op_linear_w4_workspace(desc(), 12) - 1)]:
        a = dict(ok, **kw)
        assert f(desc(), a["x"], a["ldx"], a["M"], a["bias"], a["epi"], a["y"], a["ldy"], a["f32"], a["ws"], a["wn"],
                 a["flag"], None) == 1, kw
    assert f(desc(), None, 0, 0, None, 0, None, 0, 0, None, 0, None, None) == 0       # no tokens
    assert lib.bloom_op_linear_w4_wait_ns(-1) == 1 and lib.bloom_op_linear_w4_wait_ns(0) == 0


def test_workspace_sizes(lib):
    f = lib.bloom_op_linear_w4_workspace
    assert [f(desc(), M) for M in (-1, 0, 1, 8, 2 ** 20 + 1)] == [0] * 5
    last = 0
    for M in (9, 16, 17, 33, 65, 1000, 2 ** 20):
        need = f(desc(), M)
        assert need >= M * 512 * 2 and need >= last
        last = need
    assert f(desc(k=2 ** 24), 2 ** 20) > 2 ** 45          # no wrap at 32 bits


def test_sampling_refusals(lib):
    f = lib.bloom_op_sample_filtered
    ok = dict(z=X, B=2, V=8, ld=8, t=None, k=None, p=None, m=None, u=X, J=1, out=X)
    odd = C.c_void_p(18)
    for kw in [dict(z=None), dict(z=odd), dict(B=-1), dict(B=65536), dict(V=0), dict(V=-8), dict(V=2 ** 22 + 1, ld=2 ** 23), dict(J=2 ** 30 + 1), dict(ld=7), dict(ld=-8), dict(t=odd),
               dict(k=odd), dict(p=odd), dict(m=odd), dict(u=None), dict(u=odd), dict(J=-1), dict(out=None), dict(out=odd)]:
        a = dict(ok, **kw)
        assert f(a["z"], a["B"], a["V"], a["ld"], a["t"], a["k"], a["p"], a["m"], a["u"], a["J"], a["out"], None) == 1, kw
    assert f(None, 0, 8, 8, None, None, None, None, None, 1, None, None) == 0          # no rows
    assert f(None, 2, 8, 8, None, None, None, None, None, 0, None, None) == 0          # no draws


def refused(f):
    with pytest.raises(bg.BloomError) as e:
        f()
    assert e.value.status in (1, 2)


def test_python_checks(lib):
    bf, cpu = torch.bfloat16, "cpu"
    w4 = bg.W4.empty(48, 512, 64, cpu)
    assert w4.tiles.numel() == lib.bloom_w4_bytes(48, 512, 64) and (w4.n, w4.k, w4.group) == (48, 512, 64)
    w, x = torch.zeros(48, 512, dtype=bf), torch.zeros(3, 512, dtype=bf)
    # host tensors are refused
    refused(lambda: bg.op_w4_quantize(w))
    refused(lambda: bg.op_w4_read(w4))
    refused(lambda: bg.op_linear_w4(x, w4))
    refused(lambda: bg.op_sample_filtered(torch.zeros(2, 8), torch.zeros(2)))
    # sizes, types, shapes and strides
    for a in [(48, 12), (48, 0), (0, 8), (48, 512, 16), (48, 512, 0), (2 ** 32 + 16, 8), (16, 2 ** 32 + 8), (16, 8, 2 ** 32 + 64)]:
        refused(lambda: bg.W4.empty(*a, device=cpu))
    for tiles in [w4.tiles[:-1], w4.tiles.view(torch.int8), w4.tiles[None], torch.zeros(2 * w4.tiles.numel(), dtype=torch.uint8)[::2]]:
        refused(lambda: bg.W4(tiles, 48, 512, 64))
    refused(lambda: bg.op_w4_quantize(w[0]))
    refused(lambda: bg.op_linear_w4(x[0], w4))
    for z in [torch.zeros(8), torch.zeros(2, 8, dtype=bf), torch.zeros(8, 2).t(), torch.zeros(2, 8, dtype=torch.float64)]:
        refused(lambda: bg.op_sample_filtered(z, torch.zeros(2)))


@pytest.mark.gpu
def test_python_checks_on_the_device(lib):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    new = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device="cuda")
    w4 = bg.op_w4_quantize(new(48, 512))
    x, y = new(3, 512), new(3, 48)
    for w in [new(48, 512, dtype=f32), new(48, 508), new(512, 48).t(), new(48, 1, 512), new(48, 516)[:, :512], new(48 * 512 + 8)[4:-4].view(48, 512),
              new(1, 512).expand(48, 512)]:
        refused(lambda: bg.op_w4_quantize(w))
    for out in [bg.W4.empty(48, 504), bg.W4.empty(64, 512), bg.W4.empty(48, 512, device="cpu")]:
        refused(lambda: bg.op_w4_quantize(new(48, 512), out=out))
    for out in [new(48, 504), new(48, 512, dtype=f32), new(512, 48).t(), torch.zeros(48, 512, dtype=bf), new(1, 512).expand(48, 512)]:
        refused(lambda: bg.op_w4_read(w4, out))
    for a, kw in [((new(3, 504), w4), {}), ((x.float(), w4), {}), ((new(512, 3).t(), w4), {}), ((new(3, 516)[:, :512], w4), {}),
                  ((new(1, 512).expand(3, 512), w4), {}), ((x, bg.W4.empty(48, 512, device="cpu")), {}),
                  ((x, w4, new(47)), {}), ((x, w4, new(48, dtype=f32)), {}), ((x, w4, new(96)[::2]), {}),
                  ((x, w4), dict(epilogue=3)), ((x, w4), dict(epilogue=2)), ((x, w4), dict(dtype=torch.float16)),
                  ((x, w4), dict(y=y.half())), ((x, w4), dict(y=new(3, 49))), ((x, w4), dict(y=new(48, 3).t())),
                  ((x, w4), dict(y=new(1, 48).expand(3, 48))), ((x, w4), dict(y=y.cpu())),
                  ((x, w4), dict(flag=new(1, dtype=f32))), ((x, w4), dict(flag=new(2, dtype=i32))),
                  ((x, w4), dict(workspace=new(64, dtype=i32))), ((x, w4), dict(workspace=torch.zeros(64, dtype=torch.uint8))),
                  ((new(12, 512), w4), dict(workspace=new(64, dtype=torch.uint8)))]:
        refused(lambda: bg.op_linear_w4(*a, **kw))
    z, u = new(4, 100, dtype=f32), new(4, dtype=f32)
    for kw in [dict(u=u[:3]), dict(u=u.double()), dict(u=u.cpu()), dict(u=new(3, 4, dtype=f32)), dict(u=new(4, 2, 2, dtype=f32)),
               dict(u=new(2, 4, dtype=f32).t()), dict(temperature=u[:1]), dict(temperature=u.double()), dict(top_k=u), dict(top_p=u.bfloat16()),
               dict(min_p=u.cpu()), dict(top_k=new(4, dtype=torch.int64)), dict(out=u), dict(out=new(5, dtype=i32)),
               dict(out=new(4, 1, dtype=i32))]:
        refused(lambda: bg.op_sample_filtered(z, **dict(dict(u=u), **kw)))
    refused(lambda: bg.op_sample_filtered(new(1, 100, dtype=f32).expand(4, 100), u))
    assert torch.equal(bg.op_linear_w4(x, w4), y)               # and the device still answers


# ------------------------------------------------- the plain forms' own closed cases
def test_plain_quantize_closed_forms():
    w = torch.zeros(2, 40, dtype=torch.bfloat16)
    w[0, :4] = torch.tensor([14.0, -14.0, 3.0, 5.0])           # scale 2: codes 7, -7, 1.5 -> 2, 2.5 -> 2
    w[1, 32] = 2.0 ** -133                                     # its scale rounds to 0
    code, s = plain.quantize(w, 32)
    assert s.tolist() == [[2.0, 0.0], [0.0, 0.0]] and (code[1] == 0).all()
    assert code[0, :4].tolist() == [7.0, -7.0, 2.0, 2.0] and code.shape == (2, 64)
    assert plain.values(w, 32).shape == (2, 40) and plain.values(w, 32)[0, 2] == 4.0


def test_plain_bf16_rounding_is_the_types():
    v = torch.cat([torch.linspace(-3, 3, 20001), torch.logspace(-40, 38, 5001)]).float()
    assert torch.equal(plain.bf16_of(v.double()), v.to(torch.bfloat16).double())


def test_plain_sampling_closed_forms():
    z = np.log(np.array([0.5, 0.3, 0.2]))
    assert sample_plain.kept_of(z, 1.0, 2, 1.0, 0.0)[0].tolist() == [0, 1]
    assert sample_plain.kept_of(z, 1.0, 0, 0.6, 0.0)[0].tolist() == [0, 1]
    assert sample_plain.kept_of(z, 1.0, 0, 1.0, 0.5)[0].tolist() == [0, 1]
    assert sample_plain.kept_of(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0) is None
    kept = sample_plain.kept_of(z, 1.0, 0, 1.0, 0.0)
    assert [sample_plain.draw(kept, u) for u in (0.0, 0.4, 0.6, 0.9, 1.0, float("nan"))] == [0, 0, 1, 2, 2, 0]
