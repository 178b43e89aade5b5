"""The 8-bit KV cache on the GPU: write, read back, decode attention, alone and
together, against the plain float64 forms (kv8_plain).

Codes, scales and values read back must be equal to the last bit (every scale is
a power of two, so the only rounding is the code's).  Attention's bound is
derived in kv8_plain.attend."""
import ctypes as C

import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
from bloom_decoder_token_gb300 import synth
import kv8_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [torch.int8, torch.float8_e4m3fn]
codes_param = pytest.mark.parametrize("codes", CODES, ids=["int8", "e4m3"])


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def bf(shape, g, std=1.0):
    return (std * torch.randn(*shape, generator=g)).to(torch.bfloat16)


def garbage(B, n, S, d, codes, g):
    """A cache that holds anything at all, NaN codes and NaN scales too."""
    raw = [torch.randint(0, 256, (B, n, S, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    if codes is torch.float8_e4m3fn:
        raw[0][..., ::3] = 0x7F
        raw[1][..., 1::3] = 0xFF
    sc = [torch.full((B, n, -(-S // 32)), float("nan")) for _ in range(2)]
    return bg.KV8(*(r.view(codes).to(DEV) for r in raw), *(s.to(DEV) for s in sc))


def same_codes(a, b):
    """Equal codes: as values (a zero has either sign)."""
    return np.array_equal(plain.code_values(a), np.asarray(b), equal_nan=True)


def mirror(kv):
    return [plain.code_values(kv.k), plain.code_values(kv.v), plain.f64(kv.k_scale), plain.f64(kv.v_scale)]


def write_both(kv, m, k, v, start, count=None, mask=None, flag=None):
    dev = lambda t: None if t is None else t.to(DEV)
    bg.op_kv8_write(kv, k if k.is_cuda else dev(k), v if v.is_cuda else dev(v), dev(start), dev(count), dev(mask), flag)
    arr = lambda t: None if t is None else t.cpu().numpy()
    for i, x in ((0, k), (1, v)):
        plain.write(m[i], m[i + 2], kv.k.dtype, plain.f64(x), arr(start), arr(count), arr(mask))


def check(kv, m):
    assert np.array_equal(plain.f64(kv.k_scale), m[2], equal_nan=True)
    assert np.array_equal(plain.f64(kv.v_scale), m[3], equal_nan=True)
    assert same_codes(kv.k, m[0]) and same_codes(kv.v, m[1])


# --------------------------------------------------------------------- write
# (B, n, d, S, T, starts, counts, pads): one token, block borders, odd lengths, a cache
# that ends inside a block, idle rows, rows without tokens, whole prompts
WRITES = [
    (1, 1, 64, 1, 1, (0,), None, 0),
    (1, 16, 64, 40, 1, (39,), None, 0),
    (3, 2, 128, 70, 1, (31, 32, 63), None, 0),
    (3, 3, 128, 100, 33, (0, 31, 66), None, 5),
    (4, 2, 64, 129, 65, (-1, 0, 64, 17), (65, 0, 65, 40), 0),
    (2, 5, 128, 300, 257, (5, 32), (-3, 900), 7),
    (2, 4, 64, 96, 96, (0, 0), (96, 95), 96),
    (33, 2, 64, 64, 2, tuple(range(33)), None, 0),
]


@codes_param
@pytest.mark.parametrize("B,n,d,S,T,starts,counts,pads", WRITES)
def test_write(codes, B, n, d, S, T, starts, counts, pads):
    g = rng(B + n + d + S + T)
    kv = garbage(B, n, S, d, codes, g)
    # rows that start inside a block hold tokens before it: scales that a write makes
    for i, s in enumerate(starts):
        if s > 0:
            kv.k_scale[i] = 2.0 ** -9
            kv.v_scale[i] = 0.0
            kv.k.view(torch.uint8)[i] &= 0x3F
            kv.v.view(torch.uint8)[i] = 0
    m = mirror(kv)
    k, v = bf((B, T, n, d), g), bf((B, T, n, d), g, 30.0)
    k[..., ::7] = 0
    mask = (torch.arange(T)[None] >= torch.tensor([[pads]] * B)).to(torch.uint8) if pads else None
    write_both(kv, m, k, v, i32(*starts), None if counts is None else i32(*counts), mask)
    check(kv, m)


@codes_param
def test_write_token_by_token_grows_scales(codes):
    """70 single-token calls: every scale and every second rounding on the way."""
    g = rng(3)
    kv = garbage(2, 2, 72, 64, codes, g)
    m = mirror(kv)
    for t in range(70):
        size = 2.0 ** float(torch.randint(-6, 7, (1,), generator=g))
        write_both(kv, m, bf((2, 1, 2, 64), g, size), bf((2, 1, 2, 64), g, 1.0 + t), i32(t, t))
        if t % 9 == 0 or t > 60:
            check(kv, m)
    check(kv, m)


@codes_param
@pytest.mark.parametrize("layout", ["qkv", "heads", "wide"])
def test_write_strides(codes, layout):
    g = rng(5)
    B, T, n, d, S = 2, 45, 3, 64, 80
    if layout == "qkv":
        x = bf((B, T, n, 3, d), g).to(DEV)
        k, v = x[:, :, :, 1], x[:, :, :, 2]
    elif layout == "heads":
        k, v = bf((B, n, T, d), g).to(DEV).transpose(1, 2), bf((B, T, n, d), g).to(DEV)
    else:
        x = bf((T, B, n, 2 * d + 8), g).to(DEV)
        k, v = (x[..., o:o + d].transpose(0, 1) for o in (0, d + 8))
    kv = garbage(B, n, S, d, codes, g)
    m = mirror(kv)
    write_both(kv, m, k, v, i32(0, 32))
    check(kv, m)
    # and read back, K into a view inside a larger buffer
    dst = torch.full((B, n, T + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = dst[:, :, 1:T + 1].transpose(1, 2)
    _, vo = bg.op_kv8_read(kv, i32(0, 32).to(DEV), T, k=ko)
    assert np.array_equal(plain.f64(ko), plain.read(m[0], m[2], [0, 32], T))
    assert np.array_equal(plain.f64(vo), plain.read(m[1], m[3], [0, 32], T))
    assert (dst[:, :, 0] == 7).all() and (dst[:, :, T + 1:] == 7).all()   # nothing beside the view


@codes_param
def test_write_magnitudes(codes):
    """From bf16's smallest subnormal to its largest number, one magnitude a head; and
    values at the edge between two scales, and ties of the rounding."""
    tiny = 2.0 ** -133
    mags = [tiny, 2.0 ** -127, 2.0 ** -126, 2.0 ** -120, 1e-30, 1.0, 126.5, 127.0, 128.0, 254.0, 255.0, 448.0, 450.0,
            1e30, 2.0 ** 127, 3.2e38]
    n, T, d = len(mags), 32, 64
    g = rng(8)
    x = (torch.rand(1, T, n, d, generator=g) * 2 - 1).double() * torch.tensor(mags, dtype=torch.float64)[None, None, :, None]
    x[0, 0, :, 0] = torch.tensor(mags, dtype=torch.float64)
    x[0, 1, :, :32] = (torch.arange(32).double() + 0.5)[None] * torch.tensor(mags, dtype=torch.float64)[:, None] / 64
    x = x.to(torch.bfloat16)
    x[0, 0, -1, 0] = torch.finfo(torch.bfloat16).max
    kv = garbage(1, n, T, d, codes, g)
    m = mirror(kv)
    write_both(kv, m, x, -x, i32(0))
    check(kv, m)


@codes_param
def test_write_infinities_and_nans(codes):
    """An infinity or NaN makes its block's scale NaN (K and V, heads and blocks apart);
    under a mask it is not looked at; a block started afresh is clean again."""
    g = rng(9)
    k, v = bf((1, 64, 2, 64), g), bf((1, 64, 2, 64), g)
    k[0, 3, 0, 5] = float("inf")
    v[0, 40, 1, 63] = float("nan")
    kv = garbage(1, 2, 70, 64, codes, g)
    m = mirror(kv)
    write_both(kv, m, k, v, i32(0))
    check(kv, m)
    assert torch.isnan(kv.k_scale.cpu()[0, :, :2]).tolist() == [[True, False], [False, False]]
    assert torch.isnan(kv.v_scale.cpu()[0, :, :2]).tolist() == [[False, False], [False, True]]
    write_both(kv, m, bf((1, 1, 2, 64), g), bf((1, 1, 2, 64), g), i32(20))   # the NaN stays
    check(kv, m)
    assert torch.isnan(kv.k_scale[0, 0, 0])
    mask = torch.ones(1, 64, dtype=torch.uint8)
    mask[0, 3] = mask[0, 40] = 0
    write_both(kv, m, k, v, i32(0), None, mask)
    check(kv, m)
    assert not torch.isnan(kv.k_scale[0, :, :2]).any() and not torch.isnan(kv.v_scale[0, :, :2]).any()


@codes_param
def test_write_beyond_the_cache_and_flag(codes):
    g = rng(10)
    kv = garbage(3, 2, 45, 64, codes, g)
    m = mirror(kv)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    write_both(kv, m, bf((3, 20, 2, 64), g), bf((3, 20, 2, 64), g), i32(0, 32, 2 ** 31 - 1), i32(20, 13, 0), flag=flag)
    check(kv, m)
    assert flag.item() == 2      # a row that starts beyond the cache
    flag.zero_()
    write_both(kv, m, bf((3, 20, 2, 64), g), bf((3, 20, 2, 64), g), i32(0, -1, -7), flag=flag)
    check(kv, m)
    assert flag.item() == 0
    write_both(kv, m, bf((3, 20, 2, 64), g), bf((3, 20, 2, 64), g), i32(32, -1, 64), flag=flag)
    check(kv, m)
    assert flag.item() == 2
    k, v = bg.op_kv8_read(kv, i32(32, 0, 45).to(DEV), 20, flag=flag.zero_())
    assert flag.item() == 2
    assert np.array_equal(plain.f64(k), plain.read(m[0], m[2], [32, 0, 45], 20), equal_nan=True)


# ---------------------------------------------------------------------- read
@codes_param
@pytest.mark.parametrize("B,n,d,S,T,starts,counts", [
    (1, 1, 64, 1, 1, (0,), None), (2, 3, 128, 77, 40, (37, 0), None), (4, 2, 64, 130, 130, (0, -1, 0, 0), (130, 5, 0, 31)),
    (2, 25, 64, 700, 613, (3, 87), (613, 500)), (1, 16, 128, 33, 0, (0,), None)])
def test_read(codes, B, n, d, S, T, starts, counts):
    g = rng(B * n + d + S + T)
    kv = bg.KV8.empty(B, n, S, d, codes, DEV)
    m = mirror(kv)
    write_both(kv, m, bf((B, S, n, d), g), bf((B, S, n, d), g, 0.01), i32(*[0] * B))
    cnt = None if counts is None else i32(*counts)
    k, v = bg.op_kv8_read(kv, i32(*starts).to(DEV), T, None if cnt is None else cnt.to(DEV))
    assert k.shape == v.shape == (B, T, n, d)
    assert np.array_equal(plain.f64(k), plain.read(m[0], m[2], starts, T, counts))
    assert np.array_equal(plain.f64(v), plain.read(m[1], m[3], starts, T, counts))


@codes_param
def test_read_every_code(codes):
    """All 256 codes (but e4m3's NaNs) at several scales, powers of two or not."""
    kv = bg.KV8.empty(1, 4, 32, 64, codes, DEV)
    c = (torch.arange(32 * 64) % 256).to(torch.uint8).view(1, 1, 32, 64).expand(1, 4, 32, 64).clone()
    if codes is torch.float8_e4m3fn:
        c[(c & 0x7F) == 0x7F] = 0
    kv.k.view(torch.uint8).copy_(c)
    kv.k_scale.copy_(torch.tensor([1.0, 2.0 ** -126, 2.0 ** 100, 0.3]).view(1, 4, 1))
    k, _ = bg.op_kv8_read(kv, i32(0).to(DEV), 32)
    ref = torch.from_numpy(plain.wide(plain.code_values(kv.k), plain.f64(kv.k_scale)))
    assert torch.equal(k.cpu().transpose(1, 2).float(), ref.float().to(torch.bfloat16).float())


# ----------------------------------------------------------------- attention
def filled(B, n, S, d, codes, lens, g, pads=0, holes=(), std=1.0):
    """A written cache, its slots beyond each row's length and its masked ones full of
    garbage; positions; the plain values."""
    kv = garbage(B, n, S, d, codes, g)
    m = mirror(kv)
    write_both(kv, m, bf((B, S, n, d), g, std), bf((B, S, n, d), g), i32(*[0] * B), i32(*[max(0, x) for x in lens]))
    pos = torch.full((B, S), -1, dtype=torch.int32)
    for b in range(B):
        c = 0
        for t in range(max(0, min(S, lens[b]))):
            if t < pads or t in holes:
                for raw, x in ((kv.k, m[0]), (kv.v, m[1])):
                    raw.view(torch.uint8)[b, :, t] = 0x7F
                    x[b, :, t] = 0.0
                continue
            pos[b, t] = c
            c += 1
    m = [np.nan_to_num(x) for x in m]
    return kv, pos, plain.wide(m[0], m[2]), plain.wide(m[1], m[3])


def slopes_of(n):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / n) for i in range(n)], dtype=torch.float32)


def check_attention(kv, pos, kf, vf, q, slopes, lens, **kw):
    dv = lambda t: None if t is None else t.to(DEV)
    o = bg.op_attn_decode_kv8(dv(q), kv, dv(pos), dv(slopes), i32(*lens).to(DEV), **kw)
    B, T, n, d = q.shape
    assert o.shape == (B, T, n * d)
    sl = np.zeros(n) if slopes is None else plain.f64(slopes)
    ref, tol = plain.attend(plain.f64(q), kf, vf, pos.numpy(), sl, lens)
    got = plain.f64(o).reshape(ref.shape)
    assert bool(np.isfinite(got).all())
    bad = np.abs(got - ref) > tol + 2.0 ** -134      # half the smallest bf16 number
    assert not bool(bad.any()), (int(bad.sum()), float(np.abs(got - ref)[bad].max()), np.argwhere(bad)[:4].tolist())
    return o


# (B, T, n, kv, d, S, lens, pads, holes)
ATTN = [
    (1, 1, 16, 16, 64, 1, (1,), 0, ()),                       # one key
    (1, 1, 1, 1, 64, 1, (1,), 0, ()),                         # a cache of one slot in all
    (1, 2, 3, 1, 128, 2, (2,), 0, ()),
    (1, 1, 4, 4, 128, 33, (33,), 0, ()),                      # the cache ends one slot into a block
    (3, 1, 16, 16, 64, 140, (37, 0, 140), 5, (9,)),           # an idle row; pads and a hole
    (2, 1, 12, 12, 64, 100, (31, 32), 0, ()),
    (2, 1, 32, 32, 128, 700, (699, 130), 64, (200, 201)),     # whole blocks masked
    (2, 1, 7, 7, 64, 257, (5, 257), 5, ()),                   # a row of pads only
    (2, 3, 8, 8, 128, 96, (2, 96), 0, ()),                    # fewer slots than new tokens
    (2, 4, 32, 8, 128, 300, (299, 65), 3, (64,)),             # 16 columns a key head
    (1, 5, 10, 2, 64, 513, (511,), 0, ()),                    # 25
    (3, 1, 71, 1, 128, 200, (200, 1, 77), 0, ()),             # one key head, odd group
    (2, 32, 16, 16, 64, 200, (190, 33), 0, ()),               # the most tokens
    (1, 32, 24, 3, 128, 90, (88,), 2, ()),                    # 256 columns
    (33, 1, 4, 4, 64, 140, tuple(range(33)), 0, ()),
    (40, 1, 25, 5, 64, 95, tuple((7 * i) % 96 for i in range(40)), 1, ()),
    (1, 1, 2, 2, 64, 9000, (8987,), 11, (8000,)),             # few heads, long: the most splitting
    (1, 1, 1, 1, 128, 40000, (39990,), 3, ()),                # one head: partials by the hundred
    (1, 4, 5, 1, 64, 30000, (29999,), 0, (29998,)),
    (300, 1, 1, 1, 64, 64, tuple((i * 13) % 65 for i in range(300)), 0, ()),
]


@codes_param
@pytest.mark.parametrize("B,T,n,kv,d,S,lens,pads,holes", ATTN)
def test_attention(codes, B, T, n, kv, d, S, lens, pads, holes):
    g = rng(B + T + n + kv + d + S)
    cache, pos, kf, vf = filled(B, kv, S, d, codes, lens, g, pads, holes)
    check_attention(cache, pos, kf, vf, bf((B, T, n, d), g, 1.5), slopes_of(n), lens)


@codes_param
def test_attention_without_slopes_and_3d_query(codes):
    g = rng(21)
    cache, pos, kf, vf = filled(2, 4, 90, 64, codes, (90, 41), g, std=0.1)   # near-uniform weights
    q = bf((2, 1, 8, 64), g)
    o = check_attention(cache, pos, kf, vf, q, None, (90, 41))
    o3 = bg.op_attn_decode_kv8(q[:, 0].contiguous().to(DEV), cache, pos.to(DEV), None, i32(90, 41).to(DEV))
    assert o3.shape == (2, 8 * 64) and torch.equal(o3, o[:, 0])


def test_attention_one_key_is_its_value():
    g = rng(22)
    cache, pos, kf, vf = filled(2, 4, 8, 128, torch.float8_e4m3fn, (1, 1), g)
    o = bg.op_attn_decode_kv8(bf((2, 4, 128), g).to(DEV), cache, pos.to(DEV), slopes_of(4).to(DEV), i32(1, 1).to(DEV))
    assert np.array_equal(plain.f64(o).reshape(2, 4, 128), vf[:, :, 0])


@codes_param
@pytest.mark.parametrize("qs,ks,vs", [(1e4, 1.0, 1.0), (1e-4, 1e-4, 1e-30), (1e30, 1e-30, 1e30), (1e-37, 1e37, 1.0),
                                      (0.0, 1.0, 1.0), (1.0, 1.0, 1e-37), (1.0, 1.0, 1e37), (1e-39, 1e-39, 1e-39)])
def test_attention_magnitudes(codes, qs, ks, vs):
    """Queries, keys and values far from 1; scores stay moderate or one key takes all."""
    g = rng(23)
    B, n, S, d = 2, 3, 120, 64
    kv = bg.KV8.empty(B, n, S, d, codes, DEV)
    m = mirror(kv)
    write_both(kv, m, bf((B, S, n, d), g, ks), bf((B, S, n, d), g, vs), i32(0, 0))
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    check_attention(kv, pos, plain.wide(m[0], m[2]), plain.wide(m[1], m[3]), bf((B, 1, n, d), g, qs), slopes_of(n), (120, 77))


@codes_param
def test_attention_value_scales_far_apart(codes):
    """Blocks whose V scales differ by 2^60: a block of large values that the scores
    all but rule out, and one of tiny values that they single out."""
    g = rng(24)
    B, n, S, d = 1, 2, 160, 64
    kv = bg.KV8.empty(B, n, S, d, codes, DEV)
    m = mirror(kv)
    k, v = bf((B, S, n, d), g, 0.1), bf((B, S, n, d), g)
    v[:, 32:64] *= 2.0 ** 30
    v[:, 96:128] *= 2.0 ** -30
    v[:, 128:150] = 0
    write_both(kv, m, k, v, i32(0))
    q = bf((B, 1, n, d), g, 0.1)
    for lens, slope in [((160,), 4.0), ((128,), 8.0), ((100,), 1.0), ((64,), 2.0), ((150,), 16.0)]:
        pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
        check_attention(kv, pos, plain.wide(m[0], m[2]), plain.wide(m[1], m[3]), q, torch.full((n,), slope), lens)


def test_attention_far_positions():
    """Positions past 2^20, as of a row that was cut: the near keys' weights stay exact."""
    g = rng(25)
    cache, pos, kf, vf = filled(1, 4, 300, 64, torch.int8, (300,), g)
    pos = pos + 3_000_000
    check_attention(cache, pos, kf, vf, bf((1, 1, 4, 64), g), slopes_of(4), (300,))


@codes_param
def test_attention_nan_scale_reaches_only_queries_that_see_it(codes):
    g = rng(26)
    cache, pos, kf, vf = filled(2, 2, 128, 64, codes, (128, 128), g)
    cache.k_scale[0, 0, 3] = float("nan")
    cache.v_scale[1, 1, 3] = float("nan")
    q = bf((2, 1, 2, 64), g).to(DEV)
    o = bg.op_attn_decode_kv8(q, cache, pos.to(DEV), slopes_of(2).to(DEV), i32(128, 128).to(DEV)).view(2, 2, 64)
    assert torch.isnan(o).all(-1).tolist() == [[True, False], [False, True]]
    assert torch.isnan(o).any(-1).tolist() == [[True, False], [False, True]]
    o = bg.op_attn_decode_kv8(q, cache, pos.to(DEV), slopes_of(2).to(DEV), i32(96, 96).to(DEV))
    assert torch.isfinite(o).all()
    q[0, 0, 1, 3] = float("nan")
    o = bg.op_attn_decode_kv8(q, cache, pos.to(DEV), slopes_of(2).to(DEV), i32(96, 96).to(DEV)).view(2, 2, 64)
    assert torch.isnan(o[0, 1]).all() and torch.isfinite(o[0, 0]).all() and torch.isfinite(o[1]).all()


def test_attention_length_beyond_the_cache_sets_the_flag():
    g = rng(27)
    cache, pos, kf, vf = filled(2, 2, 50, 64, torch.int8, (50, 50), g)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_attention(cache, pos, kf, vf, bf((2, 2, 2, 64), g), slopes_of(2), (51, 50), flag=flag)
    assert flag.item() == 2
    o = bg.op_attn_decode_kv8(bf((2, 1, 2, 64), g).to(DEV), cache, pos.to(DEV), None, i32(-5, -2 ** 31).to(DEV), flag=flag.zero_())
    assert flag.item() == 0 and (o == 0).all()


def test_attention_repeats_to_the_bit():
    g = rng(28)
    cache, pos, kf, vf = filled(5, 6, 3000, 128, torch.int8, (3000, 1, 1999, 640, 2500), g)
    q = bf((5, 1, 6, 128), g).to(DEV)
    a = [bg.op_attn_decode_kv8(q, cache, pos.to(DEV), slopes_of(6).to(DEV), i32(3000, 1, 1999, 640, 2500).to(DEV)) for _ in range(4)]
    assert all(torch.equal(a[0], x) for x in a[1:])


def test_attention_long_cache():
    """Code offsets past 2^32 bytes: 4.4 G of K; the last row's last slots."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    B, n, S, d = 3, 112, 102_400, 128
    g = torch.Generator(device=DEV).manual_seed(29)
    kv = bg.KV8.empty(B, n, S, d, torch.int8, DEV)
    assert kv.k.numel() > 2 ** 32
    T = 200
    k, v = (torch.randn(B, T, n, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    at = S - T
    bg.op_kv8_write(kv, k, v, i32(0, -1, at).to(DEV))
    rk, rv = bg.op_kv8_read(kv, i32(0, at, at).to(DEV), T)
    assert (rk[1] == 0).all() and (rk[2].float() - k[2].float()).abs().max() < 0.05 and (rv[0].float() - v[0].float()).abs().max() < 0.05
    pos = torch.full((B, S), -1, dtype=torch.int32)
    pos[0, :T] = torch.arange(T, dtype=torch.int32)
    pos[2, at:] = torch.arange(T, dtype=torch.int32)
    q = torch.randn(B, 1, n, d, generator=g, device=DEV).to(torch.bfloat16)
    lens = (T, S, S)
    o = bg.op_attn_decode_kv8(q, kv, pos.to(DEV), slopes_of(n).to(DEV), i32(*lens).to(DEV))
    vals = [plain.f64(x).transpose(0, 2, 1, 3) for x in (rk, rv)]
    small = torch.arange(T, dtype=torch.int32).repeat(B, 1)
    ref, tol = plain.attend(plain.f64(q), vals[0], vals[1], small.numpy(), plain.f64(slopes_of(n)), (T, T, T))
    got = plain.f64(o).reshape(ref.shape)
    for b in (0, 2):
        assert bool((np.abs(got[b] - ref[b]) <= tol[b] + 2.0 ** -134).all())
    assert (got[1] == 0).all()      # every position masked


# more work than the GPU's warps hold at once: many short rows among long ones, rows whose
# every visible slot lies at the end, lengths at the borders of blocks
BUSY = [
    (24, 1, 40, 40, 128, 1600, lambda b: (1600, 129, 128, 160, 1, 0, 1599, 33)[b % 8], 0),
    (6, 1, 112, 112, 64, 4100, lambda b: (4100, 4033, 193, 0, 2048, 3000)[b], 3900),
    (9, 3, 64, 64, 128, 1400, lambda b: 1400 - 37 * b, 3),
    (16, 2, 96, 32, 64, 3000, lambda b: 3000 - 150 * b, 0),
    (8, 4, 64, 16, 128, 6000, lambda b: 6000 - 700 * b, 0),
]


@codes_param
@pytest.mark.parametrize("B,T,n,kv,d,S,length,pads", BUSY)
def test_attention_busy(codes, B, T, n, kv, d, S, length, pads):
    g = torch.Generator(device=DEV).manual_seed(B + n + S)
    lens = [length(b) for b in range(B)]
    cache = bg.KV8.empty(B, kv, S, d, codes, DEV)
    x = torch.randn(2, B, S, kv, d, generator=g, device=DEV).to(torch.bfloat16)
    bg.op_kv8_write(cache, x[0], x[1], torch.zeros(B, dtype=torch.int32, device=DEV))
    pos = torch.arange(S, dtype=torch.int32)[None].repeat(B, 1) - pads
    pos = torch.where(pos < 0, torch.tensor(-1, dtype=torch.int32), pos)
    q = torch.randn(B, T, n, d, generator=g, device=DEV).to(torch.bfloat16)
    sl = slopes_of(n)
    o = bg.op_attn_decode_kv8(q, cache, pos.to(DEV), sl.to(DEV), i32(*lens).to(DEV))
    again = bg.op_attn_decode_kv8(q, cache, pos.to(DEV), sl.to(DEV), i32(*lens).to(DEV))
    assert torch.equal(o, again)
    # float64 on the device, all rows and heads
    kf, vf = (c.double() * s.double().repeat_interleave(32, 2)[:, :, :S, None] for c, s in ((cache.k.float(), cache.k_scale), (cache.v.float(), cache.v_scale)))
    qd, posd, grp = q.double(), pos.to(DEV).double(), n // kv
    for b in range(B):
        ln = lens[b]
        for t in range(T):
            upto = max(0, ln - T + t + 1) if ln > 0 else 0
            see = posd[b, :upto] >= 0
            got = o[b, t].double().view(n, d)
            if not bool(see.any()):
                assert (got == 0).all()
                continue
            k, v = kf[b, :, :upto][:, see].repeat_interleave(grp, 0), vf[b, :, :upto][:, see].repeat_interleave(grp, 0)
            far = sl.to(DEV).double()[:, None] * (posd[b, :upto][see] - posd[b, :upto][see].max())
            s = (k @ qd[b, t][:, :, None])[..., 0] / d ** 0.5 + far
            p = torch.softmax(s, 1)
            ref = (p[:, None] @ v)[:, 0]
            # the bound of kv8_plain.attend
            size = (k.abs() @ qd[b, t].abs()[:, :, None])[..., 0] / d ** 0.5 + far.abs()
            es = (d + 16) * 2.0 ** -23 * torch.where(p > 1e-9, size, torch.zeros_like(size)).amax(1)
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * es)[:, None] * (p[:, None] @ v.abs())[:, 0]
            assert bool(((got - ref).abs() <= tol + 2.0 ** -134).all()), (b, t, float((got - ref).abs().max()))


def test_attention_explicit_workspace():
    g = rng(32)
    lens = (1500, 700)
    cache, pos, kf, vf = filled(2, 4, 1600, 64, torch.int8, lens, g)
    q = bf((2, 2, 8, 64), g)
    c = cache.c()
    need = bg.lib().bloom_op_attn_decode_kv8_workspace(C.byref(c), 2, 8)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)      # NaNs: contents do not matter
    o = check_attention(cache, pos, kf, vf, q, slopes_of(8), lens, workspace=ws)
    out = torch.full_like(o, 3.0)
    o2 = bg.op_attn_decode_kv8(q.to(DEV), cache, pos.to(DEV), slopes_of(8).to(DEV), i32(*lens).to(DEV), o=out, workspace=ws[:need])
    assert o2 is out and torch.equal(o, out)
    assert (ws[need:] == 0xFF).all()
    for bad in (ws[:need - 1], ws[1:need + 1], ws[:0], ws.cpu(), ws.view(torch.int8)):
        with pytest.raises(bg.BloomError):
            bg.op_attn_decode_kv8(q.to(DEV), cache, pos.to(DEV), slopes_of(8).to(DEV), i32(*lens).to(DEV), workspace=bad)


def test_attention_many_rows():
    """More rows than a warp scans at once, most of them idle or short, some cut."""
    g = rng(33)
    B, S = 2500, 600
    lens = [0] * B
    for i in range(0, B, 7):
        lens[i] = (i * 37) % 601
    cache, pos, kf, vf = filled(B, 1, S, 64, torch.float8_e4m3fn, lens, g)
    check_attention(cache, pos, kf, vf, bf((B, 1, 2, 64), g), slopes_of(2), lens)


def test_first_call_of_a_form_inside_a_capture():
    """Nothing that a form sets up on its first call is forbidden in a capture."""
    g = rng(34)
    lens = (400, 90)
    for T, n, kv, codes in [(3, 3, 3, torch.int8), (7, 5, 5, torch.float8_e4m3fn), (11, 4, 2, torch.int8)]:
        cache, pos, kf, vf = filled(2, kv, 420, 128, codes, lens, g)
        q, posd, sl, ln = bf((2, T, n, 128), g), pos.to(DEV), slopes_of(n).to(DEV), i32(*lens).to(DEV)
        qd = q.to(DEV)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = bg.op_attn_decode_kv8(qd, cache, posd, sl, ln)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, check_attention(cache, pos, kf, vf, q, slopes_of(n), lens))


def test_write_of_one_head_to_all():
    """Source strides of 0: one key head's values written to every head of the cache."""
    g = rng(35)
    k, v = bf((2, 40, 1, 64), g).to(DEV).expand(2, 40, 5, 64), bf((1, 40, 5, 64), g).to(DEV).expand(2, 40, 5, 64)
    kv = garbage(2, 5, 64, 64, torch.int8, g)
    m = mirror(kv)
    write_both(kv, m, k, v, i32(0, 0))
    check(kv, m)


# ------------------------------------------------------ streams, graphs, a run
def test_another_stream():
    g = rng(30)
    cache, pos, kf, vf = filled(2, 4, 500, 64, torch.int8, (500, 77), g)
    q, posd, sl, ln = bf((2, 1, 4, 64), g).to(DEV), pos.to(DEV), slopes_of(4).to(DEV), i32(500, 77).to(DEV)
    here = bg.op_attn_decode_kv8(q, cache, posd, sl, ln)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    there = bg.op_attn_decode_kv8(q, cache, posd, sl, ln, stream=s)
    with torch.cuda.stream(s):
        also = bg.op_attn_decode_kv8(q, cache, posd, sl, ln)
        k, _ = bg.op_kv8_read(cache, i32(0, 0).to(DEV), 50)
    s.synchronize()
    assert torch.equal(here, there) and torch.equal(here, also)
    assert np.array_equal(plain.f64(k), kf[:, :, :50].transpose(0, 2, 1, 3))


@codes_param
def test_captured_steps_follow_the_device_lengths(codes):
    """A serving step (append, attend, log probabilities) captured once and replayed:
    start and lens are advanced on the device; a second graph over other buffers
    runs in between.  Every replay equals the eager call to the bit."""
    g = rng(31)
    B, n, d, S, V = 3, 4, 64, 200, 777
    sl = slopes_of(n).to(DEV)

    def state(lens):
        kv = bg.KV8.empty(B, n, S, d, codes, DEV)
        m = mirror(kv)
        write_both(kv, m, bf((B, S, n, d), g), bf((B, S, n, d), g), i32(*[0] * B), i32(*lens))
        return dict(kv=kv, pos=torch.arange(S, dtype=torch.int32, device=DEV).repeat(B, 1), start=i32(*lens).to(DEV),
                    lens=i32(*lens).to(DEV) + 1, x=bf((B, 1, n, 3, d), g).to(DEV), z=torch.randn(B, V, generator=g).to(DEV),
                    tok=i32(1, -1, 700).to(DEV))

    def step(s):
        bg.op_kv8_write(s["kv"], s["x"][:, :, :, 1], s["x"][:, :, :, 2], s["start"])
        o = bg.op_attn_decode_kv8(s["x"][:, :, :, 0].contiguous(), s["kv"], s["pos"], sl, s["lens"])
        return (o, *bg.op_logprobs(s["z"], s["tok"], 3))

    states = [state((30, 100, 0)), state((90, 31, 150))]
    graphs = []
    for s in states:
        step(s)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(s)
        graphs.append((gr, out))
    for it in range(4):
        for s in states:
            s["x"].copy_(bf((B, 1, n, 3, d), g).to(DEV) * 2.0 ** it)
            s["z"].copy_(torch.randn(B, V, generator=g).to(DEV))
            s["start"] += 1
            s["lens"] += 1
        want = []
        for s in states:
            kv = s["kv"]
            s["kv"] = bg.KV8(*(t.clone() for t in kv))
            want.append((step(s), s["kv"]))
            s["kv"] = kv
        torch.cuda.synchronize()
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for (gr, out), (ref, kv), s in zip(graphs, want, states):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
            assert torch.equal(s["kv"].k.view(torch.uint8), kv.k.view(torch.uint8)) and torch.equal(s["kv"].v_scale, kv.v_scale)


@codes_param
def test_a_run_beside_the_model(codes):
    """Generation with the framework's model; one layer's bf16 cache is quantised after
    the prompt and then appended to step by step.  Attention over it stays near the
    framework's bf16 decode attention (the codes' own error: half a step of the
    block's largest value, int8 2^-7, e4m3 2^-4 of the value), and equals the plain
    form on the values it stands for; the step's logits give the greedy token as the
    most probable one."""
    shape = synth.PRESETS["560m"].with_(n_layer=2, vocab=3000, batch=3, prompt=37, ragged=True)
    w = synth.make_weights(shape, seed=4, random_affine=True).to(DEV)
    ids, mask = synth.make_prompts(shape, seed=4)
    B, T = ids.shape
    S, n, d = T + 8, shape.n_head, shape.head_dim
    gm = bg.Model(w, max_batch=B, max_tokens=B * T, max_seq=S)
    kv = gm.new_kv(B, S)
    lg = torch.empty(B, shape.vocab, device=DEV)
    tok = gm.prefill(kv, ids.to(DEV), mask.to(DEV), logits=lg)
    t = kv.tensors(gm)
    cache = bg.KV8.empty(B, n, S, d, codes, DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    bg.op_kv8_write(cache, t["k"][1].transpose(1, 2)[:, :T], t["v"][1].transpose(1, 2)[:, :T], zero, mask=mask.to(DEV))
    g = rng(6)
    sl = slopes_of(n)
    for step in range(6):
        logp, ent, top, tlp = bg.op_logprobs(lg, tok, 4)
        assert torch.equal(top[:, 0], tok) and torch.equal(tlp[:, 0], logp)
        assert (tlp[:, :-1] >= tlp[:, 1:]).all() and (ent >= 0).all()
        tok = gm.decode_step(kv, tok, logits=lg)
        at = T + step
        bg.op_kv8_write(cache, t["k"][1][:, :, at:at + 1].transpose(1, 2), t["v"][1][:, :, at:at + 1].transpose(1, 2), zero + at)
        q = bf((B, 1, n, d), g)
        lens = [at + 1] * B
        pos = t["pos"]
        kq, vq = bg.op_kv8_read(cache, zero, S)
        vals = [plain.f64(x).transpose(0, 2, 1, 3) for x in (kq, vq)]
        o = check_attention(cache, pos.cpu(), vals[0], vals[1], q, sl, lens)
        ref = bg.op_attn_decode(q[:, 0].to(DEV), t["k"][1].contiguous(), t["v"][1].contiguous(), pos.contiguous(), sl.to(DEV), at)
        near = (o[:, 0].float() - ref.float()).norm() / ref.float().norm()
        assert near < (2.0 ** -5 if codes is torch.int8 else 2.0 ** -4), float(near)
    gm.check_device()
    gm.close()
