"""Decode attention over the 8-bit cache with waits that run out: the bound is set to a
microsecond, less than the copies of a long cache take while all warps load.  The call
ends, flag 8 says so, the outputs that depend on a lost wait are NaN (whole heads of a
row), the others are the ordinary call's to the bit, and the device goes on as before."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# (B, T, n, kv, d, S, lens): whole heads and cut ones, one column and several, two chunks
CASES = [
    (3, 1, 32, 32, 128, 9000, (9000, 150, 4001)),
    (40, 1, 16, 16, 64, 1600, tuple((331 * i) % 1601 for i in range(40))),
    (6, 2, 16, 16, 64, 3000, (3000, 0, 190, 2999, 64, 1500)),
    (16, 4, 32, 8, 128, 2000, tuple(2000 - 90 * i for i in range(16))),
    (4, 5, 16, 4, 128, 3000, (3000, 2000, 1, 700)),
    (64, 1, 16, 16, 128, 130, tuple(1 + 2 * i for i in range(64))),
]


@pytest.mark.parametrize("B,T,n,kv,d,S,lens", CASES)
@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
def test_expired_waits(codes, B, T, n, kv, d, S, lens):
    g = torch.Generator(device=DEV).manual_seed(B + T + S)
    cache = bg.KV8.empty(B, kv, S, d, codes, DEV)
    x = torch.randn(2, B, S, kv, d, generator=g, device=DEV).to(torch.bfloat16)
    bg.op_kv8_write(cache, x[0], x[1], torch.zeros(B, dtype=torch.int32, device=DEV))
    pos = torch.arange(S, dtype=torch.int32, device=DEV).repeat(B, 1)
    q = torch.randn(B, T, n, d, generator=g, device=DEV).to(torch.bfloat16)
    slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / n) for i in range(n)], device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)

    def call():
        return bg.op_attn_decode_kv8(q, cache, pos, slopes, ln, flag=flag).view(B, T, n, d)

    want = call()
    assert flag.item() == 0 and torch.isfinite(want).all()
    lost = 0
    try:
        assert bg.lib().bloom_op_attn_decode_kv8_wait_us(1) == 0
        for _ in range(20):
            flush.zero_()                 # the codes come from memory
            flag.zero_()
            got = call()
            torch.cuda.synchronize()
            nan = torch.isnan(got)
            assert (nan.all(-1) == nan.any(-1)).all()
            assert flag.item() == (8 if nan.any() else 0)
            assert torch.equal(torch.where(nan, want, got), want)
            lost += int(nan.any())
    finally:
        assert bg.lib().bloom_op_attn_decode_kv8_wait_us(0) == 0
    assert lost > 0
    flag.zero_()
    assert torch.equal(call(), want) and flag.item() == 0
