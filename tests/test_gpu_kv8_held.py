"""Writes into blocks that hold something already: codes under a scale of 0 stand for 0
and stay 0 when the scale grows; what the header says of slots behind the write."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [torch.int8, torch.float8_e4m3fn]
codes_param = pytest.mark.parametrize("codes", CODES, ids=["int8", "e4m3"])


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@codes_param
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [1, 7, 31])
def test_codes_under_a_scale_of_zero_stay_zero(codes, d, at):
    """A cache of the caller's own: any codes (e4m3 NaNs too), scale 0.  Every value is 0 (a
    NaN code's is not looked at here) before a token is written behind them and after."""
    g = torch.Generator().manual_seed(at + d)
    kv = bg.KV8.empty(2, 3, 64, d, codes, DEV)
    kv.k.view(torch.uint8).copy_(torch.randint(0, 256, kv.k.shape, generator=g, dtype=torch.uint8))
    kv.v.view(torch.uint8).fill_(0x31)
    x = torch.randn(2, 1, 3, d, generator=g).to(torch.bfloat16).to(DEV)
    x[1] = 0                                              # a row whose scale stays 0
    before = kv.k.clone().view(torch.uint8)
    bg.op_kv8_write(kv, x, x, i32(at, at))
    k, v = bg.op_kv8_read(kv, i32(0, 0), at + 1)
    assert (k[0, :at] == 0).all() and (v[0, :at] == 0).all()
    assert (v[1] == 0).all() and (kv.k_scale[1] == 0).all()
    # the token itself: half a step of its head's largest value at most
    step = (2.0 ** -6 if codes is torch.int8 else 2.0 ** -4) * x[0, 0].float().abs().amax(-1, keepdim=True)
    assert ((k[0, at].float() - x[0, 0].float()).abs() <= step).all()
    # row 1's held codes and everything behind the written slot are as they were
    assert torch.equal(kv.k.view(torch.uint8)[1, :, :at], before[1, :, :at])
    assert torch.equal(kv.k.view(torch.uint8)[:, :, at + 1:], before[:, :, at + 1:])


@codes_param
def test_slots_behind_the_write_keep_their_codes_only(codes):
    """A filled block overwritten in its middle with larger values: the slots before keep their
    values (rounded again), those behind their codes, which the block's new scale now covers."""
    kv = bg.KV8.empty(1, 1, 32, 64, codes, DEV)
    x = torch.full((1, 32, 1, 64), 1.0, dtype=torch.bfloat16, device=DEV)
    bg.op_kv8_write(kv, x, x, i32(0))
    old = kv.k_scale.item()
    behind = kv.k.clone().view(torch.uint8)[:, :, 6:]
    bg.op_kv8_write(kv, x[:, :3] * 16, x[:, :3] * 16, i32(3))
    assert kv.k_scale.item() == 16 * old
    k, _ = bg.op_kv8_read(kv, i32(0), 32)
    assert (k[0, :3] == 1).all() and (k[0, 3:6] == 16).all() and (k[0, 6:] == 16).all()
    assert torch.equal(kv.k.view(torch.uint8)[:, :, 6:], behind)
