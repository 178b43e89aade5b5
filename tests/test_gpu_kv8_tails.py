"""Rows whose last slots are all masked (prompts padded on the right, slots taken back):
positions count from the highest one left, however far back it lies, and finding it does
not hold a call up."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import kv8_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("T,n,kv,d", [(1, 4, 4, 64), (1, 2, 2, 128), (2, 8, 2, 128), (5, 4, 1, 64)])
def test_masked_tails(codes, T, n, kv, d):
    g = torch.Generator().manual_seed(T + d)
    S = 1700
    tails = [0, 31, 32, 33, 64, 500, 543, 544, 545, 600, 1056, 1057, 1690]
    B = len(tails)
    cache = bg.KV8.empty(B, kv, S, d, codes, DEV)
    x = torch.randn(2, B, S, kv, d, generator=g).to(torch.bfloat16).to(DEV)
    bg.op_kv8_write(cache, x[0], x[1], torch.zeros(B, dtype=torch.int32, device=DEV))
    lens = [S - 3 * b for b in range(B)]
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1) + 3_000_000      # as of rows that were cut
    for b, tail in enumerate(tails):
        pos[b, max(0, lens[b] - tail):] = -1
    q = torch.randn(B, T, n, d, generator=g).to(torch.bfloat16)
    slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / n) for i in range(n)])
    o = bg.op_attn_decode_kv8(q.to(DEV), cache, pos.to(DEV), slopes.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    kf, vf = (plain.wide(plain.code_values(c), plain.f64(s)) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    ref, tol = plain.attend(plain.f64(q), kf, vf, pos.numpy(), plain.f64(slopes), lens)
    got = plain.f64(o).reshape(ref.shape)
    assert (np.abs(got - ref) <= tol + 2.0 ** -134).all()


def test_a_long_masked_tail_holds_nothing_up():
    """A batch with rows that are masked but for their first slots, 100000 long: within five
    times the time of the same rows unmasked (ten times with one load of 32 positions after the
    other)."""
    B, n, d, S = 4, 16, 64, 100_000
    cache = bg.KV8.empty(B, n, S, d, torch.int8, DEV)
    q = torch.randn(B, 1, n, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    slopes = torch.full((n,), 0.1, device=DEV)
    us = []
    for seen in (S, 5, 0):
        pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
        pos[:, seen:] = -1
        pos = pos.to(DEV)
        t = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            o = bg.op_attn_decode_kv8(q, cache, pos, slopes, lens)
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b) * 1e3)
        us.append(sorted(t)[len(t) // 2])
    assert max(us) < 5 * us[0], us
