"""Log probabilities where many logits compete for the top places: many alternatives of
many short rows, rows ruled out by a finite value, ties, values that a few threads
hold alone.  Which tokens are on top is exact (kv8_plain.logprobs); and none of these
costs many times what ordinary rows cost."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import kv8_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def check(z, top, rows):
    """z float32 [B][V] on the device; the rows compared.  A probability's logarithm is off by
    the float32 sum of V exponentials, whatever their order (2^-24 V at most, and no more than
    2^-13 here, for the longest chain of additions is V / 128), and 2^-22 of its size."""
    B, V = z.shape
    tok = torch.full((B, 1), V // 2, dtype=torch.int32, device=DEV)
    logp, ent, ids, tlp = bg.op_logprobs(z, tok, top)
    rl, re, ri, rt = plain.logprobs(z[rows].double().cpu().numpy(), tok[rows].cpu().numpy(), top)
    assert np.array_equal(ids[rows].cpu().numpy(), ri)
    for got, ref in ((logp, rl), (tlp, rt)):
        got = plain.f64(got[rows])
        fin = np.isfinite(ref)
        assert np.array_equal(np.isfinite(got), fin)
        assert (np.abs(got[fin] - ref[fin]) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(ref[fin])).all()
    assert np.isfinite(plain.f64(ent)).all()


def normal(B, V, seed):
    return torch.randn(B, V, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 3


@pytest.mark.parametrize("V", [3000, 8191, 16000, 50000, 65535])
@pytest.mark.parametrize("top", [24, 25, 32])
def test_many_alternatives_of_many_short_rows(V, top):
    check(normal(700, V, V + top), top, slice(0, 700, 7))


# (rows, vocabulary): one CTA of 128 threads a row, of 512, clusters of 8
SHAPES = [(700, 5000), (700, 30000), (320, 50000), (5, 250880), (2, 600001)]


@pytest.mark.parametrize("B,V", SHAPES)
@pytest.mark.parametrize("top", [1, 5, 20, 32])
@pytest.mark.parametrize("ruled_out", [LOWEST, -1e9, -1e4, 0.0])
def test_finite_values_for_ruled_out_tokens(B, V, top, ruled_out):
    for allowed in (0, 3, 31, 200):
        z = torch.full((B, V), ruled_out, device=DEV)
        at = torch.randperm(V, generator=torch.Generator().manual_seed(allowed))[:allowed].to(DEV)
        z[:, at] = normal(B, allowed, allowed + top)
        check(z, top, slice(0, B, max(1, B // 2)))


@pytest.mark.parametrize("B,V", SHAPES)
@pytest.mark.parametrize("top", [5, 32])
def test_ascending_descending_and_tied(B, V, top):
    up = torch.arange(V, device=DEV).float() * 1e-3
    g = torch.Generator(device=DEV).manual_seed(top)
    few = torch.randint(0, 3, (V,), generator=g, device=DEV).float()
    steps = torch.floor(up * 2)
    for row in (up, -up, few, steps, -steps, torch.where(few > 1, -float("inf"), few)):
        check(row.repeat(B, 1), top, slice(0, B, max(1, B - 1)))


@pytest.mark.parametrize("B,V,span", [(700, 60000, 512), (700, 64000, 512), (2, 1 << 21, 2048), (400, 131072, 2048)])
@pytest.mark.parametrize("top", [2, 32])
def test_values_that_few_threads_hold(B, V, span, top):
    """Sixteen neighbours of every `span` logits hold all that takes part: a bound from
    several groups of threads finds none, or one far below them."""
    row = normal(1, V, V)[0]
    at = torch.arange(V, device=DEV) % span
    for rest in (-float("inf"), -50.0):
        for first in (0, 80):
            z = torch.where((at >= first) & (at < first + 16), row, torch.full_like(row, rest))
            check(z.repeat(B, 1), top, slice(0, B, max(1, B - 1)))


def gpu_us(z, top, flush):
    bg.op_logprobs(z, None, top)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        bg.op_logprobs(z, None, top)
    us = []
    for _ in range(15):
        flush.zero_()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        gr.replay()
        b.record()
        torch.cuda.synchronize()
        us.append(a.elapsed_time(b) * 1e3)
    return sorted(us)[len(us) // 2]


def test_finite_values_cost_little_more():
    """A finite value against -inf for ruled-out tokens, which leaves more candidates than are
    ranked: within four times (two more passes over the row; one for each alternative took 11
    times as long)."""
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    for B, V in [(700, 16000), (32, 250880)]:
        us = []
        for ruled_out in (-float("inf"), LOWEST, -1e9, 0.0):
            z = torch.full((B, V), ruled_out, device=DEV)
            z[:, 7:300:97] = 1.0
            us.append(gpu_us(z, 20, flush))
        assert max(us) < 4 * us[0], (B, V, us)


def test_the_most_alternatives_cost_little_more():
    """top 32 against top 16 for many short rows: within four times (3 to 22 times as long with
    CTAs of 128 threads for both)."""
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    for B, V in [(512, 8000), (700, 16000), (700, 50000), (700, 65000)]:
        z = normal(B, V, V)
        few, all32 = gpu_us(z, 16, flush), gpu_us(z, 32, flush)
        assert all32 < 4 * few, (B, V, few, all32)
