"""Log probabilities, entropy and top alternatives (bloom_op_logprobs) against the plain
float64 form.  Which tokens are on top is exact; values: the maximum is subtracted
exactly rounded (2^-24 of the difference), the sum of V exponentials is float32
(relative error at most 2^-24 times the exponent's size, the exponential's own few
ulps, and the longest chain of additions, V / 512 + 32), and one rounding at the end."""
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


def check(z, tokens, top, view=None):
    """z float32 [B][V] on the host; tokens int32 [B][J]; view: the device logits to pass."""
    zd = z.to(DEV) if view is None else view
    logp, ent, ids, tlp = bg.op_logprobs(zd, tokens.to(DEV), top)
    again = bg.op_logprobs(zd, tokens.to(DEV), top)
    for a, b in zip((logp, ent, ids, tlp), again):
        assert torch.equal(a.nan_to_num(7e7), b.nan_to_num(7e7))
    rl, re, ri, rt = plain.logprobs(z.double().numpy(), tokens.numpy(), top)
    assert ids.shape == ri.shape and np.array_equal(ids.cpu().numpy(), ri)
    V = z.shape[1]
    rel = 2.0 ** -24 * (V / 512 + 64)

    def near(got, ref, size):
        got = plain.f64(got)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(np.isinf(got), np.isinf(ref)) and (got[np.isinf(ref)] < 0).all()
        ok = np.isfinite(ref)
        err = np.abs(got[ok] - ref[ok])
        assert (err <= size(np.abs(ref[ok]))).all(), float(err.max())

    near(logp, rl, lambda r: rel + 2.0 ** -22 * r)
    near(tlp, rt, lambda r: rel + 2.0 ** -22 * r)
    # sum d e^d / S: every term has the relative error above, and |d| up to ~30 where e^d counts
    near(ent, re, lambda r: 32 * rel + 2.0 ** -22 * r)


def rows(V, seed):
    g = np.random.default_rng(seed)
    r = [g.normal(size=V) * 2.0, g.normal(size=V) * 6.0, np.round(g.normal(size=V) * 3.0, 1),   # ties
         np.zeros(V), np.arange(V) * 1e-3, -np.arange(V) * 1e-3, g.normal(size=V) * 2.0, g.normal(size=V),
         np.full(V, -np.inf), g.normal(size=V) * 1e4, g.normal(size=V), np.full(V, np.nan), -np.zeros(V), g.normal(size=V) + 3.0]
    r[6][g.choice(V, V // 2, replace=False)] = -np.inf
    r[7][g.choice(V, V // 3, replace=False)] = np.nan
    r[8][V // 2] = 1.5                      # one token left
    r[10][[0, V // 2]] = np.inf
    r[12][V // 2:] = 0.0                    # -0 and +0 are equal
    return torch.tensor(np.stack(r), dtype=torch.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099, 50021, 250880, 600001])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_rows(V, top):
    z = rows(V, V)
    B = len(z)
    g = torch.Generator().manual_seed(V)
    tokens = torch.randint(0, V, (B, 3), generator=g, dtype=torch.int32)
    tokens[0] = torch.tensor([-1, -2, V])
    tokens[1, 0] = 2 ** 31 - 1
    tokens[2, 0] = -2 ** 31
    check(z, tokens, top)


@pytest.mark.parametrize("period", [2048, 512, 4096, 64, 31360])
def test_large_logits_at_regular_places(period):
    """The highest logits at a fixed stride, and bunched: places that one thread, warp or
    slice of a kernel would own alone."""
    V = 250880
    g = np.random.default_rng(period)
    z = g.normal(size=(4, V))
    n = len(range(7, V, period))
    z[0, 7::period] += 50 + g.random(n)
    z[1, 7::period] = 60.0                                # equal
    z[2, 1000:1000 + 700] += 40
    z[3, :] = np.sort(z[3])
    z[3, ::period] = z[3, ::period][::-1]
    check(torch.tensor(z, dtype=torch.float32), torch.tensor([[7], [7 + period], [1003], [5]], dtype=torch.int32), 32)


@pytest.mark.parametrize("B", [2, 200])
def test_vocabularies_ruled_out_in_bulk(B):
    """Rows whose logits are -inf but for one range, or for every k-th token: the range begins
    late in a slice, in its last round, or at the row's end."""
    V = 250880
    g = torch.Generator().manual_seed(B)
    z = torch.full((B, V), -float("inf"))
    for b in range(B):
        lo = (200_000, 12_345, 250_000, 31_360 + 20_480, 0, 123_456)[b % 6]
        n = (50_000, 20_000, 880, 9_000, 5, 1)[b % 6]
        n = min(n, V - lo)
        z[b, lo:lo + n] = torch.randn(n, generator=g) * 3
    z[0, :] = -float("inf")
    z[0, 77::1009] = torch.randn(len(range(77, V, 1009)), generator=g)
    check(z, torch.full((B, 1), 200_001, dtype=torch.int32), 20)


@pytest.mark.parametrize("V", [2000, 2049, 7001])
@pytest.mark.parametrize("B", [1, 3, 40, 700])
def test_row_counts_and_strides(B, V):
    g = torch.Generator().manual_seed(B)
    buf = torch.randn(B, V + 13, generator=g)
    d = buf.to(DEV)
    tokens = torch.randint(0, V, (B, 1), generator=g, dtype=torch.int32)
    for off in (0, 1, 5):      # rows that start at any float
        check(buf[:, off:off + V].contiguous(), tokens, 4, view=d[:, off:off + V])


def test_tokens_of_one_dimension_none_and_no_rows():
    z = torch.randn(3, 100, generator=torch.Generator().manual_seed(1)).to(DEV)
    t = torch.tensor([4, -1, 99], dtype=torch.int32, device=DEV)
    logp, ent, ids, tlp = bg.op_logprobs(z, t)
    assert logp.shape == (3,) and ids.shape == (3, 0) and logp[1] == 0
    ref = torch.log_softmax(z.double(), 1)[[0, 2], [4, 99]].float()
    assert torch.allclose(logp[[0, 2]], ref, rtol=1e-6, atol=1e-6)
    none, ent2, ids, tlp = bg.op_logprobs(z, top=2)
    assert none is None and torch.equal(ent, ent2) and ids.shape == (3, 2)
    logp, ent, ids, tlp = bg.op_logprobs(z[:0], t[:0], 3)
    assert logp.shape == (0,) and ent.shape == (0,) and ids.shape == (0, 3)


def test_rows_past_two_gigabytes_of_offset():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    B, V = 2, 1000
    buf = torch.zeros(2, (1 << 31) + 64, device=DEV)
    view = buf[:, :V]
    z = torch.randn(B, V, generator=torch.Generator().manual_seed(2))
    view.copy_(z)
    check(z, torch.tensor([[3], [999]], dtype=torch.int32), 5, view=view)
