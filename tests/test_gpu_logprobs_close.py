"""How close the log probabilities and entropies are, with the longest chain of float32
additions taken from the kernel's own split: S = sum exp(d), d = z - max, relative error
   2^-24 (chain + joins) + 3 * 2^-22 (exponentials, rescalings) + 2^-23 E|d| (d log2 e
   rounded, and log2 e itself),
chain = V / (2 * threads of the row) additions in each of a thread's two sums, and at most
64 of lanes, warps and slices.  sum d exp(d) has the same, relative to sum |d| exp(d), and
2^-24 more for d.  Results are rounded a few times at the size of their largest part."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# rows, vocabulary, threads that share a row at least
@pytest.mark.parametrize("B,V,threads", [(1, 250880, 4096), (32, 250880, 4096), (509, 250880, 512), (700, 16000, 128), (5000, 2000, 128), (3, 700, 128)])
@pytest.mark.parametrize("std", [0.01, 1.0, 4.0, 30.0])
def test_close(B, V, threads, std):
    z = torch.randn(B, V, generator=torch.Generator(device=DEV).manual_seed(V + B), device=DEV) * std
    tok = torch.randint(0, V, (B, 4), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV, dtype=torch.int32)
    logp, ent, ids, tlp = bg.op_logprobs(z, tok, 5)
    step = max(1, B // 16)
    zd = z[::step].double()
    m = zd.amax(1, keepdim=True)
    d = zd - m
    p = torch.softmax(d, 1)
    far = (p * d.abs()).sum(1, keepdim=True)
    ls = torch.logsumexp(d, 1, keepdim=True)
    rel = 2.0 ** -24 * (V / (2 * threads) + 64) + 3 * 2.0 ** -22 + 2.0 ** -23 * far
    for got, at in ((logp, tok), (tlp, ids)):
        dd = d.gather(1, at[::step].long())
        tol = rel + 2.0 ** -24 * (dd.abs() + 2 * ls.abs() + (dd - ls).abs())
        err = (got[::step].double() - (dd - ls)).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
    ref = ls[:, 0] + far[:, 0]
    tol = (rel * (1 + 2 * far) + 2.0 ** -24 * (2 * ls.abs() + 3 * far + ref[:, None]))[:, 0]
    err = (ent[::step].double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
