"""Filtered sampling at the ends of the floats' range: logits further apart than the largest float, which
take no part; temperatures from subnormal ones, which count as 2^-126, to infinity."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import sample_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
SETTINGS = [dict(), dict(k=20), dict(p=0.9), dict(mp=0.2), dict(k=400, p=0.95, mp=0.01)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def check(z, t, k=0, p=1.0, mp=0.0, J=48):
    B = len(z)
    u = np.random.default_rng(z.shape[1]).random((B, J), dtype=np.float32)
    row = lambda v, dt: torch.full((B,), v, dtype=dt, device=DEV)
    got = bg.op_sample_filtered(z.to(DEV), torch.from_numpy(u).to(DEV), t.to(DEV), row(k, torch.int32), row(p, torch.float32),
                                row(mp, torch.float32)).cpu().numpy()
    p, mp, zc, t = float(np.float32(p)), float(np.float32(mp)), z.numpy(), t.clamp(min=2.0 ** -126)
    with np.errstate(over="ignore"):
        zc = np.where(zc.max(1, keepdims=True) - zc < np.inf, zc, -np.inf)
    for b in range(B):
        for j in range(J):
            assert plain.agrees(int(got[b, j]), zc[b], float(t[b]), k, p, mp, float(u[b, j])), (b, j, int(got[b, j]))


@pytest.mark.parametrize("f", SETTINGS)
@pytest.mark.parametrize("V", [4, 1003, 20000])
def test_logits_further_apart_than_the_largest_float(V, f):
    t = torch.tensor([2.0 ** 99, 2.0 ** 100, 2.0 ** 120, 1e38, 3e38, float("inf")])
    z = (torch.rand(len(t), V, generator=torch.Generator().manual_seed(V)) * 2 - 1) * 3.4e38
    z[:, :2] = torch.tensor([3.4e38, -3.4e38])      # the others' differences to the maximum are floats or not
    z[1::2, 3] = -torch.inf
    check(z, t, **f)
    check(z * 2.0 ** -2, t, **f)       # all are
    check(z * 2.0 ** -27, t, **f)


@pytest.mark.parametrize("f", SETTINGS)
@pytest.mark.parametrize("V", [4, 1003, 20000])
def test_subnormal_temperatures(V, f):
    """Subnormal logits a few temperatures apart; then ordinary ones, of which only the largest have mass."""
    bits = torch.tensor([1, 7, 1000, 2 ** 22, 2 ** 23 - 1, 2 ** 23], dtype=torch.int32)
    t = bits.view(torch.float32)
    near = torch.randint(0, 12, (len(t), V), generator=torch.Generator().manual_seed(V), dtype=torch.int32)
    check((near * bits[:, None] // 2).view(torch.float32), t, **f)
    check(near.float(), t, **f)
    check(near.float() * 2.0 ** 120, t, **f)
