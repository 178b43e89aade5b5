"""Sampling with temperature, top-k, top-p and min-p on the GPU against its definition in float64."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import sample_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def run(z, u, t=None, k=None, p=None, mp=None):
    f = lambda x, dt: None if x is None else torch.as_tensor(x, dtype=dt, device=DEV)
    return bg.op_sample_filtered(z, f(u, torch.float32), f(t, torch.float32), f(k, torch.int32), f(p, torch.float32), f(mp, torch.float32))


def check(z, u, t, k, p, mp, exact=False):
    """Every draw against the definition; with `exact`, no allowance for draws beside a border."""
    zd = z if z.is_cuda else z.to(DEV)
    got = run(zd, u, t, k, p, mp)
    assert torch.equal(got, run(zd, u, t, k, p, mp))
    got, zc = got.cpu().numpy(), z.cpu().numpy()
    f32 = lambda x, off: [np.float32(off)] * len(zc) if x is None else np.asarray(x, dtype=np.float32)
    t, p, mp = f32(t, 1.0), f32(p, 1.0), f32(mp, 0.0)
    k = [0] * len(zc) if k is None else k
    u = np.asarray(u, dtype=np.float32).reshape(len(zc), -1)
    off = 0
    for b in range(len(zc)):
        kept = plain.kept_of(zc[b], float(t[b]), int(k[b]), float(p[b]), float(mp[b]))
        for j in range(u.shape[1]):
            g = int(got.reshape(len(zc), -1)[b, j])
            want = -1 if kept is None else plain.draw(kept, float(u[b, j]))
            if g != want:
                off += 1
                assert not exact, (b, j, g, want)
                assert plain.agrees(g, zc[b], float(t[b]), int(k[b]), float(p[b]), float(mp[b]), float(u[b, j])), (b, j, g, want)
    return off


def logits(B, V, std, seed=0, ruled_out=True):
    z = torch.randn(B, V, generator=torch.Generator().manual_seed(seed + B + V)) * std
    if ruled_out and V > 4:
        z[:, 3::97] = -torch.inf
    return z


MODES = {  # temperature, top-k, top-p, min-p of row b
    "chat": lambda b: (0.7 + 0.1 * (b % 5), 20 + 7 * b, 0.9 + 0.01 * (b % 9), 0.0),
    "nucleus": lambda b: (0.6 + 0.2 * (b % 4), 0, 0.5 + 0.49 * ((b * 7) % 10) / 10, 0.0),
    "minp": lambda b: (1.0 + 0.3 * (b % 3), 0, 1.0, 0.01 + 0.05 * (b % 6)),
    "k": lambda b: (1.1, 2 + 61 * b * b, 1.0, 0.0),
    "all": lambda b: (0.9 + 0.2 * (b % 3), 300 + 900 * b, 0.97, 0.001),
    "none": lambda b: (1.0, 0, 1.0, 0.0),
}


def settings(mode, B):
    return [list(x) for x in zip(*(MODES[mode](b) for b in range(B)))]


def uniforms(B, J, seed=0):
    return np.random.default_rng(seed + 1000 * B + J).random((B, J), dtype=np.float32)


@pytest.mark.parametrize("B,V,J", [(1, 1, 1), (2, 2, 3), (3, 5, 4), (4, 31, 5), (7, 1003, 20), (5, 4096, 33), (6, 4097, 17), (9, 9001, 8),
                                   (3, 50257, 40), (4, 250880, 64), (40, 32003, 2), (700, 1203, 1), (320, 33000, 1)])
@pytest.mark.parametrize("mode", list(MODES))
def test_against_the_definition(B, V, J, mode):
    z = logits(B, V, 2.5)
    off = check(z, uniforms(B, J), *settings(mode, B))
    assert off <= 1 + B * J // 100      # draws beside a border are rare


@pytest.mark.parametrize("std", [0.001, 0.05, 1.0, 8.0])
@pytest.mark.parametrize("mode", ["nucleus", "all", "none"])
def test_flat_and_peaked_rows(std, mode):
    """Flat rows: bands of more tokens than the list holds; peaked ones: a few tokens with all mass."""
    z = logits(4, 250880, std, ruled_out=False)
    check(z, uniforms(4, 32, 1), *settings(mode, 4))


@pytest.mark.parametrize("levels", [1, 2, 3, 17])
@pytest.mark.parametrize("V", [900, 5000, 100001])
@pytest.mark.parametrize("k,p", [(0, 0.5), (7, 1.0), (3000, 1.0), (3000, 0.9), (0, 0.999), (60000, 0.5), (0, 1.0)])
def test_ties(levels, V, k, p):
    """Few values, many tokens of each: the cut falls among equal logits, which are kept by index."""
    z = (torch.arange(V) * 7919 % levels).float().repeat(3, 1)
    check(z, uniforms(3, 40, levels), [1.0, 0.5, 3.0], [k] * 3, [p] * 3, None)


def test_greedy_and_switched_off_settings():
    z = logits(10, 3000, 2.0)
    z[:, 777] = z[:, 5] = z.amax() + 1
    nan = float("nan")
    t = [0.0, -1.0, nan, 1.0, 1.0, 0.7, 0.7, 0.7, 0.7, 0.7]
    k = [0, 5, 0, 1, 0, 0, -3, 5000, 0, 0]
    p = [1.0, 1.0, 0.9, 1.0, 0.0, -0.5, 1.0, 2.0, nan, 1.0]
    m = [0.0, 0.1, 0.0, 0.0, 0.0, 0.0, 0.0, -1.0, 0.0, nan]
    u = uniforms(10, 6)
    got = run(z.to(DEV), u, t, k, p, m).cpu()
    assert (got[:6] == 5).all()
    for b in range(6, 10):                      # as with no settings but the temperature
        assert torch.equal(got[b], run(z[b:b + 1].to(DEV), u[b:b + 1], [0.7]).cpu()[0])
    ones = run(z.to(DEV), u, [1.0] * 10, None, None, [1.0] * 10).cpu()
    assert ((ones == 5) | (ones == 777)).all() and (ones == 777).any() and (ones == 5).any()


def test_uniforms_at_the_ends():
    z = logits(1, 1000, 1.0)
    u = np.array([[0.0, -1.0, float("nan"), 1.0, 2.0, float("inf"), 1.0 - 2.0 ** -24]], dtype=np.float32)
    got = run(z.to(DEV), u, [1.0], [50]).cpu()[0].tolist()
    tokens = plain.kept_of(z[0].numpy(), 1.0, 50, 1.0, 0.0)[0]
    assert got == [tokens[0]] * 3 + [tokens[-1]] * 4


@pytest.mark.parametrize("k", [50, 0])
@pytest.mark.parametrize("V", [1000, 90000])
def test_the_smallest_uniforms(V, k):
    """-0, subnormal and tiny numbers take the first kept token; so does a top-p next to 0."""
    z = logits(1, V, 1.0)
    u = np.array([[-0.0, 1e-45, 1e-40, 1.2e-38, 1e-30, -1e-40]], dtype=np.float32)
    got = run(z.to(DEV), u, [1.0], [k], [0.9]).cpu()[0]
    assert (got == int(plain.kept_of(z[0].numpy(), 1.0, k, 0.9, 0.0)[0][0])).all()
    for p in (1e-45, 1e-39, 1e-20):
        assert (run(z.to(DEV), u, [1.0], [k], [p]).cpu() == int(z[0].argmax())).all()


def test_infinities_nan_and_empty_rows():
    z = logits(8, 6000, 1.5)
    z[0] = -torch.inf
    z[1] = float("nan")
    z[2, 100] = z[2, 5000] = torch.inf
    z[3, ::2] = float("nan")
    z[4] = -torch.inf
    z[4, 4321] = -3.0
    z[5, 7] = 0.0
    z[5, 3] = -0.0
    z[5, 8:] = -torch.inf
    z[5, :3] = z[5, 4:7] = -5.0
    z[6] = torch.inf
    u = uniforms(8, 16)
    for k, p, m in ((0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.7, 0.0), (5, 0.7, 0.2), (1, 1.0, 0.0)):
        check(z, u, [1.0] * 8, [k] * 8, [p] * 8, [m] * 8)
    got = run(z.to(DEV), u, [1.0] * 8, [1] * 8).cpu()
    assert (got[0] == -1).all() and (got[1] == -1).all() and (got[2] == 100).all() and (got[4] == 4321).all()
    assert (got[5] == 3).all()                  # -0 and 0 are equal logits
    assert set(run(z.to(DEV), u).cpu()[2].tolist()) == {100, 5000}


@pytest.mark.parametrize("scale,shift", [(1.0, 1e6), (1e-3, 100.0), (1e30, 0.0), (1e-30, 0.0), (3e37, 0.0)])
@pytest.mark.parametrize("t", [1.0, 1e-6, 1e6, 1e-38, float("inf"), 1e38])
def test_far_out_sizes(scale, shift, t):
    z = logits(3, 5003, 1.0) * scale + shift
    check(z, uniforms(3, 12), [t] * 3, [0, 40, 0], [0.9, 1.0, 1.0], [0.0, 0.0, 0.05])


def test_distribution_on_a_grid():
    """Draws at the midpoints of a grid count the kept tokens by their probabilities."""
    z = logits(1, 5000, 2.0)
    n = 1 << 16
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)[None]
    got = run(z.to(DEV), u, [0.8], [30], [0.95]).cpu().numpy()[0]
    tokens, prob = plain.kept_of(z[0].numpy(), float(np.float32(0.8)), 30, float(np.float32(0.95)), 0.0)
    assert set(got.tolist()) <= set(tokens.tolist()) and (np.diff(got) >= 0).all()
    for tok, pr in zip(tokens, prob):
        assert abs((got == tok).sum() - pr * n) <= 1.5


def test_strided_rows_and_outputs():
    wide = logits(5, 3000, 2.0).to(DEV)
    z = wide[:, 1:2990]                         # rows at odd addresses
    u = torch.as_tensor(uniforms(5, 1)[:, 0]).to(DEV)
    k = torch.full((5,), 40, dtype=torch.int32, device=DEV)
    out = torch.full((5,), -7, dtype=torch.int32, device=DEV)
    got = bg.op_sample_filtered(z, u, top_k=k, out=out)
    assert got is out and torch.equal(got, bg.op_sample_filtered(z.contiguous(), u, top_k=k))
    check(z.cpu(), u.cpu().numpy(), None, [40] * 5, None, None)
    assert bg.op_sample_filtered(z[:0], u[:0]).shape == (0,)
    assert bg.op_sample_filtered(z, torch.empty(5, 0, device=DEV)).shape == (5, 0)


def test_agrees_with_top_p_sampling():
    """With temperature and top-p alone it draws what op_sample draws, but beside borders."""
    z = logits(64, 50257, 2.0).to(DEV)
    u = torch.as_tensor(uniforms(64, 1)[:, 0]).to(DEV)
    t, p = torch.full((64,), 0.8, device=DEV), torch.full((64,), 0.9, device=DEV)
    same = bg.op_sample_filtered(z, u, t, None, p) == bg.op_sample(z, t, p, u)
    assert int((~same).sum()) <= 1


def test_streams_and_graphs():
    z, z2 = logits(6, 60000, 2.0).to(DEV), logits(6, 60000, 2.0, 5).to(DEV)
    u = torch.as_tensor(uniforms(6, 4)).to(DEV)
    k, p = torch.full((6,), 200, dtype=torch.int32, device=DEV), torch.full((6,), 0.9, device=DEV)
    want, want2 = bg.op_sample_filtered(z, u, None, k, p), bg.op_sample_filtered(z2, u, None, k, p)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(bg.op_sample_filtered(z, u, None, k, p, stream=s1), bg.op_sample_filtered(z2, u, None, k, p, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want2) for a, b in outs)
    buf, out = z.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.op_sample_filtered(buf, u, None, k, p, out=out)
    for src, res in ((z, want), (z2, want2), (z, want)):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, res)


@pytest.mark.parametrize("k,p", [(0, 0.5), (0, 1.0), (3000000, 1.0), (100, 0.5)])
@pytest.mark.parametrize("B", [1, 310])
def test_longest_rows_of_equal_logits(B, k, p):
    """The largest sums of masses that there are: 2^22 tokens of the maximum's."""
    V = 1 << 22
    z = torch.full((1, V), -1.5, device=DEV).expand(B, V).contiguous()
    u = np.tile(np.array([[0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24]], dtype=np.float32), (B, 1))
    got = run(z, u, [0.7] * B, [k] * B, [p] * B).cpu()
    kept = min(k or V, V)
    kept = kept if p == 1.0 else int(kept * p)
    want = [min(int(float(x) * kept), kept - 1) for x in u[0]]
    assert (got == torch.tensor(want, dtype=torch.int32)).all()


def test_rows_of_other_lengths_side_by_side():
    """Lengths around those at which clusters and lists change."""
    for V in (511, 512, 513, 8191, 8192, 8193, 65535, 65536, 131072):
        z = logits(3, V, 2.0)
        check(z, uniforms(3, 5), [0.9] * 3, [0, 60, 0], [0.8, 1.0, 1.0], [0.0, 0.0, 0.02])
    for B in (4, 5, 38, 39, 152, 153, 304, 305):
        z = logits(B, 70000 if B > 300 else 9000, 2.0)
        check(z, uniforms(B, 1), [0.9] * B, [0] * B, [0.5 + 0.4 * (b % 3) / 2 for b in range(B)], None)


def test_the_most_rows():
    """65535 short rows: as many rows of the same values in smaller calls."""
    z = logits(65535, 9, 2.0).to(DEV)
    u = torch.rand(65535, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    t, p = torch.full((65535,), 0.8, device=DEV), torch.full((65535,), 0.9, device=DEV)
    k = torch.arange(65535, device=DEV, dtype=torch.int32) % 7
    got = bg.op_sample_filtered(z, u, t, k, p)
    for a in (0, 30000, 65435):
        at = slice(a, a + 100)
        assert torch.equal(got[at], bg.op_sample_filtered(z[at], u[at], t[at], k[at], p[at]))
        for b in range(a, a + 100):
            assert plain.agrees(int(got[b]), z[b].cpu().numpy(), float(t[b]), int(k[b]), float(p[b]), 0.0, float(u[b]))
