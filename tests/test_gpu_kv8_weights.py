"""Decode attention over the 8-bit cache where the softmax weights' own rounding and
range show: outputs that cancel, V scales far apart with sparse blocks, and a key of
zeros that takes nearly all of the mass.

The bound is the one of kv8_plain.attend: scores off by es (float32 sums of exact
products), 2^-11 of sum p |V| at most for the weights, one bf16 rounding of the result.
Where 16 bits of the weights are asked for: the weight is held as two bf16 parts, the
first cut to 8 bits, the second (below 2^-7 of the weight) rounded to 8, half a step
2^-9 of it: 2^-16 of the weight, and 2^-21 for the exponential and the sums."""
import numpy as np
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import kv8_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [torch.int8, torch.float8_e4m3fn]
codes_param = pytest.mark.parametrize("codes", CODES, ids=["int8", "e4m3"])
# (T, query heads, key heads, d): one column a key head; 3; 8; 12 and 20 columns
FORMS = [(1, 2, 2, 64), (1, 2, 2, 128), (3, 2, 2, 64), (2, 8, 2, 128), (3, 8, 2, 64), (3, 8, 2, 128), (5, 4, 1, 128)]
forms_param = pytest.mark.parametrize("T,n,kv,d", FORMS)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def cache_of(k, v, codes):
    """k, v float64 [B][S][kv][d] (bf16 numbers) written to a cache; the values it stands for."""
    B, S, kv, d = k.shape
    c = bg.KV8.empty(B, kv, S, d, codes, DEV)
    bf = lambda x: torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    bg.op_kv8_write(c, bf(k), bf(v), torch.zeros(B, dtype=torch.int32, device=DEV))
    kf = plain.wide(plain.code_values(c.k), plain.f64(c.k_scale))
    vf = plain.wide(plain.code_values(c.v), plain.f64(c.v_scale))
    return c, kf, vf


def attend(c, kf, vf, q, slopes, lens, weight_error=2.0 ** -11):
    B, T, n, d = q.shape
    pos = torch.arange(c.k.shape[2], dtype=torch.int32).repeat(B, 1)
    qb = torch.from_numpy(q).to(torch.bfloat16)
    o = bg.op_attn_decode_kv8(qb.to(DEV), c, pos.to(DEV), torch.from_numpy(slopes).float().to(DEV),
                              torch.tensor(lens, dtype=torch.int32, device=DEV))
    ref, tol = plain.attend(plain.f64(qb), kf, vf, pos.numpy(), slopes, lens)
    if weight_error != 2.0 ** -11:      # sum p |V| as attend() has it, for V's magnitudes
        mass, _ = plain.attend(plain.f64(qb), kf, np.abs(vf), pos.numpy(), slopes, lens)
        tol = tol - (2.0 ** -11 - weight_error) * mass
    got = plain.f64(o).reshape(ref.shape)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol + 2.0 ** -134
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / (tol + 1e-300))[bad].max()), np.argwhere(bad)[:4].tolist())


@codes_param
@forms_param
@pytest.mark.parametrize("apart", [20, 26, 32, 60, 100])
def test_a_block_with_one_outlier_channel(codes, T, n, kv, d, apart):
    """Near-equal scores; one block's V is 2^apart in a single channel and 0 in the others,
    whose outputs come from the other blocks alone."""
    g = np.random.default_rng(apart + T + d)
    for first in (0, 64, 128):        # before, among and behind the others
        S = 160
        k = 0.1 * g.normal(size=(1, S, kv, d))
        v = g.normal(size=(1, S, kv, d))
        v[:, first:first + 32] = 0
        v[:, first + 5, :, 3] = 2.0 ** apart
        c, kf, vf = cache_of(k, v, codes)
        attend(c, kf, vf, 0.1 * g.normal(size=(1, T, n, d)), np.zeros(n), (S,))


@codes_param
@forms_param
@pytest.mark.parametrize("bits", [12, 18, 24, 30, 32, 60, 100])
@pytest.mark.parametrize("at", [3, 40, 2500])
def test_a_key_of_zeros_takes_the_mass(codes, T, n, kv, d, bits, at):
    """One key `bits` binades above all others, its V 0: the outputs are the others'."""
    g = np.random.default_rng(bits + T + d + at)
    S = 2600
    k = 0.02 * g.normal(size=(1, S, kv, d))
    k[:, :, :, 0] = 0
    k[:, at, :, 0] = 1.0
    v = g.normal(size=(1, S, kv, d))
    v[:, at] = 0
    q = 0.2 * g.normal(size=(1, T, n, d))
    q[..., 0] = bits * np.log(2.0) * np.sqrt(d)
    c, kf, vf = cache_of(k, v, codes)
    attend(c, kf, vf, q, np.zeros(n), (S,))


@codes_param
@forms_param
def test_steep_slopes_over_values_that_begin_late(codes, T, n, kv, d):
    """ALiBi slopes up to 1 a position, and channels whose recent values are all 0: what is
    left of them lies up to 2^-100 below the newest key's weight."""
    g = np.random.default_rng(T + d)
    S = 300
    k, v = 0.1 * g.normal(size=(1, S, kv, d)), g.normal(size=(1, S, kv, d))
    for e in range(d):
        v[:, S - 1 - e * 70 // d:, :, e] = 0
    c, kf, vf = cache_of(k, v, codes)
    attend(c, kf, vf, 0.1 * g.normal(size=(1, T, n, d)), np.linspace(0.2, 1.0, n), (S,))


@codes_param
@forms_param
def test_weights_have_sixteen_bits(codes, T, n, kv, d):
    """Two keys whose weighted values nearly cancel in every channel, so that neither the
    result's rounding nor that of the codes hides the weights'."""
    g = np.random.default_rng(7 * T + d)
    for ratio in (0.9, 0.77, 0.61, 0.53):
        k = np.zeros((1, 2, kv, d))
        k[:, 1, :, 0] = -1.0
        q = np.zeros((1, T, n, d))
        q[..., 0] = -np.log(ratio) * np.sqrt(d)
        q = plain.f64(torch.from_numpy(q).to(torch.bfloat16))
        real = np.exp(-q[0, -1, 0, 0] / np.sqrt(d))
        v = np.zeros((1, 2, kv, d))
        v[:, 1] = g.integers(64, 128, size=(kv, d))
        if codes is torch.float8_e4m3fn:
            v[:, 1] = plain.round_codes(v[:, 1], codes)
        v[:, 0] = -plain.round_codes(v[:, 1] * real, codes)
        v[:, 0, :, 0] = 127 if codes is torch.int8 else 448        # the block's scale is 1
        c, kf, vf = cache_of(k, v, codes)
        attend(c, kf, vf, q, np.zeros(n), (2,), weight_error=2.0 ** -16 + 2.0 ** -21)
