"""Operators behind a kernel that lets them start early and writes what they read late: whatever the kernel before
writes (tiles, weights, activations, rows that are added to, logits, settings), a call finds it written."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg
from early_copy import early_copy

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16
SIZES = [(256, 512), (4096, 1024), (3000, 8200), (16384, 4096)]     # from fewer CTAs than SMs to many tiles a warp


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rand(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed + sum(7919 ** i * s for i, s in enumerate(shape)) % 2 ** 31)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def late(buf, contents, call, turns=6):
    """call() behind copies of contents[0], contents[1], ... in turn into buf that are late."""
    want = []
    for c in contents:
        buf.copy_(c)
        torch.cuda.synchronize()
        want.append(call())
        torch.cuda.synchronize()
    assert not all(torch.equal(a, b) for a, b in zip(want[0], want[1]))     # it shows which of them is read
    got = []
    for i in range(turns):
        early_copy(buf, contents[i & 1])
        got.append(call())
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i & 1])), i


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("M", [1, 8, 12, 40])
def test_tiles(M, n, k):
    q, x = [bg.op_w4_quantize(rand(n, k, seed=s, std=0.02), 64) for s in (0, 1)], rand(M, k)
    w4 = bg.W4.empty(n, k, 64)
    late(w4.tiles, [w.tiles for w in q], lambda: (bg.op_linear_w4(x, w4),))


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("M", [1, 8, 12, 40])
def test_activations_and_rows_added_to(M, n, k):
    w4, xs, ys = bg.op_w4_quantize(rand(n, k, std=0.02), 64), [rand(M, k, seed=s) for s in (0, 1)], [rand(M, n, seed=s) for s in (0, 1)]
    bias, x, y = [rand(n, seed=s) for s in (0, 1)], xs[0].clone(), ys[0].clone()
    b = bias[0].clone()
    late(x, xs, lambda: (bg.op_linear_w4(x, w4),))
    late(b, bias, lambda: (bg.op_linear_w4(x, w4, b),))
    late(y, ys, lambda: (bg.op_linear_w4(x, w4, epilogue=bg.EPI_RESID, y=y).clone(),))


@pytest.mark.parametrize("M", [1, 8])
def test_rows_added_to_and_then_read(M):
    """Layers that add to y and read it at once: an odd start puts two CTAs' numbers into one piece of a cache line."""
    n, steps = 4096, 12
    w4 = [bg.op_w4_quantize(rand(n, n, seed=s, std=0.02), 64) for s in range(2)]
    first, want = [rand(M, n, seed=s) for s in (5, 6)], []
    rooms = [torch.zeros(M * (n + 24), dtype=BF, device=DEV)[8:].as_strided((M, n), (n + 8, 1)) for _ in range(2)]

    def step(i):
        bg.op_linear_w4(rooms[i & 1], w4[i & 1], epilogue=bg.EPI_RESID, y=rooms[~i & 1])
    for apart in (True, False):
        for r, f in zip(rooms, first):
            r.copy_(f)
        for i in range(steps):
            step(i)
            if apart:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        want.append([r.clone() for r in rooms])
    assert all(torch.equal(a, b) for a, b in zip(*want))


@pytest.mark.parametrize("B,V", [(1, 1003), (1, 250880), (32, 50257), (400, 9001)])
def test_logits_and_settings(B, V):
    zs = [rand(B, V, seed=s, std=2.5, dtype=torch.float32) for s in (0, 1)]
    us = [torch.rand(B, 4, generator=torch.Generator(device=DEV).manual_seed(s), device=DEV) for s in (0, 1)]
    z, u = zs[0].clone(), us[0].clone()
    row = lambda v, dt=torch.float32: torch.full((B,), v, dtype=dt, device=DEV)
    t, k, p, mp = row(1.0), row(40, torch.int32), row(0.95), row(0.01)
    for f in (dict(), dict(top_k=k), dict(top_p=p), dict(min_p=mp), dict(temperature=row(0.0))):
        late(z, zs, lambda: (bg.op_sample_filtered(z, u, **f),))
    late(u, us, lambda: (bg.op_sample_filtered(z, u, t, k, p, mp),))
    hot = torch.full((B, 64), 0.999, device=DEV)       # far out, where a setting shows
    late(k, [row(2, torch.int32), row(700, torch.int32)], lambda: (bg.op_sample_filtered(z, hot, t, k),))
    late(p, [row(0.1), row(0.99)], lambda: (bg.op_sample_filtered(z, hot, t, None, p),))
    late(mp, [row(0.9), row(0.001)], lambda: (bg.op_sample_filtered(z, hot, t, None, None, mp),))
    late(t, [row(0.1), row(2.0)], lambda: (bg.op_sample_filtered(z, hot, t),))
    tok = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    late(z, zs, lambda: bg.op_logprobs(z, tok, 5))


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("op,M", [("op_linear", 1), ("op_linear", 5), ("op_linear", 40), ("op_linear_tc", 1), ("op_linear_tc", 8),
                                  ("op_linear_tc", 40), ("op_gemm", 300)])
def test_bf16_weights(op, M, n, k):
    layer, x, ws = getattr(bg, op), rand(M, k), [rand(n, k, seed=s, std=0.02) for s in (0, 1)]
    w, xs = ws[0].clone(), [rand(M, k, seed=s) for s in (0, 1)]
    late(w, ws, lambda: (layer(x, w),))
    late(x, xs, lambda: (layer(x, w),))


@pytest.mark.parametrize("n,k", [(256, 512), (16384, 4096)])
@pytest.mark.parametrize("op,M", [("op_linear", 1), ("op_linear", 5), ("op_linear_tc", 8), ("op_linear_tc", 40)])
def test_int8_weights(op, M, n, k):
    g = torch.Generator(device=DEV).manual_seed(3)
    qs = [torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    layer, x, q, scale = getattr(bg, op), rand(M, k), qs[0].clone(), rand(n, std=0.001)
    late(q, qs, lambda: (layer(x, q=q, scale=scale),))


@pytest.mark.parametrize("M", [1, 8])
def test_a_layers_output_as_weights(M):
    """Normalised rows, and another layer's output, as the next layer's matrix."""
    n, k = 2048, 1024
    layer = {1: bg.op_linear, 8: bg.op_linear_tc}[M]
    rows, x, one, zero = [rand(n, k, seed=s) for s in (0, 1)], rand(M, k), torch.ones(k, dtype=BF, device=DEV), torch.zeros(k, dtype=BF, device=DEV)
    square, w = rand(k, k, std=0.03), torch.empty(n, k, dtype=BF, device=DEV)
    for make in (lambda r: bg.op_layernorm(r, one, zero, y=w), lambda r: bg.op_gemm(r, square, y=w)):
        want = []
        for r in rows:
            make(r)
            torch.cuda.synchronize()
            want.append(layer(x, w))
            torch.cuda.synchronize()
        got = []
        for i in range(10):
            make(rows[i & 1])
            got.append(layer(x, w))
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i & 1]) for i, y in enumerate(got))


def test_lm_head():
    """Its scratch is cleared between the writer and the layer."""
    x, es = rand(4, 1024), [rand(30000, 1024, seed=s) for s in (0, 1)]
    e = es[0].clone()
    late(e, es, lambda: bg.op_lmhead_argmax(x, e))
    late(e, es, lambda: bg.op_lmhead_argmax_noalloc(x, e))
