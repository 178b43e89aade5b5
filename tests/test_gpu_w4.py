"""4-bit weights on the GPU: quantising, reading back and the linear layer against plain
float64 forms, over sizes, groups, token counts, strides, epilogues and odd values."""
import pytest
import torch

import bloom_decoder_token_gb300 as bg
import sample_plain
import w4_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def weights(n, k, seed=0, std=0.02):
    g = torch.Generator(device=DEV).manual_seed(seed + 7919 * n + k)
    w = torch.randn(n, k, generator=g, device=DEV) * std
    w[:, 5::61] *= 4.0
    return w.to(torch.bfloat16)


def acts(M, k, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * M + k)
    x = torch.randn(M, k, generator=g, device=DEV)
    x[:, 7::113] *= 30.0
    return x.to(torch.bfloat16)


def check(y, want, far):
    eps = torch.finfo(y.dtype).eps / 2
    off = (y.double() - want).abs()
    assert (off <= want.abs() * eps + far * (1 + eps)).all(), (off - want.abs() * eps - far).max()


# ------------------------------------------------------------ quantise, read back
@pytest.mark.parametrize("n,k", [(1, 8), (16, 256), (17, 264), (5, 72), (100, 1000), (33, 4096), (1000, 520)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_and_read(n, k, group):
    w = weights(n, k)
    got = bg.op_w4_read(bg.op_w4_quantize(w, group))
    # the values to the bit: codes and scales as in exact arithmetic, their product rounded once
    assert torch.equal(got.double(), plain.bf16_of(plain.values(w, group)))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_bf16_magnitude(group):
    """Groups whose largest weight takes every positive finite bf16 value, the others spread below it, ties among
    them: multiples of an eighth of it."""
    top = torch.arange(1, 0x7F80, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    part = (torch.arange(group, device=DEV) % 17 - 8).float() / 8
    w = (top.float()[:, None] * part).to(torch.bfloat16)
    w[:, 8] = top
    got = bg.op_w4_read(bg.op_w4_quantize(w, group))
    assert torch.equal(got.double(), plain.bf16_of(plain.values(w, group)))


def test_ties_go_to_the_even_code():
    w = torch.zeros(2, 32, device=DEV)
    w[0, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 6.5])
    w[1, :8] = w[0, :8] * 2.0 ** -100
    want = torch.tensor([7.0, 0.0, 2.0, 2.0, 0.0, -2.0, -2.0, 6.0], device=DEV)
    got = bg.op_w4_read(bg.op_w4_quantize(w.to(torch.bfloat16), 32))
    assert torch.equal(got[0, :8].float(), want) and torch.equal(got[1, :8].float(), want * 2.0 ** -100)


def test_zero_nan_and_infinite_groups():
    w = weights(4, 192).float()
    w[0, :64] = 0.0
    w[1, 70] = float("inf")
    w[2, 10] = float("nan")
    w[3, 64:128] = 2.0 ** -133          # the scale rounds to 0
    w = w.to(torch.bfloat16)
    got = bg.op_w4_read(bg.op_w4_quantize(w, 64))
    want = plain.bf16_of(plain.values(w, 64))
    assert torch.isnan(got[1, 64:128]).all() and torch.isnan(got[2, :64]).all()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.double().nan_to_num(0.0), want.nan_to_num(0.0))
    assert (got[3, 64:128] == 0).all()


def test_strided_rows_and_reuse():
    wide = weights(50, 512)
    w = wide[:, 128:392]                # 264 columns, rows 512 apart, 16-byte aligned
    w4 = bg.op_w4_quantize(w, 64)
    again = bg.op_w4_quantize(w.contiguous(), 64, out=bg.W4(torch.full_like(w4.tiles, 255), 50, 264, 64))
    assert torch.equal(again.tiles, w4.tiles)        # every byte is written
    out = torch.full((50, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    bg.op_w4_read(w4, out[:, 64:328])
    assert torch.equal(out[:, 64:328], bg.op_w4_read(w4))
    assert (out[:, :64] == 3).all() and (out[:, 328:] == 3).all()


# ------------------------------------------------------------ the linear layer
SHAPES = [  # tokens in one to eight column tiles and several blocks; one to eight CTAs a cluster, passes, chunks
    (1, 1, 8), (1, 16, 256), (1, 4096, 1024), (2, 100, 264), (3, 1000, 4096), (4, 17, 4104), (5, 333, 1000),
    (7, 2100, 8200), (8, 64, 16384), (9, 48, 520), (16, 1003, 4096), (13, 40, 12296), (17, 129, 2048), (31, 500, 2056),
    (32, 4096, 1024), (24, 64, 16392), (33, 100, 776), (64, 257, 2304), (65, 33, 264), (200, 40, 512),
    (2, 33, 33000), (12, 20, 40968), (20, 24, 20000), (1, 90000, 4360), (20, 12000, 2112), (10, 20000, 4608),
    (1, 40000, 64), (12, 90000, 520), (50, 45000, 264), (300, 5000, 512),
]


@pytest.mark.parametrize("M,n,k", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear(M, n, k, group):
    w, x = weights(n, k), acts(M, k)
    w4 = bg.op_w4_quantize(w, group)
    want, far = plain.linear(x, plain.values(w, group), group=group)
    y = bg.op_linear_w4(x, w4, dtype=torch.float32)
    check(y, want, far)
    z = bg.op_linear_w4(x, w4)
    assert torch.equal(z, y.to(torch.bfloat16))          # the same sums, rounded
    assert torch.equal(y, bg.op_linear_w4(x, w4, dtype=torch.float32))


@pytest.mark.parametrize("M,n,k", [(1, 100, 264), (6, 500, 4104), (16, 33, 1024), (40, 70, 2304)])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("epilogue", [0, 1, 2], ids=["store", "gelu", "resid"])
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
def test_epilogues(M, n, k, f32, epilogue, bias):
    g = torch.Generator(device=DEV).manual_seed(M)
    w, x = weights(n, k, 1), acts(M, k, 1)
    b = torch.randn(n, generator=g, device=DEV).to(torch.bfloat16) if bias else None
    y0 = torch.randn(M, n, generator=g, device=DEV).to(torch.float32 if f32 else torch.bfloat16)
    y = y0.clone() if epilogue == 2 else None
    got = bg.op_linear_w4(x, bg.op_w4_quantize(w, 64), b, epilogue, y, dtype=y0.dtype)
    assert got.dtype == y0.dtype and (y is None or got is y)
    check(got, *plain.linear(x, plain.values(w, 64), b, epilogue, y0, group=64))


def test_strided_activations_and_outputs():
    M, n, k = 5, 70, 520
    w, wide = weights(n, k), acts(M, 1024)
    x = wide[:, 8:528]
    out = torch.full((M, 200), 3.0, device=DEV)
    w4 = bg.op_w4_quantize(w, 32)
    got = bg.op_linear_w4(x, w4, y=out[:, 50:120])
    assert torch.equal(got, bg.op_linear_w4(x.contiguous(), w4, dtype=torch.float32))
    assert (out[:, :50] == 3).all() and (out[:, 120:] == 3).all()


def test_rows_of_activations_are_their_own():
    """A token's outputs do not depend on the tokens beside it, up to the tiles that the count picks."""
    w4, x = bg.op_w4_quantize(weights(200, 4608), 64), acts(32, 4608)
    for M, step in ((4, 1), (8, 5), (16, 9), (32, 17)):
        a = bg.op_linear_w4(x[:M], w4, dtype=torch.float32)
        for m in range(step, M + 1):
            assert torch.equal(bg.op_linear_w4(x[:m], w4, dtype=torch.float32), a[:m])


def test_activations_of_far_apart_sizes():
    """Outliers far above the others lose nothing; one that is larger still costs what the tolerance says."""
    M, n, k = 6, 64, 1024
    w, x = weights(n, k), acts(M, k).float()
    x[:, 3::256] *= 2.0 ** 9
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 60
    x[3, 256:512] *= 2.0 ** -40
    x[4, 9] = 2.0 ** 40
    x[5] = 0.0
    x = x.to(torch.bfloat16)
    w4 = bg.op_w4_quantize(w, 64)
    check(bg.op_linear_w4(x, w4, dtype=torch.float32), *plain.linear(x, plain.values(w, 64)))


def test_many_tokens_of_far_apart_sizes():
    M, n, k = 20, 64, 1024
    w, x = weights(n, k), acts(M, k).float()
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 60
    x[3, 256:512] *= 2.0 ** -40
    x[4, 9] = 2.0 ** 40
    x[5] = 0.0
    x[6] = 0.0
    x[6, 1000] = 2.0 ** -133
    x = x.to(torch.bfloat16)
    w4 = bg.op_w4_quantize(w, 64)
    check(bg.op_linear_w4(x, w4, dtype=torch.float32), *plain.linear(x, plain.values(w, 64), group=64))


def test_small_activations_beside_large_ones_of_zero_weight():
    """A large activation whose own weight is 0 hides nothing of the others."""
    n, k = 16, 256
    w = torch.zeros(n, k, device=DEV)
    w[:, 100:132] = 7.0 * 0.01
    x = torch.full((1, k), 1.0, device=DEV)
    x[0, 0] = 2.0 ** 13
    x = x.to(torch.bfloat16)
    w = w.to(torch.bfloat16)
    got = bg.op_linear_w4(x, bg.op_w4_quantize(w, 32), dtype=torch.float32)
    want = x.double() @ plain.values(w, 32).t()
    assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -20).all()


def test_nan_and_infinities():
    w, x = weights(40, 600), acts(9, 600)
    clean = bg.op_linear_w4(x, bg.op_w4_quantize(w, 64), dtype=torch.float32)
    x2 = x.clone()
    x2[3, 599] = float("nan")
    x2[5, 0] = float("inf")
    got = bg.op_linear_w4(x2, bg.op_w4_quantize(w, 64), dtype=torch.float32)
    bad = torch.tensor([3, 5], device=DEV)
    assert torch.isnan(got[bad]).all()
    ok = [i for i in range(9) if i not in (3, 5)]
    assert torch.equal(got[ok], clean[ok])
    w[7, 70] = float("nan")             # a weight of one row
    got = bg.op_linear_w4(x, bg.op_w4_quantize(w, 64), dtype=torch.float32)
    assert torch.isnan(got[:, 7]).all()
    got[:, 7] = clean[:, 7]
    assert torch.equal(got, clean)


def test_no_tokens():
    w4 = bg.op_w4_quantize(weights(40, 64), 32)
    assert bg.op_linear_w4(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), w4).shape == (0, 40)


@pytest.mark.parametrize("M,n,k", [(3, 40000, 4608), (1, 40000, 2048), (12, 9000, 33000), (32, 20000, 4096), (12, 90000, 520)])
def test_expired_waits(M, n, k):
    """Waits bounded by a few nanoseconds: the call ends, flag 8 says so, whole outputs are NaN or as ever.  (Up to
    8 tokens the copies may land while the activations are converted, and no wait runs out.)"""
    w4, x = bg.op_w4_quantize(weights(n, k), 64), acts(M, k)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    want = bg.op_linear_w4(x, w4, flag=flag)
    assert flag.item() == 0
    lost = 0
    try:
        assert bg.lib().bloom_op_linear_w4_wait_ns(20) == 0
        for _ in range(10):
            flush.zero_()
            flag.zero_()
            got = bg.op_linear_w4(x, w4, flag=flag)
            torch.cuda.synchronize()
            nan = torch.isnan(got)
            assert flag.item() == (8 if nan.any() else 0)
            assert torch.equal(torch.where(nan, want, got), want)
            lost += int(nan.any())
    finally:
        assert bg.lib().bloom_op_linear_w4_wait_ns(0) == 0
    assert lost > 0 or M <= 8
    flag.zero_()
    assert torch.equal(bg.op_linear_w4(x, w4, flag=flag), want) and flag.item() == 0


def test_streams_and_graphs():
    """Two streams at once on the same weights, and a captured call replayed with new activations."""
    w4, x, x2 = bg.op_w4_quantize(weights(3000, 8200), 128), acts(4, 8200), acts(4, 8200, 9)
    want, want2 = bg.op_linear_w4(x, w4), bg.op_linear_w4(x2, w4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append((bg.op_linear_w4(x, w4, stream=s1), bg.op_linear_w4(x2, w4, stream=s2)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want2) for a, b in outs)
    buf, y = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.op_linear_w4(buf, w4, y=y)
    for src, res in ((x, want), (x2, want2), (x, want)):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, res)


@pytest.mark.parametrize("M", [9, 40])
def test_workspace(M):
    """A workspace of the caller's: any content, no byte behind it touched, reused by the next call; a smaller or
    misaligned one is refused."""
    w4, x = bg.op_w4_quantize(weights(500, 2056), 64), acts(M, 2056)
    want = bg.op_linear_w4(x, w4)
    need = bg.lib().bloom_op_linear_w4_workspace(w4.ref, M)
    room = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert torch.equal(bg.op_linear_w4(x, w4, workspace=room[:need]), want)
    assert (room[need:] == 255).all()
    few = bg.op_linear_w4(x[:9], w4, workspace=room)
    assert torch.equal(few, want[:9]) if M == 9 else few.shape == (9, 500)
    for bad in (room[: need - 1], room[8: need + 8], room[:0]):
        with pytest.raises(bg.BloomError):
            bg.op_linear_w4(x, w4, workspace=bad)


def chained(step, turns=20):
    """The results of step(0), step(1), ... launched back to back from one graph."""
    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(i) for i in range(turns)]
    graph.replay()
    torch.cuda.synchronize()
    return got


SOON = [(256, 512), (1024, 1024), (4096, 1024), (16384, 4096)]     # from one wave of CTAs to many


@pytest.mark.parametrize("n,k", SOON)
@pytest.mark.parametrize("M", [1, 8, 300])
def test_read_back_then_other_layers(M, n, k):
    """The matrix read back is another layer's weights at once, though that layer loads weights ahead."""
    x = acts(M, k)
    w4s = [bg.op_w4_quantize(weights(n, k, s), 64) for s in (0, 1)]
    out = torch.zeros(n, k, dtype=torch.bfloat16, device=DEV)
    layer = {1: bg.op_linear, 8: bg.op_linear_tc, 300: bg.op_gemm}[M]
    want = [layer(x, bg.op_w4_read(w)) for w in w4s]

    def step(i):
        bg.op_w4_read(w4s[i & 1], out)
        return layer(x, out)

    for i, y in enumerate(chained(step)):
        assert torch.equal(y, want[i & 1])


@pytest.mark.parametrize("n,k", SOON)
@pytest.mark.parametrize("M", [1, 12])
def test_quantized_anew_before_each_layer(M, n, k):
    """Tiles that are written just before the layer that reads them, on both of its forms."""
    ws, x = [weights(n, k, s) for s in (0, 1)], acts(M, k)
    want = [bg.op_linear_w4(x, bg.op_w4_quantize(w, 64)) for w in ws]
    q = bg.op_w4_quantize(ws[0], 64)

    def step(i):
        bg.op_w4_quantize(ws[i & 1], 64, out=q)
        return bg.op_linear_w4(x, q)

    for i, y in enumerate(chained(step)):
        assert torch.equal(y, want[i & 1])


@pytest.mark.parametrize("B", [3, 12])
def test_a_step_of_a_small_model(B):
    """Layers and the LM head over 4-bit weights, filtered sampling of the head's logits and the drawn tokens' log
    probabilities, captured in one graph and replayed over new activations and uniform numbers."""
    h, V, J = 512, 9001, 4
    up, down, head = (bg.op_w4_quantize(weights(n, k, s), g) for n, k, s, g in ((4 * h, h, 0, 32), (h, 4 * h, 1, 64), (V, h, 2, 128)))
    wide = [plain.values(weights(n, k, s), g) for n, k, s, g in ((4 * h, h, 0, 32), (h, 4 * h, 1, 64), (V, h, 2, 128))]
    bias = torch.randn(4 * h, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(torch.bfloat16)
    t, p = torch.full((B,), 0.7, device=DEV), torch.full((B,), 0.9, device=DEV)
    k, mp = torch.full((B,), 50, dtype=torch.int32, device=DEV), torch.full((B,), 0.01, device=DEV)
    x, u = acts(B, h), torch.rand(B, J, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)

    def step():
        a = bg.op_linear_w4(x, up, bias, bg.EPI_GELU)
        y = bg.op_linear_w4(a, down, None, bg.EPI_RESID, y=x.clone())
        z = bg.op_linear_w4(y, head, dtype=torch.float32)
        tok = bg.op_sample_filtered(z, u, t, k, p, mp)
        return a, y, z, tok, bg.op_logprobs(z, tok)[0]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(acts(B, h, seed))
        u.copy_(torch.rand(B, J, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        a, y, z, tok, logp = out
        assert all(torch.equal(g, e) for g, e in zip(out, step()))
        check(a, *plain.linear(x, wide[0], bias, 1, group=32))
        check(y, *plain.linear(a, wide[1], None, 2, x, group=64))
        check(z, *plain.linear(y, wide[2], group=128))
        zc = z.cpu().numpy()
        f = [float(s[0]) for s in (t, p, mp)]
        for b in range(B):
            for j in range(J):
                assert sample_plain.agrees(int(tok[b, j]), zc[b], f[0], 50, f[1], f[2], float(u[b, j]))
        want = torch.log_softmax(z.double(), 1).gather(1, tok.long())
        assert ((logp.double() - want).abs() <= 2.0 ** -24 * (V / 512 + 64) + 2.0 ** -22 * want.abs()).all()


def test_more_blocks_of_tokens_than_fit_at_once():
    """70000 tokens: more blocks of 64 than CTAs are resident, each going through all rows."""
    M, n, k = 70000, 300, 264
    w, x = weights(n, k), acts(M, k)
    w4 = bg.op_w4_quantize(w, 64)
    y = bg.op_linear_w4(x, w4, dtype=torch.float32)
    check(y, *plain.linear(x, plain.values(w, 64), group=64))
    assert torch.equal(bg.op_linear_w4(x[-64:], w4, dtype=torch.float32), y[-64:])


def test_streams_and_graphs_of_many_tokens():
    """Two streams at once on the same weights, two graphs with a workspace each, replayed side by side."""
    w4, xs = bg.op_w4_quantize(weights(9000, 2056), 64), [acts(24, 2056, s) for s in (0, 9)]
    want = [bg.op_linear_w4(x, w4) for x in xs]
    need = bg.lib().bloom_op_linear_w4_workspace(w4.ref, 24)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[bg.op_linear_w4(x, w4, stream=s) for x, s in zip(xs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in outs for a, b in zip(pair, want))
    graphs, bufs, ys = [], [x.clone() for x in xs], [torch.empty_like(w) for w in want]
    rooms = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in xs]
    for buf, y, room in zip(bufs, ys, rooms):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            bg.op_linear_w4(buf, w4, y=y, workspace=room)
    for turn in range(10):
        for i in (0, 1):
            bufs[i].copy_(xs[(i + turn) & 1])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ys[i], want[(i + turn) & 1]) for i in (0, 1))
