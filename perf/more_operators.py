"""Cases of the 4-bit weight operators and of sampling with all filters.

Three operators, each called as a serving program calls it:

  quantize  bf16 weights into 4 bits with group scales (and read back as bf16)
  linear    the linear layer of a decode step over such weights
  sample    tokens drawn with temperature, top-k, top-p and min-p from given
            uniform numbers

A group is 32, 64 or 128 neighbouring weights of a row: value = code * scale,
codes -7 .. 7, the scale bf16(amax / 7), codes w / scale rounded half to even.

Sampling of a row of logits z at temperature t: p = softmax(z / t).  Ordered by
probability, highest first, equal logits by index, the kept tokens are a
prefix: the first top_k, of those the shortest prefix that holds top_p of their
mass, and of those the ones with p >= min_p * max p.  The token is where the
kept mass, summed in vocabulary order, first exceeds u times the whole of it.
"""
import torch

own = False
_bg = None


def listed():
    return [
        # a projection of a small model, converted when its weights are loaded
        dict(name="quantize_small", op="quantize", N=1024, K=1024, group=32),
        # an MLP matrix of a middling model
        dict(name="quantize_up", op="quantize", N=16384, K=4096, group=128),
        # the widest matrix of a large model
        dict(name="quantize_wide", op="quantize", N=57344, K=14336, group=64),
        # one token through an MLP's first matrix of a small model: latency
        dict(name="linear_first", op="linear", M=1, N=4096, K=1024, group=32, epilogue="gelu", bias=True, f32=False),
        # one sequence through an MLP's second matrix: long rows, few of them
        dict(name="linear_down", op="linear", M=1, N=4096, K=16384, group=128, epilogue="store", bias=True, f32=False),
        # a few sequences through the fused QKV projection
        dict(name="linear_qkv", op="linear", M=5, N=12288, K=4096, group=64, epilogue="store", bias=True, f32=False),
        # a decode batch through an MLP's first matrix
        dict(name="linear_serve", op="linear", M=32, N=16384, K=4096, group=128, epilogue="gelu", bias=True, f32=False),
        # the logits of eight sequences from a 4-bit head
        dict(name="linear_head", op="linear", M=8, N=250880, K=4096, group=64, epilogue="store", bias=False, f32=True),
        # one short row: latency
        dict(name="sample_short", op="sample", B=1, V=1003, J=1, std=2.0, mode="chat"),
        # one sequence, the usual settings
        dict(name="sample_one", op="sample", B=1, V=250880, J=1, std=3.0, mode="chat"),
        # a batch whose members have settings of their own, four draws each
        dict(name="sample_batch", op="sample", B=32, V=250880, J=4, std=3.0, mode="mixed"),
        # many sequences, a nucleus without top-k
        dict(name="sample_many", op="sample", B=509, V=250880, J=1, std=2.5, mode="nucleus"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear", "sample", "sample"])
    if op == "sample":
        V = _log(rng, 700, 250880)
        return dict(op=op, B=_log(rng, 1, min(512, 120_000_000 // V)), V=V, J=rng.choice([1, 1, 1, 2, 5]),
                    std=rng.choice([1.5, 2.5, 4.0]), mode=rng.choice(["chat", "nucleus", "minp", "mixed", "k"]))
    group = rng.choice([32, 64, 128])
    K = 8 * _log(rng, 32, 2048)
    N = _log(rng, 60, min(60000, 500_000_000 // K))
    if op == "quantize":
        return dict(op=op, N=N, K=K, group=group)
    return dict(op=op, M=_log(rng, 1, 64), N=N, K=K, group=group, epilogue=rng.choice(["store", "store", "gelu"]),
                bias=rng.random() < 0.6, f32=rng.random() < 0.2)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(N, K, g):
    """Normal weights, a few channels and rows wider than the others."""
    w = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, 8192):
        x = torch.randn((min(8192, N - a), K), generator=g, device="cuda") * 0.02
        x[:, 5::61] *= 4.0
        x[3::37] *= 0.25
        w[a: a + 8192] = x.to(torch.bfloat16)
    return w


def _quantize(w, group):
    """(codes as float32 [N][groups][group], scales bf16 [N][groups])"""
    N, K = w.shape
    groups = -(-K // group)
    x = torch.nn.functional.pad(w.float(), (0, groups * group - K)).view(N, groups, group)
    s = (x.abs().amax(2) / 7).to(torch.bfloat16)
    wide = s.float()[..., None]
    code = torch.where(wide > 0, torch.round(x / torch.where(wide > 0, wide, torch.ones_like(wide))).clamp(-7, 7), torch.zeros_like(x))
    return code, s


def _settings(c, g):
    """Temperature, top-k, top-p and min-p of every row, None where a program has no such setting."""
    B = c["B"]
    u = lambda: torch.rand(B, generator=g, device="cuda")
    t, k, p, m = 0.6 + 0.5 * u(), (5 + 75 * u()).to(torch.int32), 0.85 + 0.13 * u(), 0.02 + 0.1 * u()
    if c["mode"] == "chat":
        return t, k, p, None
    if c["mode"] == "nucleus":
        return t, None, p, None
    if c["mode"] == "minp":
        return t + 0.4, None, None, m
    if c["mode"] == "k":
        return t, k * 12, None, None
    which = torch.arange(B, device="cuda") % 4  # mixed: some filters off in each row
    t = torch.where(which == 3, torch.zeros_like(t), t)  # greedy
    k = torch.where(which == 0, k, torch.where(which == 2, k * 10, torch.zeros_like(k)))
    p = torch.where(which == 1, p, torch.where(which == 2, p, torch.ones_like(p)))
    m = torch.where(which == 0, m, torch.zeros_like(m))
    return t, k, p, m


def prepare(case, seed):
    global _bg
    c, g = case, _generator(seed)
    if own and _bg is None:
        import bloom_decoder_token_gb300 as _bg
    st = dict(case=c)
    if c["op"] == "sample":
        z = torch.randn(c["B"], c["V"], generator=g, device="cuda") * c["std"]
        z[:, 3::97] = -torch.inf  # tokens that a serving program rules out
        st["logits"] = z
        st["t"], st["k"], st["p"], st["m"] = _settings(c, g)
        st["u"] = torch.rand((c["B"], c["J"]), generator=g, device="cuda")
        return st
    w = _weights(c["N"], c["K"], g)
    if c["op"] == "quantize":
        st["w"] = w
        return st
    x = torch.randn((c["M"], c["K"]), generator=g, device="cuda")
    x[:, 7::113] *= 8.0
    st["x"] = x.to(torch.bfloat16)
    st["bias"] = (torch.randn(c["N"], generator=g, device="cuda") * 0.5).to(torch.bfloat16) if c["bias"] else None
    if own:
        st["w4"] = _bg.op_w4_quantize(w, c["group"])
        return st
    groups = -(-c["K"] // c["group"])
    st["codes"] = torch.empty((c["N"], groups, c["group"]), dtype=torch.int8, device="cuda")
    st["scales"] = torch.empty((c["N"], groups), dtype=torch.bfloat16, device="cuda")
    for a in range(0, c["N"], 16384):
        code, st["scales"][a: a + 16384] = _quantize(w[a: a + 16384], c["group"])
        st["codes"][a: a + 16384] = code.to(torch.int8)
    return st


def _linear(s, c):
    w = (s["codes"].float() * s["scales"].float()[..., None]).view(c["N"], -1)[:, : c["K"]]
    y = torch.matmul(s["x"].float(), w.t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["epilogue"] == "gelu":
        y = y * 0.5 * (1 + torch.tanh(0.79788456 * y * (1 + 0.044715 * y * y)))
    return y if c["f32"] else y.to(torch.bfloat16)


def _sample(s):
    # in 64 bits: the draws fall between masses that lie close to one another
    z = s["logits"]
    B, V = z.shape
    top = z.amax(1, keepdim=True)
    t = s["t"].double()[:, None]
    greedy = t <= 0
    p = torch.exp((z.double() - top.double()) / torch.where(greedy, torch.ones_like(t), t))
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    ranked = p.gather(1, order)
    rank = torch.arange(V, device=z.device)[None]
    if s["k"] is not None:
        k = s["k"][:, None]
        ranked = torch.where((k > 0) & (rank >= k), torch.zeros_like(ranked), ranked)
    if s["p"] is not None:
        tp = s["p"].double()[:, None]
        before = torch.cumsum(ranked, 1)
        need = tp * before[:, -1:]
        ranked = torch.where((tp < 1) & (before - ranked >= need), torch.zeros_like(ranked), ranked)
    if s["m"] is not None:
        ranked = torch.where(ranked < s["m"].double()[:, None], torch.zeros_like(ranked), ranked)
    ranked = torch.where(greedy & (rank > 0), torch.zeros_like(ranked), ranked)
    kept = torch.cumsum(torch.zeros_like(p).scatter_(1, order, ranked), 1)
    at = torch.searchsorted(kept, s["u"].double() * kept[:, -1:], right=True)
    return at.clamp(max=V - 1).to(torch.int32)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "sample":
        return _bg.op_sample_filtered(s["logits"], s["u"], s["t"], s["k"], s["p"], s["m"]) if own else _sample(s)
    if c["op"] == "quantize":
        if own:
            return _bg.op_w4_read(_bg.op_w4_quantize(s["w"], c["group"]))
        code, scale = _quantize(s["w"], c["group"])
        return (code * scale.float()[..., None]).view(c["N"], -1)[:, : c["K"]].to(torch.bfloat16)
    if own:
        epilogue = _bg.EPI_GELU if c["epilogue"] == "gelu" else _bg.EPI_STORE
        return _bg.op_linear_w4(s["x"], s["w4"], s["bias"], epilogue, dtype=torch.float32 if c["f32"] else torch.bfloat16)
    return _linear(s, c)


def work(case):
    c = case
    if c["op"] == "sample":
        # the logits once, one exponential a logit; settings, draws and tokens
        return {"bytes": 4 * c["B"] * (c["V"] + 4 + 2 * c["J"]), "flops": 4 * c["B"] * c["V"]}
    held = c["N"] * (c["K"] // 2 + 2 * -(-c["K"] // c["group"]))
    if c["op"] == "quantize":
        # weights in, codes and scales out; codes and scales in, weights out
        return {"bytes": 4 * c["N"] * c["K"] + 2 * held, "flops": 4 * c["N"] * c["K"]}
    data = held + 2 * c["M"] * c["K"] + (4 if c["f32"] else 2) * c["M"] * c["N"] + (2 * c["N"] if c["bias"] else 0)
    return {"bytes": data, "flops": 2 * c["M"] * c["N"] * c["K"]}


def _scale_exact(amax):
    """amax / 7 rounded to 8 significant bits, float64 (a tie cannot come up: seven times one has more bits than amax)."""
    bits = (amax / 7).view(torch.int64)
    return ((bits + (1 << 44)) & -(1 << 45)).view(torch.float64)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        out = torch.empty((c["N"], c["K"]), dtype=torch.float64, device="cuda")
        for a in range(0, c["N"], 4096):
            w = s["w"][a: a + 4096].double()
            for j in range(0, c["K"], 8 * c["group"]):
                part = w[:, j: j + 8 * c["group"]]
                for i in range(0, part.shape[1], c["group"]):
                    x = part[:, i: i + c["group"]]
                    sc = _scale_exact(x.abs().amax(1, keepdim=True))
                    out[a: a + 4096, j + i: j + i + c["group"]] = torch.nan_to_num(torch.round(x / sc), nan=0.0) * sc
        return out
    if c["op"] == "linear":
        x = s["x"].double()
        out = torch.empty((c["M"], c["N"]), dtype=torch.float64, device="cuda")
        for a in range(0, c["N"], 8192):
            w = s["codes"][a: a + 8192].double().mul_(s["scales"][a: a + 8192].double().unsqueeze(2)).flatten(1)[:, : c["K"]]
            out[:, a: a + 8192] = x @ w.t()
        if s["bias"] is not None:
            out += s["bias"].double()
        if c["epilogue"] == "gelu":
            out = 0.5 * out * (1 + torch.tanh(0.79788456 * (out + 0.044715 * out ** 3)))
        return out
    tokens = torch.empty((c["B"], c["J"]), dtype=torch.int32)
    value = lambda x, b, off: off if x is None else float(x[b])
    for b in range(c["B"]):
        z = s["logits"][b].double()
        t, k, tp, mp = (value(s[n], b, off) for n, off in (("t", 1.0), ("k", 0), ("p", 1.0), ("m", 0.0)))
        best = int(torch.nonzero(z == z.max())[0])
        if t <= 0:
            tokens[b] = best
            continue
        p = torch.softmax(z / t, 0)
        # by probability, equal logits by index: sorting -z leaves equal ones as they lie
        order = torch.argsort(-z, stable=True)
        n = int((p > 0).sum())
        if 0 < k < n:
            n = int(k)
        q = p[order[:n]]
        if tp < 1:
            share = torch.cumsum(q / q.sum(), 0)
            n = min(n, int((share < tp).sum()) + 1)
        n = min(n, int((p[order[:n]] >= mp * p[best]).sum()))
        keep = torch.sort(order[: max(n, 1)]).values
        mass = torch.cumsum(p[keep], 0)
        for j in range(c["J"]):
            at = int((mass <= float(s["u"][b, j]) * mass[-1]).sum())
            tokens[b, j] = int(keep[min(at, len(keep) - 1)])
    return tokens.cuda()
