"""Cases of the operators on an 8-bit key / value cache and on the logits of a step.

Four operators, each called as a serving program calls it:

  write     new keys and values of every row quantised into the 8-bit cache
  read      slots of the cache widened back to bf16
  attn      ALiBi attention of one or a few new tokens a row over the cache
  logprobs  log probabilities of given tokens, entropy and top alternatives

The cache of one layer is k / v codes [B][n][S][d] (int8 or float8_e4m3fn) and
float32 scales [B][n][ceil(S / 32)], one for every 32 slots of a head, powers of
two: value = code * scale.  A block's scale is the smallest power of two (2^-126
at least) with amax <= 127 * scale (int8) or 448 * scale (e4m3); it only grows
while the block fills, and tokens that the block held before are rounded again
(half to even) when it does.
"""
import math

import torch

own = False
_bg = None

BLOCK = 32
LARGEST = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one token of each of 32 sequences appended in a decode step; K and V are views of the fused QKV output
        dict(name="write_step", op="write", codes="int8", B=32, T=1, n=32, d=128, S=544, first=37, last=500, pads=0, layout="qkv"),
        # a ragged chunk of left-padded prompts that continues filled blocks, copied from a bf16 cache's [B][n][T][d]
        dict(name="write_chunk", op="write", codes="e4m3", B=3, T=517, n=16, d=64, S=1312, first=5, last=700, pads=40, layout="heads"),
        # whole prompts of eight sequences
        dict(name="write_prompt", op="write", codes="int8", B=8, T=2048, n=32, d=128, S=2112, first=0, last=0, pads=0, layout="qkv"),
        # a short sequence read back, as when a row leaves the 8-bit cache
        dict(name="read_row", op="read", codes="int8", B=1, T=100, n=16, d=64, S=160, first=3, last=3),
        # long rows read back to bf16 for the attention of the prompt's next chunk
        dict(name="read_long", op="read", codes="e4m3", B=4, T=8191, n=32, d=128, S=8224, first=0, last=0),
        # the first tokens of one sequence of a small model: latency
        dict(name="attn_first", op="attn", codes="int8", B=1, T=1, n=16, kv=16, d=64, S=160, shortest=41, longest=41, pads=0),
        # a decode step of 32 sequences of different lengths
        dict(name="attn_serve", op="attn", codes="int8", B=32, T=1, n=32, kv=32, d=128, S=2048, shortest=130, longest=2011, pads=9),
        # four drafted tokens a sequence checked at once, four query heads to each key head
        dict(name="attn_verify", op="attn", codes="e4m3", B=16, T=4, n=32, kv=8, d=128, S=4096, shortest=1025, longest=4090, pads=0),
        # few sequences with long caches
        dict(name="attn_long", op="attn", codes="e4m3", B=4, T=1, n=32, kv=32, d=128, S=32800, shortest=29999, longest=32777, pads=0),
        # the sampled token of one sequence and five alternatives
        dict(name="logprobs_one", op="logprobs", B=1, V=250880, J=1, top=5, std=3.0),
        # 32 sequences, four candidates each, twenty alternatives
        dict(name="logprobs_batch", op="logprobs", B=32, V=250880, J=4, top=20, std=3.0),
        # the tokens of prompts scored
        dict(name="logprobs_prompt", op="logprobs", B=509, V=250880, J=1, top=1, std=2.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "logprobs"])
    codes = rng.choice(["int8", "e4m3"])
    d = rng.choice([64, 128])
    if op == "logprobs":
        V = _log(rng, 700, 250880)
        return dict(op=op, B=_log(rng, 1, min(512, 120_000_000 // V)), V=V, J=rng.choice([1, 1, 2, 5]), top=rng.choice([0, 1, 5, 20, 32]), std=rng.choice([1.0, 2.0, 4.0]))
    n = rng.choice([16, 32, 112] if d == 128 else [12, 16, 25])
    if op == "attn":
        T = rng.choice([1, 1, 1, 2, 5])
        kv = n if rng.random() < 0.6 else n // rng.choice([g for g in (2, 4, 5, 8) if n % g == 0] or [1])
        longest = _log(rng, 9, 30000)
        B = _log(rng, 1, max(1, min(64, 120_000_000 // (longest * n * d))))
        S = (longest + rng.randrange(0, 70) + 31) // 32 * 32
        return dict(op=op, codes=codes, B=B, T=T, n=n, kv=kv, d=d, S=S, shortest=max(T, _log(rng, max(1, longest // 16), longest)), longest=max(T, longest), pads=rng.choice([0, 0, 3]))
    T = _log(rng, 1, 4000)
    B = _log(rng, 1, max(1, min(64, 50_000_000 // (T * n * d))))
    first, last = sorted((rng.randrange(0, 300), rng.randrange(0, 300)))
    S = (last + T + 63) // 32 * 32 + 32
    if op == "read":
        return dict(op=op, codes=codes, B=B, T=T, n=n, d=d, S=S, first=first, last=last)
    return dict(op=op, codes=codes, B=B, T=T, n=n, d=d, S=S, first=first, last=last, pads=rng.choice([0, 0, min(T - 1, 11)]), layout=rng.choice(["qkv", "heads"]))


def _spread(B, lo, hi):
    """B whole numbers from lo to hi, spread evenly and out of order; the last row gets hi."""
    return [lo + int((hi - lo) * ((b + 1) * 0.6180339887 % 1.0)) for b in range(B - 1)] + [hi]


def _values(shape, g, std):
    """Keys or values: normal, with every 16th channel four times as wide."""
    x = torch.randn(shape, generator=g, device="cuda") * std
    x[..., ::16] *= 4.0
    return x.to(torch.bfloat16)


def _scale_of(amax, codes):
    """The smallest power of two (2^-126 at least) whose LARGEST multiple covers amax; 0 for 0."""
    m, e = torch.frexp(amax)
    top_m, top_e = math.frexp(LARGEST[codes])
    e = (e - top_e + (m > top_m).int()).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _code(x, scale, codes):
    """x / scale (exact: the scale is a power of two, or 0 where every x is) rounded to the codes' type, as float32."""
    y = x / torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(y) if codes == "int8" else y.to(torch.float8_e4m3fn).float()


def _filled(B, n, S, d, codes, g, std):
    """A cache whose blocks were each written at once: codes and scales of random values."""
    x = _values((B, n, S // BLOCK, BLOCK, d), g, std).float()
    s = _scale_of(x.abs().amax((3, 4)), codes)
    return _code(x, s[..., None, None], codes).to(DTYPE[codes]).view(B, n, S, d), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    if c["op"] == "logprobs":
        z = torch.randn(c["B"], c["V"], generator=g, device="cuda") * c["std"]
        z[:, 3::97] = -torch.inf  # tokens that a serving program rules out
        tokens = torch.randint(0, c["V"] // 97, (c["B"], c["J"]), generator=g, device="cuda", dtype=torch.int32) * 97
        return dict(case=c, logits=z, tokens=tokens)
    B, n, d, S, T = c["B"], c["kv"] if c["op"] == "attn" else c["n"], c["d"], c["S"], c["T"]
    st = dict(case=c)
    # tokens that the cache holds already are narrower than the new ones, so that scales of half-filled blocks grow
    std = 0.4 if c["op"] == "write" else 1.0
    st["k"], st["ks"] = _filled(B, n, S, d, c["codes"], g, std)
    st["v"], st["vs"] = _filled(B, n, S, d, c["codes"], g, std)
    if c["op"] == "attn":
        lens = torch.tensor(_spread(B, c["shortest"], c["longest"]), dtype=torch.int32)
        slot = torch.arange(S)[None]
        pos = torch.where((slot >= c["pads"]) | (lens[:, None] <= c["pads"] + T), slot - c["pads"], torch.tensor(-1))
        pos = torch.where(lens[:, None] <= c["pads"] + T, slot, pos)  # rows too short for pads have none
        st["pos"] = pos.to(torch.int32).cuda()
        st["lens"] = lens.cuda()
        st["q"] = torch.randn((B, T, c["n"], d), generator=g, device="cuda").to(torch.bfloat16)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["n"]) for h in range(c["n"])], device="cuda")
        return st
    start = torch.tensor(_spread(B, c["first"], c["last"]), dtype=torch.int32)
    st["start"] = start.cuda()
    if c["op"] == "write":
        if c["layout"] == "qkv":
            qkv = _values((B, T, n, 3, d), g, 1.0)
            st["new_k"], st["new_v"] = qkv[:, :, :, 1], qkv[:, :, :, 2]
        else:
            st["new_k"], st["new_v"] = (_values((B, n, T, d), g, 1.0).transpose(1, 2) for _ in range(2))
        st["mask"] = None
        if c["pads"]:
            width = torch.tensor(_spread(B, 0, c["pads"]))
            st["mask"] = (torch.arange(T)[None] >= width[:, None]).to(torch.uint8).cuda()
        # the blocks that the new tokens touch, from their first slot
        st["from"] = (start // BLOCK * BLOCK).to(torch.int32).cuda()
        st["slots"] = T + int((start % BLOCK).max())
        st["count"] = (start % BLOCK + T).to(torch.int32).cuda()
    return st


def _read(codes, scale, start, T, count=None):
    """Slots start .. start + T of every row as bf16 [B][T][n][d]; zeros from `count` on."""
    B = codes.shape[0]
    t = torch.arange(T, device=codes.device)
    slot = (start[:, None] + t).long()
    row = torch.arange(B, device=codes.device)[:, None]
    slot = slot.clamp(max=codes.shape[2] - 1)
    x = codes.transpose(1, 2)[row, slot].float() * scale.transpose(1, 2)[row, slot // BLOCK][..., None]
    if count is not None:
        x = x * (t < count[:, None])[:, :, None, None]
    return x.to(torch.bfloat16)


def _write(cache, scale, x, start, mask, codes):
    """x [B][T][n][d] into slots start .. start + T of the cache, in place."""
    B, T, n, d = x.shape
    blocks = (T + 2 * BLOCK - 2) // BLOCK
    row = torch.arange(B, device=x.device)[:, None]
    first = (start // BLOCK).long()[:, None]
    at = first * BLOCK + torch.arange(blocks * BLOCK, device=x.device)  # slots of the blocks touched
    t = at - start[:, None].long()
    new = (t >= 0) & (t < T)
    held = (t < 0)[:, :, None, None]
    y = x[row, t.clamp(0, T - 1)].float()
    put = new if mask is None else new & (mask[row, t.clamp(0, T - 1)] != 0)
    y = torch.where(put[:, :, None, None], y, torch.zeros((), device=x.device))
    old = cache.transpose(1, 2)[row, at].float()
    at_block = first + torch.arange(blocks, device=x.device)
    before = scale.transpose(1, 2)[row, at_block]  # [B][blocks][n]
    holds = (t < 0).view(B, blocks, BLOCK).any(2)[:, :, None]
    touched = new.view(B, blocks, BLOCK).any(2)[:, :, None]
    after = _scale_of(y.abs().view(B, blocks, BLOCK, n, d).amax((2, 4)), codes)
    after = torch.where(holds, torch.maximum(after, before), after)
    after = torch.where(touched, after, before)
    wide = lambda s: s.repeat_interleave(BLOCK, 1)[..., None]
    again = _code(old * wide(before), wide(after), codes)
    code = torch.where(new[:, :, None, None], _code(y, wide(after), codes), torch.where(held & wide(touched.expand_as(after)), again, old))
    cache.transpose(1, 2)[row, at] = code.to(DTYPE[codes])
    scale.transpose(1, 2)[row, at_block] = after


def _attend(q, k, ks, v, vs, pos, slopes, lens):
    B, T, n, d = q.shape
    kv, S = k.shape[1], k.shape[2]
    g = n // kv
    kf = (k.float().view(B, kv, S // BLOCK, BLOCK, d) * ks[..., None, None]).view(B, kv, S, d)
    qf = q.float().view(B, T, kv, g, d).permute(0, 2, 3, 1, 4).reshape(B, kv, g * T, d)
    s = (torch.matmul(qf, kf.transpose(2, 3)) * d ** -0.5).view(B, kv, g, T, S)
    far = (pos - pos.amax(1, keepdim=True)).double()
    s = s + (slopes.double().view(kv, g, 1, 1) * far[:, None, None, None]).float()
    upto = lens[:, None] - T + torch.arange(T, device=q.device)
    see = (pos >= 0)[:, None] & (torch.arange(S, device=q.device) <= upto[:, :, None])
    s = s.masked_fill(~see[:, None, None], -torch.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    vf = (v.float().view(B, kv, S // BLOCK, BLOCK, d) * vs[..., None, None]).view(B, kv, S, d)
    o = torch.matmul(p.view(B, kv, g * T, S), vf).view(B, kv, g, T, d)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, n * d).to(torch.bfloat16)


def _logprobs(z, tokens, top):
    m = z.amax(1, keepdim=True)
    x = z - m
    e = torch.exp(x)
    s = e.sum(1, keepdim=True)
    logp = x.gather(1, tokens.long()) - torch.log(s)
    entropy = torch.log(s)[:, 0] - torch.where(e > 0, e * x, torch.zeros((), device=z.device)).sum(1) / s[:, 0]
    # the highest logits, equal ones by index: one whole number that orders by both
    bits = z.view(torch.int32).long()
    key = (torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) << 32) + (2 ** 31 - 1 - torch.arange(z.shape[1], device=z.device))
    ids = torch.topk(key, top, 1).indices
    return logp, entropy, ids.to(torch.int32), x.gather(1, ids) - torch.log(s)


def run(state):
    global _bg
    s, c = state, state["case"]
    if own:
        if _bg is None:
            import bloom_decoder_token_gb300 as _bg
        if c["op"] == "logprobs":
            return _bg.op_logprobs(s["logits"], s["tokens"], c["top"])
        cache = _bg.KV8(s["k"], s["v"], s["ks"], s["vs"])
        if c["op"] == "attn":
            return _bg.op_attn_decode_kv8(s["q"], cache, s["pos"], s["slopes"], s["lens"])
        if c["op"] == "read":
            return _bg.op_kv8_read(cache, s["start"], c["T"])
        _bg.op_kv8_write(cache, s["new_k"], s["new_v"], s["start"], mask=s["mask"])
        k, v = _bg.op_kv8_read(cache, s["from"], s["slots"], count=s["count"])
        return k, v, s["ks"], s["vs"]
    if c["op"] == "logprobs":
        return _logprobs(s["logits"], s["tokens"], c["top"])
    if c["op"] == "attn":
        return _attend(s["q"], s["k"], s["ks"], s["v"], s["vs"], s["pos"], s["slopes"], s["lens"])
    if c["op"] == "read":
        return _read(s["k"], s["ks"], s["start"], c["T"]), _read(s["v"], s["vs"], s["start"], c["T"])
    _write(s["k"], s["ks"], s["new_k"], s["start"], s["mask"], c["codes"])
    _write(s["v"], s["vs"], s["new_v"], s["start"], s["mask"], c["codes"])
    # the cache is held in 8 bits: the values it stands for, read back from the blocks written
    return _read(s["k"], s["ks"], s["from"], s["slots"], s["count"]), _read(s["v"], s["vs"], s["from"], s["slots"], s["count"]), s["ks"], s["vs"]


def work(case):
    c = case
    if c["op"] == "logprobs":
        # the logits once; two exponential-weighted sums
        return {"bytes": 4 * c["B"] * (c["V"] + 2 * c["J"] + 1 + 2 * c["top"]), "flops": 5 * c["B"] * c["V"]}
    if c["op"] == "attn":
        lens = _spread(c["B"], c["shortest"], c["longest"])
        keys, blocks = sum(lens), sum(-(-x // BLOCK) for x in lens)
        data = 2 * c["kv"] * (keys * c["d"] + 4 * blocks) + 4 * keys + 4 * c["B"] * c["T"] * c["n"] * c["d"]
        return {"bytes": data, "flops": 4 * c["T"] * c["n"] * c["d"] * keys}
    a = c["B"] * c["n"]
    if c["op"] == "read":
        return {"bytes": 2 * a * (3 * c["T"] * c["d"] + 4 * (-(-c["T"] // BLOCK))), "flops": 2 * a * c["T"] * c["d"]}
    # new values in, codes and scales out; then the touched blocks' codes in and their values out
    start = _spread(c["B"], c["first"], c["last"])
    back = sum(s % BLOCK + c["T"] for s in start) * c["n"]
    return {"bytes": 2 * (3 * a * c["T"] * c["d"] + 3 * back * c["d"] + 8 * a * (-(-c["T"] // BLOCK))), "flops": 2 * (3 * a * c["T"] + back) * c["d"]}


def _round_e4m3(y):
    """float64 to the nearest value with 3 fraction bits and exponents from -6, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "logprobs":
        z = s["logits"].double()
        p = torch.log_softmax(z, 1)
        entropy = -torch.special.xlogy(p.exp(), p.exp()).sum(1)
        v, i = torch.sort(z, dim=1, descending=True, stable=True)
        ids = i[:, : c["top"]]
        return p.gather(1, s["tokens"].long()), entropy, ids.to(torch.int32), p.gather(1, ids)
    wide = lambda x, sc: x.double() * sc.double().repeat_interleave(BLOCK, 2)[..., None]
    if c["op"] == "read":
        out = []
        for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = wide(x, sc)
            out.append(torch.stack([x[b, :, a: a + c["T"]].transpose(0, 1) for b, a in enumerate(s["start"].tolist())]))
        return tuple(out)
    if c["op"] == "attn":
        rows = []
        g = c["n"] // c["kv"]
        for b, ln in enumerate(s["lens"].tolist()):
            k, v = (wide(x[b:b + 1, :, :], sc[b:b + 1])[0, :, :ln].repeat_interleave(g, 0) for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            pos = s["pos"][b, :ln].double()
            bias = s["slopes"].double()[:, None] * pos
            for t in range(c["T"]):
                w = (k @ s["q"][b, t].double()[:, :, None])[..., 0] / c["d"] ** 0.5 + bias
                w[:, (pos < 0) | (torch.arange(ln, device=pos.device) > ln - c["T"] + t)] = -torch.inf
                rows.append((torch.softmax(w, 1)[:, None] @ v).reshape(-1))
        return torch.stack(rows).view(c["B"], c["T"], -1)
    big = LARGEST[c["codes"]]
    out, scales = [], []
    for x, sc, new in ((s["k"], s["ks"], s["new_k"]), (s["v"], s["vs"], s["new_v"])):
        got = torch.zeros(c["B"], s["slots"], c["n"], c["d"], dtype=torch.float64, device="cuda")
        x, sc, sc2 = x.double(), sc.double(), sc.double()
        for b, a in enumerate(s["start"].tolist()):
            y = new[b].double()
            if s["mask"] is not None:
                y = y * s["mask"][b].double()[:, None, None]
            for j in range(a // BLOCK, (a + c["T"] - 1) // BLOCK + 1):
                lo, hi = max(a, j * BLOCK), min(a + c["T"], (j + 1) * BLOCK)
                fresh = y[lo - a: hi - a].transpose(0, 1)  # [n][tokens][d]
                amax = fresh.abs().amax((1, 2))
                grown = torch.exp2(torch.ceil(torch.log2(amax / big)))
                grown = torch.where(amax <= grown / 2 * big, grown / 2, grown)  # the quotient may have come out above its power
                if a > j * BLOCK:
                    grown = torch.maximum(grown, sc[b, :, j])
                    fresh = torch.cat((x[b, :, j * BLOCK: a] * sc[b, :, j, None, None], fresh), 1)
                unit = torch.where(grown > 0, grown, torch.ones_like(grown))[:, None, None]
                code = torch.round(fresh / unit) if c["codes"] == "int8" else _round_e4m3(fresh / unit)
                at = j * BLOCK - a // BLOCK * BLOCK
                got[b, at: at + fresh.shape[1]] = (code * unit).transpose(0, 1)
                sc2[b, :, j] = grown
        out.append(got)
        scales.append(sc2)
    return out[0], out[1], scales[0], scales[1]
