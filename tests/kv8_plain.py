"""Plain float64 forms of the operators on the 8-bit KV cache and of the token log
probabilities, written from their definitions (numpy, loops over rows and blocks)."""
import numpy as np
import torch

BLOCK = 32
LARGEST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def code_values(t):
    """Codes as float64 (a cache's k or v)."""
    t = t.detach().cpu()
    return t.float().double().numpy() if t.dtype is torch.float8_e4m3fn else t.double().numpy()


def round_codes(y, codes):
    """float64 to the codes' type, ties to even."""
    if codes is torch.int8:
        return np.round(y)
    mag = np.maximum(np.abs(y), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(mag)) - 3)   # 3 fraction bits, exponents from -6
    return np.round(y / step) * step


def scale_of(amax, codes):
    if amax == 0:
        return 0.0
    if not np.isfinite(amax):
        return np.nan
    e = -126
    while amax > LARGEST[codes] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def write(code, scale, codes, x, start, count=None, mask=None):
    """x [B][T][n][d] into code [B][n][S][d] and scale [B][n][blocks], in place."""
    B, T, n, d = x.shape
    S = code.shape[2]
    for b in range(B):
        if start[b] < 0:
            continue
        end = min(int(start[b]) + (T if count is None else min(max(int(count[b]), 0), T)), S)
        for blk in range(start[b] // BLOCK, -(-end // BLOCK)):
            base = blk * BLOCK
            lo, hi = max(base, start[b]), min(end, base + BLOCK)
            if lo >= hi:
                continue
            t = np.arange(lo, hi) - start[b]
            new = np.where(mask[b, t][:, None, None] != 0, x[b, t], 0.0) if mask is not None else x[b, t]
            for h in range(n):
                s = scale_of(np.abs(new[:, h]).max(), codes)
                if lo > base:
                    old = scale[b, h, blk]
                    if np.isnan(old) or np.isnan(s):
                        s = np.nan
                    elif s > old:
                        if old > 0:
                            code[b, h, base:lo] = round_codes(code[b, h, base:lo] * old / s, codes)
                    else:
                        s = old
                scale[b, h, blk] = s
                code[b, h, lo:hi] = round_codes(new[:, h] / s, codes) if s > 0 else 0.0


def wide(code, scale):
    """values [B][n][S][d]"""
    s = np.repeat(scale, BLOCK, axis=2)[:, :, :code.shape[2]]
    return code * s[..., None]


def read(code, scale, start, T, count=None):
    v = wide(code, scale)
    B, n, S, d = v.shape
    out = np.zeros((B, T, n, d))
    for b in range(B):
        if start[b] < 0:
            continue
        c = T if count is None else min(max(count[b], 0), T)
        c = min(c, S - start[b])
        if c > 0:
            out[b, :c] = v[b, :, start[b]:start[b] + c].transpose(1, 0, 2)
    return out


def attend(q, k, v, pos, slopes, lens):
    """q [B][T][n][d], k and v [B][kv][S][d] -> (o, bound) [B][T][n][d]: the outputs and
    what a kernel may be off by: float32 scores (d products summed in any order, 2^-23
    of the magnitudes each), probabilities rounded to f16 (2^-11), a bf16 result (2^-8)."""
    B, T, n, d = q.shape
    kv, S = k.shape[1:3]
    o, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        ln = min(int(lens[b]), S)
        for t in range(T):
            upto = ln - T + t + 1 if ln > 0 else 0
            see = np.nonzero(pos[b, :max(upto, 0)] >= 0)[0]
            if not len(see):
                continue
            p0 = pos[b, see].astype(np.float64)
            far = p0 - p0.max()
            for j in range(n):
                kk, vv = k[b, j // (n // kv), see], v[b, j // (n // kv), see]
                s = kk @ q[b, t, j] / np.sqrt(d) + slopes[j] * far
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, t, j] = p @ vv
                size = np.abs(kk) @ np.abs(q[b, t, j]) / np.sqrt(d) + np.abs(slopes[j] * far)
                es = (d + 16) * 2.0 ** -23 * np.max(np.where(p > 1e-9, size, 0.0))
                tol[b, t, j] = 2.0 ** -8 * np.abs(o[b, t, j]) + (2.0 ** -11 + 2 * es) * (p @ np.abs(vv))
    return o, tol


def logprobs(z, tokens, top):
    """Rows of float64 logits: (logp [B][J], entropy [B], ids [B][top], logp [B][top])."""
    B, V = z.shape
    J = tokens.shape[1]
    logp, ent = np.zeros((B, J)), np.zeros(B)
    ids, lps = np.full((B, top), -1), np.full((B, top), -np.inf)
    for b in range(B):
        y = np.where(np.isnan(z[b]), -np.inf, z[b])
        m = y.max()
        if m == -np.inf:
            lp = np.full(V, -np.inf)
        else:
            with np.errstate(invalid="ignore"):
                dd = np.where(y == m, 0.0, y - m)
            lp = dd - np.log(np.exp(dd).sum())
            p = np.exp(lp)
            ent[b] = -np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0))
        for j in range(J):
            t = tokens[b, j]
            logp[b, j] = 0.0 if t == -1 else np.nan if t < -1 or t >= V else lp[t]
        order = np.argsort(-y, kind="stable")[:top]
        order = order[y[order] > -np.inf]
        ids[b, :len(order)], lps[b, :len(order)] = order, lp[order]
    return logp, ent, ids, lps
