"""Plain float64 form of sampling with temperature, top-k, top-p and min-p."""
import numpy as np

# How far a mass may be off, relative to the whole: an exponential within 2^-22 of its value, its exponent by the
# rounding of a difference (2^-24 of at most 18 binades, where the mass lies in 2^18 tokens), the fixed point's last place of
# a token (2^-40 of the largest) for 2^18 tokens at most: 2^-22 + 0.7 * 18 * 2^-24 + 2^-22.
NEAR = 2.0 ** -19


def kept_of(z, t, k, p, mp):
    """(kept tokens in vocabulary order, their probabilities) of a row of float32 logits; None where nothing takes part."""
    z = np.asarray(z, dtype=np.float64)
    part = np.flatnonzero(z > -np.inf)
    if len(part) == 0:
        return None
    top = z[part].max()
    best = part[z[part] == top][0]
    if not t > 0 or p <= 0 or k == 1:
        return np.array([best]), np.ones(1)
    if top == np.inf:
        part = part[z[part] == np.inf]
        d = np.zeros(len(part))
    else:
        d = (top - z[part]) / np.float64(t)
    near = d * np.log2(np.e) < 40
    part, d = part[near], d[near]
    mass = np.exp(-d)
    order = np.lexsort((part, -z[part]))
    n = len(order)
    if k > 0:
        n = min(n, k)
    if p < 1:
        cum = np.cumsum(mass[order[:n]])
        n = min(n, int(np.searchsorted(cum, p * cum[-1], side="left")) + 1)
    if mp > 0:
        n = min(n, max(1, int((mass[order[:n]] >= min(mp, 1.0)).sum())))
        if mp >= 1:
            n = min(n, int((z[part][order] == top).sum()))
    keep = np.sort(order[:n])
    return part[keep], mass[keep] / mass[keep].sum()


def draw(kept, u):
    tokens, prob = kept
    u = 0.0 if not u > 0 else u
    i = int(np.searchsorted(np.cumsum(prob), u, side="right"))
    return int(tokens[min(i, len(tokens) - 1)])


def agrees(got, z, t, k, p, mp, u):
    """Whether a token is the definition's, or one beside a border that lies within NEAR of the draw."""
    kept = kept_of(z, t, k, p, mp)
    if kept is None:
        return got == -1
    if got == draw(kept, u):
        return True
    for near in (kept, kept_of(z, t, k, p * (1 + NEAR), mp), kept_of(z, t, k, p * (1 - NEAR), mp)):
        if got in (draw(near, u + NEAR), draw(near, max(u - NEAR, 0.0))):
            return True
    return False
