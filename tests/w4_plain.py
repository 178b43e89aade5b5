"""Plain float64 forms of the 4-bit weight operators, from their definitions."""
import torch


def bf16_of(v):
    """float64 values rounded to bf16 numbers (half to even, subnormals too), as float64."""
    _, e = torch.frexp(v.double())
    step = (((e.long() - 8).clamp(min=-133) + 1023) << 52).view(torch.float64)   # a power of two, exactly
    r = torch.round(v.double() / step) * step
    return torch.where(r.abs() >= 2.0 ** 128, torch.sign(r) * torch.inf, r)   # past the largest bf16, as IEEE rounds


def quantize(w, group):
    """bf16 [n][k] -> codes [n][groups * group] and scales [n][groups], float64 (a short last group is filled with zeros)."""
    n, k = w.shape
    groups = -(-k // group)
    x = torch.zeros(n, groups * group, dtype=torch.float64, device=w.device)
    x[:, :k] = w.double()
    x = x.view(n, groups, group)
    amax = x.abs().amax(2)
    amax = torch.where(torch.isfinite(x).all(2), amax, torch.nan)
    s = bf16_of(amax / 7)
    unit = torch.where(s > 0, s, 1.0)[..., None]
    code = torch.where(s[..., None] > 0, torch.round(x / unit).clamp(-7, 7), 0.0)
    return code.view(n, -1), s


def values(w, group):
    """What the quantised weights stand for, float64 [n][k]."""
    code, s = quantize(w, group)
    return (code * s.repeat_interleave(group, 1))[:, : w.shape[1]]


def gelu(v):
    return v * 0.5 * (1.0 + torch.tanh(0.79788456 * v * (1.0 + 0.044715 * v * v)))


def linear(x, wide, bias=None, epilogue=0, y=None, group=32):
    """(y, tolerance) of the linear layer over the values `wide`, float64 [M][n].

    The tolerance, before the output's own rounding: a float32 sum of products in chains of
    additions, each off by 2^-23 of the sum of magnitudes at most: up to 8 tokens 64 (8 of a tensor
    core's sums a group, 8 groups a warp, 16 warps, 8 ranks, passes); more: group / 16, 8 ranks, and one
    for every group, those to the nearest (2^-24); activations below 2^-31 of the largest
    of their 256 columns (more than 8 tokens: of all), off by 2^-39 of it; the GeLU's slope is below
    1.13, its own arithmetic off by 2^-20 of its result or 2^-22 of its argument at most."""
    x = x.double()
    M, k = x.shape
    v = x @ wide.t()
    far = x.abs() @ wide.abs().t() * ((64 if M <= 8 else group / 16 + 8 + -(-k // group) / 2) * 2.0 ** -23)
    block = 256 if M <= 8 else k
    for a in range(0, k, block):
        far += x[:, a: a + block].abs().amax(1, keepdim=True) * wide[:, a: a + block].abs().sum(1) * 2.0 ** -39
    if bias is not None:
        v = v + bias.double()
        far += v.abs() * 2.0 ** -23
    if epilogue == 1:
        far = 1.13 * far + v.abs() * 2.0 ** -20
        v = gelu(v)
    if epilogue == 2:
        v = y.double() + v
        far += v.abs() * 2.0 ** -23
    return v, far
