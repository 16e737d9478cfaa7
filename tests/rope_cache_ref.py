"""Plain 64-bit forms of the rotation and of the quantised key cache, for the tests."""
import math

import torch

E4M3_MAX = 448.0
HALF_STEP = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -25}


def frequencies(n, base=10000.0, scaling=None, factor=1.0, original=4096, fast=32.0, slow=1.0,
                coef=0.1):
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    at = lambda turns: n * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), n - 1)
    out = []
    for i, v in enumerate(f):
        r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append(v * (1 - r) + v / factor * r)
    return out, (coef * math.log(factor) + 1.0 if factor > 1 else 1.0)


def rotate(x, pos, freq, mag, offset, interleaved, grad=False):
    """(y in float64, bound on |y|'s terms per element) of x (..., heads, dim) at pos (...)."""
    y = x.double().clone()
    n = len(freq)
    a = pos.double().unsqueeze(-1) * torch.tensor(freq, dtype=torch.float64)
    cos, sin = (mag * torch.cos(a)).unsqueeze(-2), (mag * torch.sin(a)).unsqueeze(-2)
    if grad:
        sin = -sin
    if interleaved:
        u, v = slice(offset, offset + 2 * n, 2), slice(offset + 1, offset + 2 * n, 2)
    else:
        u, v = slice(offset, offset + n), slice(offset + n, offset + 2 * n)
    xu, xv = x[..., u].double(), x[..., v].double()
    y[..., u] = xu * cos - xv * sin
    y[..., v] = xu * sin + xv * cos
    terms = torch.zeros_like(y)
    terms[..., u] = terms[..., v] = mag * (xu.abs() + xv.abs())
    return y, terms


MAGS = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def quantise(x, pow2=False):
    """(codes as bytes, scale in float32) of rows x (n, D), from the exact quotients."""
    x = x.double()
    fin = torch.isfinite(x)
    amax = torch.where(fin, x.abs(), torch.zeros_like(x)).amax(-1)
    if pow2:
        s = torch.ones_like(amax)
        for i, m in enumerate(amax.tolist()):
            if m > 0:
                e = -90
                while 448.0 * 2.0 ** e < m:
                    e += 1
                s[i] = 2.0 ** e
    else:
        s = torch.where(amax > 0, (amax / E4M3_MAX).float().double().clamp_min(2.0 ** -90),
                        torch.ones_like(amax))
    t = torch.where(fin, (x / s[:, None]).abs(), torch.zeros_like(x))
    hi = torch.searchsorted(MAGS, t).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    up, down = MAGS[hi] - t, t - MAGS[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).to(torch.uint8)
    code = torch.where(torch.signbit(x), code | 128, code)
    return torch.where(fin, code, torch.full_like(code, 127)), s.float()


def places(seqused_k, table, block, S=None, cu=None, used=None, k_len=None):
    """[(row index (b, i) or r, cache row)] of the rows that take part."""
    out = []
    B = len(cu) - 1 if cu is not None else len(seqused_k)
    for b in range(B):
        n = cu[b + 1] - cu[b] if cu is not None else S
        if used is not None:
            n = used[b]
        L2 = seqused_k[b] if seqused_k is not None else k_len
        for i in range(n):
            p = L2 - n + i
            row = (cu[b] + i) if cu is not None else b * S + i
            slot = table[b][p // block] * block + p % block if table is not None else b * k_len + p
            out.append((row, slot))
    return out
