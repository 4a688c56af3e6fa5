"""Newton-Schulz steps in 64 bits with the roundings of the library as it is: fp16 operands, and X between the
steps in fp32 (a matrix in one cluster's registers) or, in the tiled kernels, as an fp16 number H and a byte of
the rest in 254ths of H's step, as long as the steps to come can multiply by more than four.

Tolerance: as in ortho_ref, whose model carries the rest in fp16: errors add like independent draws of these sizes, so a
result is within twice the model's distance from the exact one, plus half a step of bf16 (2^-8 of each element, so of
the norm) for its own rounding."""
import math

import torch

from ortho_ref import USUAL, exact, start


def kernel(m, n):
    """Which form takes a matrix: "tiny" (fp32 throughout), "small" (one cluster) or "tiled"."""
    r, q = min(m, n), max(m, n)
    return "tiny" if r <= 16 and q <= 8192 else ("small" if r <= 128 and q <= 4096 else "tiled")


def powers(coefs):
    """The powers of two that X, A and B are stored with: the largest values that the coefficients allow, below 2^14."""
    s = top = 1.0
    btop = 1.0
    for a, b, c in coefs:
        x = torch.linspace(0, s, 200001, dtype=torch.float64)
        btop = max(btop, float((b * x ** 2 + c * x ** 4).abs().max()))
        s = float((a * x + b * x ** 3 + c * x ** 5).abs().max())
        top = max(top, s)
    return [math.floor(math.log2(16384 / v)) for v in (top, top * top, btop)]


def fp16(x, e):
    return (x * 2.0 ** e).half().double() * 2.0 ** -e


def rest_in_a_byte(x, h, e):
    """What H leaves of X, to 1/254 of H's step; of a subnormal H nothing."""
    x, h = x * 2.0 ** e, h * 2.0 ** e
    power = (h.half().view(torch.int16) & 0x7C00).view(torch.float16).double()         # of two, of H; zero if subnormal
    step = torch.where(power > 0, power, 1.0) * 2.0 ** -10
    byte = torch.where(power > 0, torch.round((x - h) / step * 254), 0.0)
    assert float(byte.abs().max()) <= 127
    return byte / 254 * step * 2.0 ** -e


def rounded(g, coefs=USUAL, eps=1e-7, scale=1.0, form=None):
    form = form or kernel(*g.shape)
    ex, ea, eb = powers(coefs)
    x = start(g, eps)
    for k, (a, b, c) in enumerate(coefs):
        h = fp16(x, ex)
        if form == "tiled":
            grow = math.prod(max(1.0, abs(later[0])) for later in coefs[k:])
            x = h + rest_in_a_byte(x, h, ex) if grow > 4 else h
        s = fp16(h @ h.T, ea)
        m = b * s + c * (s @ s)
        d = torch.diag(m)
        x = a * x + d[:, None] * h + fp16(m - torch.diag(d), eb) @ h
    x = x * scale
    return x.T if g.shape[0] > g.shape[1] else x


def tolerance(g, coefs=USUAL, eps=1e-7, scale=1.0):
    """(exact result, Frobenius distance allowed)."""
    want = exact(g, coefs, eps, scale)
    return want, 2 * float((rounded(g, coefs, eps, scale) - want).norm()) + float(want.norm()) * 2.0 ** -8
