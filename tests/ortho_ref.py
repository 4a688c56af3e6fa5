"""Newton-Schulz steps in 64 bits, exactly and with the roundings that the library
documents (products of fp16 operands, X carried as a pair of them).

Tolerance.  The second form has every documented rounding, half a step each (fp16
2^-11 relative), and sums in 64 bits; what it does not have are fp32 sums (2^-24 a
term, below 1% of the operands' roundings for the lengths tested) and the other
outcome of a rounding on a border.  Errors add like independent draws of the same
sizes, so a result is within twice this form's distance from the exact one, plus half
a step of bf16 (2^-8 of each element, so of the norm) for its own rounding."""
import torch

USUAL = [(3.4445, -4.7750, 2.0315)] * 5


def start(g, eps):
    x = g.double()
    x = x.T if x.shape[0] > x.shape[1] else x
    top = x.abs().max()
    if top == 0:
        return x
    norm = torch.linalg.vector_norm(x / top) * top
    return x / (norm + eps)


def exact(g, coefs=USUAL, eps=1e-7, scale=1.0):
    x = start(g, eps)
    for a, b, c in coefs:
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    x = x * scale
    return x.T if g.shape[0] > g.shape[1] else x


def half(x, e):
    return torch.ldexp(torch.ldexp(x, torch.tensor(e)).half().double(), torch.tensor(-e))


def rounded(g, coefs=USUAL, eps=1e-7, scale=1.0):
    """With H = fp16(X), L = fp16 of the rest while later steps can multiply by more than four; A and B fp16, B's
    diagonal apart and applied to H; powers of two as for singular values below 2."""
    x = start(g, eps)
    for k, (a, b, c) in enumerate(coefs):
        h = half(x, 13)
        grow = 1.0
        for later in coefs[k:]:
            grow *= max(1.0, abs(later[0]))
        x = h + half(x - h, 24) if grow > 4 else h
        s = half(h @ h.T, 12)
        m = b * s + c * (s @ s)
        d = torch.diag(m)
        x = a * x + d[:, None] * h + half(m - torch.diag(d), 10) @ h
    x = x * scale
    return x.T if g.shape[0] > g.shape[1] else x


def tolerance(g, coefs=USUAL, eps=1e-7, scale=1.0):
    """(exact result, Frobenius distance allowed)."""
    want = exact(g, coefs, eps, scale)
    return want, 2 * float((rounded(g, coefs, eps, scale) - want).norm()) + float(want.norm()) * 2.0 ** -8


def gradient(m, n, rank, seed, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    r = max(1, rank)
    return ((torch.randn((m, r), generator=g) @ torch.randn((r, n), generator=g)) * (1e-3 / r)).to(device)
