"""Definitions of the 4-bit microscaled path in 64 bits: quantisation by nearest
grid value, products of the values the codes stand for, and how far a computed
hidden may move an output.

Tolerances.  A sum of K products in fp32 (each product of two E2M1 values and a
power of two is exact there) is off by at most K 2^-23 sum |a b| (one rounding
or truncation of the running sum per term).  A stored bf16 value is off by half
a step, 2^-8 of it.  The hidden passes two roundings (bf16, then 4 bits), where
a sum's last bits may decide: `hidden_slack` gives, per element, how far its
4-bit value can be from the exact sums' one.
"""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BF16_HALF = 2.0 ** -8


def block_exp(amax):
    """Smallest e with amax <= 6 2^e, clamped to [-127, 127] (0 for a block of zeros)."""
    e = torch.full_like(amax, -127.0)
    for k in range(-126, 128):                           # a power at a time: no logarithm that may miss a border
        e = torch.where(amax > 6.0 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def quantise(x):
    """[..., K] -> (codes with the sign in bit 3, exponents [..., K / 32]), in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    e = block_exp(b.abs().amax(-1))
    a = (b / torch.exp2(e)[..., None]).abs()
    dist = (a[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    hit = dist == best                                   # two hits: a tie, which takes the even code
    idx = torch.arange(8).expand_as(dist)
    odd_tie = (hit.sum(-1) > 1)
    first = torch.where(hit, idx, torch.full_like(idx, 9)).amin(-1)
    code = torch.where(odd_tie & (first % 2 == 1), first + 1, first)
    return (code | (torch.signbit(b).long() << 3)).flatten(-2), e.long()


def value(codes, e):
    v = GRID[codes & 7] * (1 - 2 * (codes >> 3)).double()
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(e.double())[..., None]).flatten(-2)


def rounded(x):
    return value(*quantise(x))


def bf16(x):
    return x.to(torch.bfloat16).double()


def hidden(xq, w2q, w1q):
    """SiLU(x W2^T) (x W1^T) from quantised operands, and the radius of what fp32 sums may give."""
    K = xq.shape[-1]
    g, u = xq @ w2q.T, xq @ w1q.T
    eg, eu = ((xq.abs() @ w.abs().T) * K * 2.0 ** -23 for w in (w2q, w1q))
    s = g * torch.sigmoid(g)
    h = s * u
    # |SiLU'| <= 1.1; the exponential and the division: a few units of 2^-23, the exponent's rounding |g| 2^-23
    rad = 1.1 * eg * (u.abs() + eu) + (s.abs() + 1.1 * eg) * eu + h.abs() * (16 + 2 * g.abs()) * 2.0 ** -23
    return h, rad


def hidden_slack(h, rad):
    """(the hidden's 4-bit values, how far a computed one may be from them)."""
    want = rounded(bf16(h))
    slack = torch.zeros_like(want)
    sign = torch.sign(h)
    for top in (h.abs() + rad, (h.abs() - rad).clamp(min=0)):            # the block's largest, either way
        e = block_exp(bf16(top).unflatten(-1, (-1, 32)).amax(-1))
        scale = torch.exp2(e)[..., None]
        for v in (h.abs() + rad, (h.abs() - rad).clamp(min=0)):
            a = (bf16(v).unflatten(-1, (-1, 32)) / scale)
            dist = (a[..., None] - GRID).abs()
            near = dist <= dist.amin(-1, keepdim=True) + 1e-12              # a tie: either neighbour
            for pick in (torch.where(near, GRID, 9.0).amin(-1), torch.where(near, GRID, -1.0).amax(-1)):
                got = (pick * scale).flatten(-2) * torch.where(sign == 0, 1.0, sign)
                slack = torch.maximum(slack, torch.where(rad > 0, (got - want).abs(), 0.0))
    # a value whose sign the radius does not settle is below the smallest code's half step or counted by its magnitude twice
    return want, torch.where((h.abs() < rad), slack + want.abs(), slack)


def expert(xq, w1, w2, w3):
    """y = h W3^T of one expert (weights as stored, quantised here), and the bound of an fp32 result."""
    h, rad = hidden(xq, rounded(w2), rounded(w1))
    hq, slack = hidden_slack(h, rad)
    w3q = rounded(w3)
    y = hq @ w3q.T
    return y, slack @ w3q.abs().T + ((hq.abs() + slack) @ w3q.abs().T) * h.shape[-1] * 2.0 ** -23
