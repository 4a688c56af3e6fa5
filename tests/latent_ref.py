"""Plain 64-bit definitions of the attention operators, with the bound on what
bf16 storage and fp32 sums may cost each output element.

Roundings counted: a bf16 value is off by at most 2^-8 of itself (half a step);
probabilities p and their gradients ds enter the second products as bf16, so a
sum of p_j c_j is off by at most 2^-8 sum p_j |c_j|, and the output's own
storage adds 2^-8 of the output.  A score is an fp32 sum of n products: off by at
most (n + 8) 2^-24 sum |q k| scale (the 8: scaling, the exponential's argument
and result); an error d in the score multiplies p by e^d <= 1 + 2 d.
"""
import math

import torch

HALF = 2.0 ** -8          # bf16: torch.finfo(torch.bfloat16).eps / 2
ULP32 = 2.0 ** -24        # fp32: eps / 2


def inv_freq(d, base=10000.0, factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0, mscale=1.0):
    f = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if factor == 1.0:
        return f
    idx = lambda n: d * math.log(orig_len / (n * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(idx(beta_fast)), 0), min(math.ceil(idx(beta_slow)), d - 1)
    out = []
    for i, v in enumerate(f):
        r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        out.append(v / factor * r + v * (1 - r))
    return out


def rope(x, pos, d, layout, inverse=False, **kw):
    """(y, |a| + |b| of each element's pair) in 64 bits."""
    f = torch.tensor(inv_freq(d, **kw), dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * f
    c, s = ang.cos() * kw.get("mscale", 1.0), ang.sin() * kw.get("mscale", 1.0) * (-1 if inverse else 1)
    x = x.double()
    y, mag = torch.empty_like(x), torch.empty_like(x)
    ia = torch.arange(0, d, 2) if layout == "interleaved" else torch.arange(d // 2)
    ib = ia + 1 if layout == "interleaved" else ia + d // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * kw.get("mscale", 1.0)
    return y, mag


def pow2(e):
    """2^e in 64 bits from its bit pattern (a power function may be off by an ulp)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def fp8_rows(c):
    """E4M3 codes times the row's power-of-two scale, as 64-bit values, and the scales."""
    x = c.double()
    m, ex = torch.frexp(x.abs().amax(-1, keepdim=True))          # 448 = 0.875 * 2^9
    e = torch.where(m > 0, ex - 9 + (m > 0.875), 0)
    u = x * pow2(-e)
    step = pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)     # 2^(floor(log2 u) - 3)
    return torch.round(u / step) * step * pow2(e), pow2(e)


def attend(q, k, v, scale, vis):
    """out, lse, and bounds on both, of q [n, d], k [m, d], v [m, dv] (64 bits), vis [n, m]."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        z = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
        return z, z.new_full((q.shape[0],), -math.inf), z, z.new_zeros((q.shape[0],))
    s = (q @ k.T * scale).masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.softmax(s, 1).nan_to_num(0.0)
    out = p @ v
    d = ((k.shape[1] + 8) * ULP32 * abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~vis, 0.0)
    d = d.amax(1) + 8 * ULP32 * s.abs().masked_fill(~vis, 0.0).amax(1)
    # the sum's own rounding: at most m additions of positive fp32 terms
    zerr = (k.shape[0] + 8) * ULP32
    tol = HALF * out.abs() + (HALF + 4 * d + zerr)[:, None] * (p @ v.abs()) + 1e-30
    return out, lse, tol, 2 * d + zerr + 4 * ULP32 * lse.abs().nan_to_num(0, 0, 0)


def attend_grad(q, k, v, scale, vis, out, lse, do):
    """dq, dk, dv at the stored out and lse, and bounds on each (64 bits)."""
    q, k, v, out, lse, do = (t.double() for t in (q, k, v, out, lse, do))
    s = (q @ k.T * scale).masked_fill(~vis, -math.inf)
    p = (s - lse[:, None]).exp().masked_fill(~vis, 0.0)
    dp = do @ v.T - (do * out).sum(1, keepdim=True)
    ds = p * dp * scale
    d = (k.shape[1] + 8) * ULP32 * abs(scale) * (q.abs() @ k.abs().T) + 8 * ULP32 * (s.abs() + lse.abs()[:, None])
    d = d.masked_fill(~vis, 0.0)
    dperr = (v.shape[1] + 8) * ULP32 * (do.abs() @ v.abs().T + (do * out).abs().sum(1, keepdim=True))
    n = (max(s.shape) + 8) * ULP32                         # fp32 sums over rows or keys
    perr = p * (HALF + 2 * d + n)
    dserr = ds.abs() * (HALF + 2 * d + n) + p * dperr * abs(scale)
    dq, dk, dv = ds @ k, ds.T @ q, p.T @ do
    tq = HALF * dq.abs() + dserr @ k.abs() + 1e-30
    tk = HALF * dk.abs() + dserr.T @ q.abs() + 1e-30
    tv = HALF * dv.abs() + perr.T @ do.abs() + 1e-30
    return (dq, dk, dv), (tq, tk, tv)


def visible(lq, lk, causal, device):
    i, j = torch.arange(lq, device=device)[:, None], torch.arange(lk, device=device)[None]
    return j <= i + (lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device=device)


def within(got, want, tol, what):
    """|got - want| <= tol everywhere; equal infinities agree."""
    got = got.double()
    assert not got.isnan().any(), "%s: NaN" % what
    same = got == want
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(tol[bad].min()))
