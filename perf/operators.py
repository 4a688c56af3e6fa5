"""Cases of the latent-attention operators: rotary positions, the paged latent
cache (written, bf16 or FP8, and read back), absorbed attention of a few new
tokens over that cache, and expanded attention of whole sequences with its
gradient.

One token's keys and values come from one latent vector c (512) and one rotary
key k_r (64) that all heads share:
  absorbed   s = scale (q_l . c + q_r . k_r),  out = softmax(s) c          (q_l = W_UK^T q_n)
  expanded   s = scale (q_n . k_n + q_r . k_r), out = softmax(s) v         (k_n = W_UK c, v = W_UV c)
Heads: 128 (DeepSeek-V3) or 16 (DeepSeek-V2-Lite), other counts in the drawn cases.

`listed()` gives the cases, `prepare` their inputs, `run` one pass (plain torch
where `own` is false, the library's calls where it is true), `exact` the
definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LAT, ROT, NOPE, DV = 512, 64, 128, 128
REC_FP8 = LAT + 2 * ROT + 16          # codes, rotary key (bf16), scale (fp32) and 12 bytes of padding
# long-context scaling of the rotary frequencies as a 4,096-token model extended 40-fold uses it
SCALED = dict(base=10000.0, factor=40.0, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0, mscale=1.0)
PLAIN = dict(base=10000.0, factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0, mscale=1.0)


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # the query heads' rotary part in one decode step of 1,024 sequences at far positions
        dict(name="rope_decode", op="rope", T=1024, H=128, d=64, layout="interleaved", scaled=True, inverse=False,
             dtype="bf16", max_pos=163840),
        # the gradient of the rotation over a training batch of 65,536 tokens, half layout
        dict(name="rope_grad", op="rope", T=65536, H=32, d=128, layout="half", scaled=False, inverse=True,
             dtype="bf16", max_pos=2048),
        # one decode step's new tokens into a bf16 cache (rotary key rotated on the way) and back
        dict(name="cache_step", op="cache", T=1024, cache="bf16", page=64, n_pages=512, rotate=True),
        # a prefill batch quantised into an FP8 cache and read back for the next chunk's expanded form
        dict(name="cache_prefill_fp8", op="cache", T=65533, cache="fp8", page=64, n_pages=1152, rotate=True),
        # one user, one token, 16 heads: latency
        dict(name="decode_one", op="decode", H=16, B=1, n_q=1, lo=4097, hi=4097, page=64, cache="bf16", ls=1),
        # a serving batch of the 128-head model, ragged lengths
        dict(name="decode_128h", op="decode", H=128, B=64, n_q=1, lo=2000, hi=14000, page=64, cache="bf16", ls=2),
        # a large batch of the 16-head model on an FP8 cache
        dict(name="decode_16h_fp8", op="decode", H=16, B=256, n_q=1, lo=1, hi=8191, page=64, cache="fp8", ls=3),
        # two speculated tokens a sequence, 128 heads, FP8 cache, pages that end inside a tile
        dict(name="decode_spec_fp8", op="decode", H=128, B=32, n_q=2, lo=1000, hi=9000, page=48, cache="fp8", ls=4),
        # a ragged batch of short prompts, some behind an already cached prefix
        dict(name="prefill_ragged", op="prefill", H=16, lq="333,1,700,64,235", lk="333,129,700,191,235",
             causal=True),
        # a prefill batch of the 128-head model
        dict(name="prefill_128h", op="prefill", H=128, lq="2048,2048,2048,2048", lk="2048,2048,2048,2048", causal=True),
        # the gradient over a training batch of the 16-head model
        dict(name="grad_16h", op="grad", H=16, lq="2048,2048,2048,2048", lk="2048,2048,2048,2048", causal=True),
        # the gradient over packed sequences of odd lengths
        dict(name="grad_ragged", op="grad", H=16, lq="129,515,1,1000", lk="129,515,70,1000", causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "decode", "decode", "prefill", "grad"])
    if op == "rope":
        H, d = rng.choice([1, 3, 16, 32, 128]), rng.choice([32, 64, 128])
        T = _log(rng, 1, min(65536, 65536 * 32 * 128 // (H * d)))
        return dict(op=op, T=T, H=H, d=d, layout=rng.choice(["interleaved", "half"]), scaled=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]) if T * H * d < 2 ** 26
                    else "bf16", max_pos=_log(rng, 2, 1 << 20))
    if op == "cache":
        T, page = _log(rng, 1, 65533), rng.choice([1, 16, 48, 64, 100, 128])
        return dict(op=op, T=T, cache=rng.choice(["bf16", "fp8"]), page=page,
                    n_pages=(T + page - 1) // page + rng.randrange(1, 100), rotate=rng.random() < 0.7)
    if op == "decode":
        H, n_q = rng.choice([1, 5, 16, 16, 24, 64, 128, 128]), rng.choice([1, 1, 1, 2, 3, 4])
        B = _log(rng, 1, 256)
        top = min(16384, 256 * 4096 // B, 64 * 8000 * 128 // (B * H * n_q))
        hi = _log(rng, min(16, top), top)
        return dict(op=op, H=H, B=B, n_q=n_q, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi,
                    page=rng.choice([1, 16, 48, 64, 100, 128]), cache=rng.choice(["bf16", "fp8"]),
                    ls=rng.randrange(1 << 20))
    H = rng.choice([1, 3, 16, 16, 32]) if op == "grad" else rng.choice([1, 5, 16, 32, 128])
    B = rng.randrange(1, 7)
    top = 2048 if H <= 32 else 1024
    lq = [_log(rng, 1, top) for _ in range(B)]
    lk = [n if rng.random() < 0.6 else _log(rng, 1, top) for n in lq]
    return dict(op=op, H=H, lq=",".join(map(str, lq)), lk=",".join(map(str, lk)), causal=rng.random() < 0.8)


def _lens(case):
    r = random.Random(case["ls"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _seqs(case):
    """(queries, keys) of each packed sequence."""
    return [(int(a), int(b)) for a, b in zip(case["lq"].split(","), case["lk"].split(","))]


def _pairs(case):
    """Visible (query, key) pairs of a prefill case, one head."""
    n = 0
    for a, b in _seqs(case):
        if not case["causal"]:
            n += a * b
        else:                                   # query i sees keys 0 .. b - a + i
            for_first = max(0, a - b)           # queries that see nothing
            m = a - for_first
            n += m * (max(0, b - a) + 1) + m * (m - 1) // 2
    return n


def work(case):
    op = case["op"]
    if op == "rope":
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * case["H"] * case["d"]
        return {"bytes": 2 * n * es + 4 * case["T"], "flops": 3 * n}
    if op == "cache":
        row = 2 * (LAT + ROT)
        rec = REC_FP8 - 12 if case["cache"] == "fp8" else row
        return {"bytes": case["T"] * (2 * row + 2 * rec + 20), "flops": case["T"] * (4 * LAT + 3 * ROT)}
    if op == "decode":
        rows, n = case["B"] * case["n_q"] * case["H"], sum(_lens(case))
        rec = REC_FP8 - 12 if case["cache"] == "fp8" else 2 * (LAT + ROT)
        return {"bytes": n * rec + rows * (2 * (LAT + ROT) + 2 * LAT + 4),
                "flops": 2 * n * case["n_q"] * case["H"] * (2 * LAT + ROT)}
    H, p = case["H"], _pairs(case)
    tq, tk = (sum(n) for n in zip(*_seqs(case)))
    io = 2 * (tq * H * (NOPE + ROT) + tk * H * (NOPE + DV) + tk * ROT)         # q, k_n, v, k_r
    o = 2 * tq * H * DV + 4 * tq * H                                           # out, lse
    if op == "prefill":
        return {"bytes": io + o, "flops": 2 * p * H * (NOPE + ROT + DV)}
    # S, dP, dV, dK, dQ; out, lse and d_out read, a gradient for each input written
    return {"bytes": 2 * io + o + 2 * tq * H * DV, "flops": 2 * p * H * (3 * (NOPE + ROT) + 2 * DV)}


# ----------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _pow2(e):
    """2^e in 64 bits from its bit pattern (a power function may be off by an ulp)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _fp8_rows(c):
    """bf16 rows -> E4M3 codes and the power-of-two scale of each row (the smallest
    2^e with max |x| 2^-e <= 448)."""
    x = c.float()
    m, ex = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, torch.zeros_like(ex), torch.where(m <= 0.875, ex - 9, ex - 8))
    s = _pow2(e).float()
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


def _fill_cache(cache, c, kr):
    """Every slot of a cache in its record layout (what earlier steps left there)."""
    if cache.dtype == torch.bfloat16:
        cache.view(-1, LAT + ROT).copy_(torch.cat([c, kr], 1))
        return
    codes, s = _fp8_rows(c)
    rec = cache.view(-1, REC_FP8)
    rec[:, :LAT] = codes.view(torch.uint8)
    rec[:, LAT:LAT + 2 * ROT] = kr.contiguous().view(torch.uint8)
    rec[:, LAT + 2 * ROT:LAT + 2 * ROT + 4] = s[:, None].contiguous().view(torch.uint8)


def _new_cache(kind, n_pages, page):
    if kind == "bf16":
        return torch.zeros((n_pages, page, LAT + ROT), dtype=torch.bfloat16, device=DEV)
    return torch.zeros((n_pages, page, REC_FP8), dtype=torch.uint8, device=DEV)


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        T, H, d = case["T"], case["H"], case["d"]
        # the rotated part sits behind 64 unrotated elements of each head
        full = torch.randn((T, H, 64 + d), generator=g, device=DEV).to(dt)
        st.update(x=full[:, :, 64:], y=torch.empty((T, H, d), dtype=dt, device=DEV),
                  pos=torch.randint(0, case["max_pos"], (T,), generator=g, device=DEV, dtype=torch.int32))
    elif op == "cache":
        T, n = case["T"], case["n_pages"] * case["page"]
        st.update(c=_randn(g, (T, LAT)), kr=_randn(g, (T, ROT)),
                  pos=torch.randint(0, 163840, (T,), generator=g, device=DEV, dtype=torch.int32),
                  slots=torch.randperm(n, generator=g, device=DEV)[:T].contiguous(),
                  cache=_new_cache(case["cache"], case["n_pages"], case["page"]),
                  c_back=torch.empty((T, LAT), dtype=torch.bfloat16, device=DEV),
                  kr_back=torch.empty((T, ROT), dtype=torch.bfloat16, device=DEV))
    elif op == "decode":
        lens, page = _lens(case), case["page"]
        need = [(n + page - 1) // page for n in lens]
        total, width = max(1, sum(need)), max(1, max(need))
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros((case["B"], width), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        cache = _new_cache(case["cache"], total, page)
        _fill_cache(cache, _randn(g, (total * page, LAT)), _randn(g, (total * page, ROT)))
        rows, H = case["B"] * case["n_q"], case["H"]
        st.update(ql=_randn(g, (rows, H, LAT), 0.5), qr=_randn(g, (rows, H, ROT)), cache=cache, table=table,
                  lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scale=1.0 / math.sqrt(NOPE + ROT),
                  out=torch.empty((rows, H, LAT), dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty((rows, H), dtype=torch.float32, device=DEV))
    else:
        H, lq, lk = case["H"], [a for a, _ in _seqs(case)], [b for _, b in _seqs(case)]
        tq, tk = sum(lq), sum(lk)
        kv = _randn(g, (tk, H, NOPE + DV))                       # the up-projection's output: [k_n | v] per head
        st.update(q=_randn(g, (tq, H, NOPE + ROT)), kn=kv[:, :, :NOPE], v=kv[:, :, NOPE:], kr=_randn(g, (tk, ROT)),
                  cu_q=_cu(lq), cu_k=_cu(lk), scale=1.0 / math.sqrt(NOPE + ROT),
                  out=torch.empty((tq, H, DV), dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty((H, tq), dtype=torch.float32, device=DEV))
        if op == "grad":
            st["do"] = _randn(g, (tq, H, DV))
            o, lse = _plain_prefill(st)                          # what the forward pass left
            st["out"].copy_(o)
            st["lse"].copy_(lse)
            dkv = torch.empty((tk, H, NOPE + DV), dtype=torch.bfloat16, device=DEV)
            st.update(dq=torch.empty_like(st["q"]), dkn=dkv[:, :, :NOPE], dv=dkv[:, :, NOPE:],
                      dkr=torch.empty_like(st["kr"]))
    if own:
        _handles(st)
    return st


def _rope_args(case):
    if case["op"] == "rope":
        return case["d"], case["layout"], SCALED if case["scaled"] else PLAIN
    return ROT, "interleaved", SCALED


def _handles(st):
    """What a program keeps across calls: descriptors and workspaces."""
    from mixture_experts_layer_expert_gb300 import fs
    case, op = st["case"], st["case"]["op"]
    if op in ("rope", "cache"):
        d, layout, kw = _rope_args(case)
        st["rope"] = fs.make_rope(d, layout, **kw)
    if op == "cache":
        st["desc"] = fs.make_latent_cache(case["n_pages"], case["page"], case["cache"])
    if op == "decode":
        st["desc"] = fs.make_latent_cache(st["cache"].shape[0], case["page"], case["cache"])
        st["ws"] = torch.empty(fs.fs_latent_decode_ws_bytes(case["H"], case["B"], case["n_q"]), dtype=torch.uint8,
                               device=DEV)
    if op == "grad":
        st["ws"] = torch.empty(fs.fs_latent_prefill_backward_ws_bytes(case["H"], st["q"].shape[0], st["kr"].shape[0]),
                               dtype=torch.uint8, device=DEV)
    st["fs"] = fs


# ---------------------------------------------------------------- the operators

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    if "fs" not in st:
        _handles(st)
    fs, case, op = st["fs"], st["case"], st["case"]["op"]
    if op == "rope":
        fs.fs_rope(st["rope"], st["pos"], st["x"], st["y"], inverse=case["inverse"])
        return st["y"]
    if op == "cache":
        rot = case["rotate"]
        fs.fs_latent_cache_write(st["desc"], st["c"], st["kr"], st["slots"], st["cache"],
                                 rope=st["rope"] if rot else None, pos=st["pos"] if rot else None)
        fs.fs_latent_cache_read(st["desc"], st["cache"], st["slots"], st["c_back"], st["kr_back"])
        return st["c_back"], st["kr_back"]
    if op == "decode":
        fs.fs_latent_decode(st["desc"], st["ql"], st["qr"], st["cache"], st["table"], st["lens"], st["scale"],
                            st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    if op == "prefill":
        fs.fs_latent_prefill(st["q"], st["kn"], st["kr"], st["v"], st["cu_q"], st["cu_k"], case["causal"],
                             st["scale"], st["out"], st["lse"])
        return st["out"], st["lse"]
    fs.fs_latent_prefill_backward(st["q"], st["kn"], st["kr"], st["v"], st["cu_q"], st["cu_k"], case["causal"],
                                  st["scale"], st["out"], st["lse"], st["do"], st["dq"], st["dkn"], st["dkr"],
                                  st["dv"], st["ws"])
    return st["dq"], st["dkn"], st["dkr"], st["dv"]


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "rope":
        return _plain_rope(st["x"], st["pos"], *_rope_args(case), case["inverse"])
    if op == "cache":
        kr = st["kr"]
        if case["rotate"]:
            kr = _plain_rope(kr[:, None, :], st["pos"], *_rope_args(case), False)[:, 0]
        rec, slots = st["cache"].view(-1, st["cache"].shape[-1]), st["slots"]
        if case["cache"] == "bf16":
            rec[slots, :LAT] = st["c"]
            rec[slots, LAT:] = kr
        else:
            codes, s = _fp8_rows(st["c"])
            rec[slots, :LAT] = codes.view(torch.uint8)
            rec[slots, LAT:LAT + 2 * ROT] = kr.contiguous().view(torch.uint8)
            rec[slots, LAT + 2 * ROT:LAT + 2 * ROT + 4] = s[:, None].contiguous().view(torch.uint8)
        c, kr = _records(rec[slots])
        return c.to(torch.bfloat16), kr.to(torch.bfloat16)
    if op == "decode":
        return _plain_decode(st)
    if op == "prefill":
        o, lse = _plain_prefill(st)
        return o.to(torch.bfloat16), lse
    return _plain_grad(st)


def _inv_freq(d, base, factor, orig_len, beta_fast, beta_slow, **_):
    f = base ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
    if factor == 1.0:
        return f

    def dim(turns):                             # the frequency index that makes `turns` turns over orig_len
        return d * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(dim(beta_fast)), 0), min(math.ceil(dim(beta_slow)), d - 1)
    ramp = ((torch.arange(d // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp)


def _plain_rope(x, pos, d, layout, kw, inverse):
    ang = pos.double()[:, None] * _inv_freq(d, **kw)             # 64 bits: far positions lose their angle in 32
    cos, sin = (ang.cos() * kw["mscale"]).float()[:, None], (ang.sin() * kw["mscale"]).float()[:, None]
    if inverse:
        sin = -sin
    xf = x.float()
    a, b = (xf[..., 0::2], xf[..., 1::2]) if layout == "interleaved" else (xf[..., :d // 2], xf[..., d // 2:])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([ya, yb], -1).flatten(-2) if layout == "interleaved" else torch.cat([ya, yb], -1)
    return y.to(x.dtype)


def _records(rec):
    """Cache records -> latent rows and rotary keys, fp32."""
    if rec.dtype == torch.bfloat16:
        return rec[..., :LAT].float(), rec[..., LAT:].float()
    scale = rec[..., LAT + 2 * ROT:LAT + 2 * ROT + 4].contiguous().view(torch.float32)
    return (rec[..., :LAT].contiguous().view(torch.float8_e4m3fn).float() * scale,
            rec[..., LAT:LAT + 2 * ROT].contiguous().view(torch.bfloat16).float())


def _plain_decode(st):
    case, table, lens = st["case"], st["table"], st["lens"]
    B, n_q, H = case["B"], case["n_q"], case["H"]
    pages = st["cache"][table.long()]                            # [B, width, page, record]
    c, kr = _records(pages.flatten(1, 2))
    L = c.shape[1]
    q = torch.cat([st["ql"], st["qr"]], -1).float().view(B, n_q * H, LAT + ROT)
    s = torch.bmm(q, torch.cat([c, kr], -1).transpose(1, 2)).view(B, n_q, H, L) * st["scale"]
    # query j of n_q sees the positions before lens - (n_q - 1 - j)
    end = lens[:, None] - (n_q - 1 - torch.arange(n_q, device=DEV))[None]
    s = s.masked_fill(torch.arange(L, device=DEV) >= end[:, :, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = (s - m).exp()
    z = p.sum(-1, keepdim=True)
    o = torch.bmm((p / z.clamp_min(1e-30)).view(B, n_q * H, L), c)
    lse = (m + z.log()).view(B * n_q, H)
    return o.view(B * n_q, H, LAT).to(torch.bfloat16), lse


def _visible(lq, lk, causal):
    i, j = torch.arange(lq, device=DEV)[:, None], torch.arange(lk, device=DEV)[None]
    return j <= i + (lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device=DEV)


def _segments(case):
    a = b = 0
    for lq, lk in _seqs(case):
        yield slice(a, a + lq), slice(b, b + lk), lq, lk
        a, b = a + lq, b + lk


def _plain_scores(st, sq, sk, lq, lk):
    """Scaled, masked scores [H, lq, lk] of one sequence, fp32, and the key rows [H, lk, 192]."""
    H = st["q"].shape[1]
    k = torch.cat([st["kn"][sk].float(), st["kr"][sk].float()[:, None].expand(lk, H, ROT)], -1).transpose(0, 1)
    s = torch.bmm(st["q"][sq].float().transpose(0, 1), k.transpose(1, 2)) * st["scale"]
    return s.masked_fill(~_visible(lq, lk, st["case"]["causal"]), float("-inf")), k


def _plain_prefill(st):
    o = torch.zeros(st["out"].shape, device=DEV)
    lse = torch.full(st["lse"].shape, float("-inf"), device=DEV)
    for sq, sk, lq, lk in _segments(st["case"]):
        s, _ = _plain_scores(st, sq, sk, lq, lk)
        m = s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
        p = (s - m).exp()
        z = p.sum(-1, keepdim=True)
        o[sq] = torch.bmm(p / z.clamp_min(1e-30), st["v"][sk].float().transpose(0, 1)).transpose(0, 1)
        lse[:, sq] = (m + z.log())[..., 0]
    return o, lse


def _plain_grad(st):
    f32 = dict(dtype=torch.float32, device=DEV)
    dq, dkn = torch.zeros(st["q"].shape, **f32), torch.zeros(st["kn"].shape, **f32)
    dkr, dv = torch.zeros(st["kr"].shape, **f32), torch.zeros(st["v"].shape, **f32)
    for sq, sk, lq, lk in _segments(st["case"]):
        s, k = _plain_scores(st, sq, sk, lq, lk)
        lse = st["lse"][:, sq, None]
        p = torch.where(s == float("-inf"), torch.zeros_like(s), (s - lse).exp())
        do = st["do"][sq].float().transpose(0, 1)
        delta = (do * st["out"][sq].float().transpose(0, 1)).sum(-1, keepdim=True)
        dv[sk] = torch.bmm(p.transpose(1, 2), do).transpose(0, 1)
        ds = p * (torch.bmm(do, st["v"][sk].float().permute(1, 2, 0)) - delta) * st["scale"]
        dq[sq] = torch.bmm(ds, k).transpose(0, 1)
        dk = torch.bmm(ds.transpose(1, 2), st["q"][sq].float().transpose(0, 1)).transpose(0, 1)
        dkn[sk] = dk[..., :NOPE]
        dkr[sk] = dk[..., NOPE:].sum(1)
    return tuple(t.to(torch.bfloat16) for t in (dq, dkn, dkr, dv))


# ------------------------------------------------------- the definition, 64 bits

def _exact_rope(x, pos, d, layout, kw, inverse):
    """Each pair as a complex number times exp(+-i angle)."""
    pair = torch.arange(d // 2, device=DEV)
    ia, ib = (2 * pair, 2 * pair + 1) if layout == "interleaved" else (pair, pair + d // 2)
    z = torch.complex(x[..., ia].double(), x[..., ib].double())
    ang = pos.double()[:, None, None] * _inv_freq(d, **kw)
    z = z * torch.polar(torch.full_like(ang, kw["mscale"]), -ang if inverse else ang)
    y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _exact_e4m3(c):
    """The values that E4M3 codes with a power-of-two row scale stand for."""
    x = c.double()
    m, ex = torch.frexp(x.abs().amax(-1, keepdim=True))          # 448 = 0.875 * 2^9
    e = torch.where(m > 0, ex - 9 + (m > 0.875), 0)
    u = x * _pow2(-e)
    step = _pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)     # 2^(floor(log2 u) - 3)
    return torch.round(u / step) * step * _pow2(e)               # torch.round: ties to even


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rope":
        return _exact_rope(st["x"], st["pos"], *_rope_args(case), case["inverse"])
    if op == "cache":
        kr = st["kr"].double()
        if case["rotate"]:
            kr = _exact_rope(st["kr"][:, None], st["pos"], *_rope_args(case), False)[:, 0]
        return st["c"].double() if case["cache"] == "bf16" else _exact_e4m3(st["c"]), kr
    if op == "decode":
        n_q, H = case["n_q"], case["H"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(case)):
            idx = torch.arange(n, device=DEV)
            rec = st["cache"][st["table"][b].long()[idx // case["page"]], idx % case["page"]]
            c, kr = (t.double() for t in _records(rec))
            for j in range(n_q):
                r, end = b * n_q + j, n - (n_q - 1 - j)
                if end <= 0:
                    continue
                s = (st["ql"][r].double() @ c[:end].T + st["qr"][r].double() @ kr[:end].T) * st["scale"]
                lse[r] = torch.logsumexp(s, -1)
                out[r] = torch.softmax(s, -1) @ c[:end]
        return out, lse
    f64 = dict(dtype=torch.float64, device=DEV)
    H = case["H"]
    out, lse = torch.zeros(st["out"].shape, **f64), torch.full(st["lse"].shape, -math.inf, **f64)
    dq, dk = torch.zeros(st["q"].shape, **f64), torch.zeros((st["kr"].shape[0], H, NOPE + ROT), **f64)
    dv = torch.zeros(st["v"].shape, **f64)
    for sq, sk, lq, lk in _segments(case):
        hidden = ~_visible(lq, lk, case["causal"])
        for h in range(H):
            q, v = st["q"][sq, h].double(), st["v"][sk, h].double()
            k = torch.cat([st["kn"][sk, h], st["kr"][sk]], 1).double()
            s = (q @ k.T * st["scale"]).masked_fill(hidden, -math.inf)
            if op == "prefill":
                lse[h, sq] = torch.logsumexp(s, 1)
                out[sq, h] = torch.softmax(s, 1).nan_to_num(0.0) @ v
                continue
            # the gradient at the out and lse that the forward pass stored
            p = (s - st["lse"][h, sq, None].double()).exp().masked_fill(hidden, 0.0)
            do = st["do"][sq, h].double()
            dv[sk, h] = p.T @ do
            ds = p * (do @ v.T - (do * st["out"][sq, h].double()).sum(1, keepdim=True)) * st["scale"]
            dq[sq, h], dk[sk, h] = ds @ k, ds.T @ q
    if op == "prefill":
        return out, lse
    return dq, dk[..., :NOPE], dk[..., NOPE:].sum(1), dv
