"""Cases of the operators around the MoE layer's router and experts: the balance
loss with the per-expert counts and its gradient, products in microscaled 4-bit
floating point (a dense projection, the routed experts), and the orthogonalised
update of weight gradients.

  balance   s = softmax(z + b), or sigmoid(z + b) over its sum; over the n counted tokens of a
            sequence f_e = E count_e / (k n), P_e = mean s_e; loss = coef mean_seq sum_e f_e P_e
  mx4       blocks of 32 along the contraction: codes in {0, .5, 1, 1.5, 2, 3, 4, 6} times +-2^e, e the
            smallest with max <= 6 2^e; products of the values they stand for
  ortho     X = G / (|G| + eps), five steps of X <- a X + (b A + c A A) X, A = X X^T (tall G: on G^T)

`listed()` gives the cases, `prepare` their inputs, `run` one pass (plain torch
where `own` is false, the library's calls where it is true), `exact` the
definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
COEFS = (3.4445, -4.7750, 2.0315)     # of every step
EPS = 1e-7
GATES = ["softmax", "softmax_renorm", "sigmoid", "sigmoid_norm"]


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # a small test layer's microbatch: launches and latency
        dict(name="balance_small", op="balance", T=256, E=8, k=2, gate="softmax_renorm", seqs=1, masked=False, bias=False),
        # one layer of a 65,536-token training batch, 256 experts
        dict(name="balance_v3", op="balance", T=65536, E=256, k=8, gate="sigmoid_norm", seqs=1, masked=False, bias=False),
        # the loss of each sequence of a packed, partly padded batch, 128 experts with a router bias
        dict(name="balance_seqs", op="balance", T=16384, E=128, k=8, gate="softmax_renorm", seqs=13, masked=True,
             bias=True),
        # one token's projection in a decode step: the weights' bytes
        dict(name="linear_one", op="linear", rows=1, N=7168, K=2048, out="bf16"),
        # a prefill batch through a projection, odd number of rows, fp32 out
        dict(name="linear_prefill", op="linear", rows=16381, N=2048, K=7168, out="f32"),
        # the routed experts of one decode step, 64 experts, width not a multiple of 256
        dict(name="moe_decode", op="moe", T=61, d=2048, c=1408, E=64, k=6),
        # the routed experts of a prefill batch at the large layer's widths (32 of its 256 experts)
        dict(name="moe_prefill", op="moe", T=8192, d=7168, c=2048, E=32, k=8),
        # the router's weight gradient of the 64-expert layer
        dict(name="ortho_router", op="ortho", batch=1, m=64, n=2048, tokens=8192, dtype="f32", scale=1.0),
        # all down projections of a small test layer
        dict(name="ortho_small", op="ortho", batch=8, m=256, n=128, tokens=512, dtype="f32", scale=1.0),
        # a few odd matrices, bf16 gradients
        dict(name="ortho_odd", op="ortho", batch=5, m=333, n=1001, tokens=200, dtype="bf16", scale=0.2 * math.sqrt(1001)),
        # one gate projection of every expert of the 128-expert layer, fewer tokens than rows in many
        dict(name="ortho_experts", op="ortho", batch=128, m=768, n=2048, tokens=1024, dtype="f32", scale=1.0),
        # down projections of the large layer (tall)
        dict(name="ortho_tall", op="ortho", batch=3, m=7168, n=2048, tokens=2048, dtype="f32", scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "linear", "moe", "ortho"])
    if op == "balance":
        E = rng.choice([_log(rng, 2, 512), 8, 64, 128, 160, 256])
        return dict(op=op, T=_log(rng, 1, 65536 * 256 // max(E, 256)), E=E, k=rng.randint(1, min(E, 16)),
                    gate=rng.choice(GATES), seqs=rng.choice([1, 1, _log(rng, 1, 64)]), masked=rng.random() < 0.4,
                    bias=rng.random() < 0.4)
    if op == "linear":
        N, K = 8 * _log(rng, 4, 1024), 128 * _log(rng, 1, 64)
        return dict(op=op, rows=_log(rng, 1, min(65536, 16381 * 2048 * 7168 // (N * K))), N=N, K=K,
                    out=rng.choice(["bf16", "f32"]))
    if op == "moe":
        d, c, E = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16), _log(rng, 1, 64)
        k = rng.randint(1, min(E, 8))
        return dict(op=op, T=_log(rng, 1, 4096), d=d, c=c, E=E, k=k)
    m, n = _log(rng, 1, 4096), _log(rng, 1, 4096)
    lo, hi = min(m, n), max(m, n)
    top = max(1, min(64, int(2e11 / (2 * lo * lo * (2 * hi + lo)))))
    return dict(op=op, batch=_log(rng, 1, top), m=m, n=n, tokens=_log(rng, 1, 8192), dtype=rng.choice(["f32", "bf16"]),
                scale=rng.choice([1.0, 0.2 * math.sqrt(hi)]))


def work(case):
    op = case["op"]
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        # logits, indices (mask) in, the gradient, counts and mean scores out; exp, sums, products
        return {"bytes": T * (8 * E + 4 * k + case["masked"]) + 8 * S * E, "flops": 10 * T * E}
    if op == "linear":
        r, N, K = case["rows"], case["N"], case["K"]
        return {"bytes": r * K * 2 + N * K * 17 // 32 + r * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * r * N * K}
    if op == "moe":
        T, d, c, E, k = (case[x] for x in ("T", "d", "c", "E", "k"))
        used = min(E, T * k)                                         # experts that can have a token
        return {"bytes": 3 * used * d * c * 17 // 32 + T * (6 * d + 8 * k), "flops": 6 * T * k * d * c}
    b, lo, hi = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # per step the symmetric halves of X X^T and A A, and B X whole
    return {"bytes": b * lo * hi * (6 if case["dtype"] == "f32" else 4), "flops": 5 * b * (3 * lo * lo * hi + lo ** 3)}


# ----------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _cuts(case, seed):
    """Sequence borders: ragged, some of them empty, and a few rows behind the last where there are several."""
    T, S = case["T"], case["seqs"]
    if S == 1:
        return [0, T]
    r = random.Random(seed)
    end = T - r.randint(0, T // 50)
    return [0] + sorted(r.randint(0, end) for _ in range(S - 1)) + [end]


def _blocks4(x):
    """Rows -> 4-bit codes (uint8, one each) and scale bytes (one per 32): the smallest e with max <= 6 2^e."""
    b = x.float().unflatten(-1, (-1, 32))
    mant, ex = torch.frexp(b.abs().amax(-1))                          # max = mant 2^ex, mant in [0.5, 1)
    e = torch.where(mant == 0, 0, torch.where(mant <= 0.75, ex - 3, ex - 2)).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code | (torch.signbit(b).to(torch.uint8) << 3)).flatten(-2), (e + 127).to(torch.uint8)


def _chunks(sf):
    """Scale bytes [R, K / 32], R a multiple of 128 -> the order the tensor cores take: [R / 128, K / 128, 512]."""
    R, nb = sf.shape
    return sf.view(R // 128, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).reshape(R // 128, nb // 4, 512)


def _pack4(w):
    """One weight matrix [N, K] -> the library's packed codes and scale chunks, flat bytes each."""
    N, K = w.shape
    code, sf = _blocks4(w)
    N2, K2 = (N + 255) // 256 * 256, (K + 255) // 256 * 256
    c = torch.zeros((N2, K2), dtype=torch.uint8, device=DEV)
    c[:N, :K] = code
    s = torch.full((N2, K // 32), 127, dtype=torch.uint8, device=DEV)
    s[:N] = sf
    byte = c[:, 0::2] | (c[:, 1::2] << 4)
    return (byte.view(N2 // 256, 256, K2 // 256, 128).permute(0, 2, 1, 3).reshape(-1),
            _chunks(s).view(N2 // 256, 2, K // 128, 512).permute(0, 2, 1, 3).reshape(-1))


def _pack4_groups(g, G, N, K):
    """Random weights of G groups, std 1 / sqrt(K), quantised and packed: all codes, then all scale chunks."""
    codes, sfs = [], []
    for _ in range(G):
        w = torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)
        c, s = _pack4(w.to(torch.bfloat16))
        codes.append(c)
        sfs.append(s)
    return torch.cat(codes + sfs)


def _values(packed, G, N, K, dtype):
    """The values [G, N, K] that packed weights stand for."""
    NT, KT, KC = (N + 255) // 256, (K + 255) // 256, K // 128
    n = G * NT * KT * 256 * 128
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV, dtype=dtype)
    pair = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)                     # low nibble first
    c = packed[:n].view(G, NT, KT, 256, 128).permute(0, 1, 3, 2, 4).reshape(-1)
    v = pair.index_select(0, c.int()).view(G, NT * 256, KT * 256)[:, :N, :K]
    s = packed[n:].view(G, NT, KC, 2, 32, 4, 4).permute(0, 1, 3, 5, 4, 2, 6).reshape(G, NT * 256, K // 32)[:, :N]
    scale = torch.ldexp(torch.ones((), device=DEV, dtype=dtype), s.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": case}
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        # router logits with a few favoured experts, as an unbalanced layer has them
        z = torch.randn((T, E), generator=g, device=DEV) + 0.7 * torch.randn((1, E), generator=g, device=DEV)
        b = 0.3 * torch.randn((E,), generator=g, device=DEV) if case["bias"] else None
        idx = torch.topk(z if b is None else z + b, k, dim=1).indices.int()
        mask = (torch.rand((T,), generator=g, device=DEV) < 0.9).to(torch.uint8) if case["masked"] else None
        st.update(z=z, b=b, idx=idx, mask=mask, cu=torch.tensor(_cuts(case, seed), dtype=torch.int32, device=DEV),
                  g=1.0 + torch.rand((1,), generator=g, device=DEV), coef=0.01,
                  counts=torch.zeros((S, E), dtype=torch.int32, device=DEV),
                  tokens=torch.zeros((S,), dtype=torch.int32, device=DEV), probs=torch.zeros((S, E), device=DEV),
                  loss=torch.zeros((1,), device=DEV), dz=torch.zeros((T, E), device=DEV))
    elif op == "linear":
        r, N, K = case["rows"], case["N"], case["K"]
        x = torch.randn((r, K), generator=g, device=DEV) * torch.exp(0.5 * torch.randn((r, 1), generator=g, device=DEV))
        st.update(x=x.to(torch.bfloat16), w=_pack4_groups(g, 1, N, K),
                  y=torch.empty((r, N), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV))
    elif op == "moe":
        T, d, c, E, k = (case[x] for x in ("T", "d", "c", "E", "k"))
        z = torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn((1, E), generator=g, device=DEV)
        top = torch.topk(z, k, dim=1)
        st.update(u=torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16), idx=top.indices.int(),
                  tw=torch.softmax(top.values, 1), o_prev=(0.25 * torch.randn((T, d), generator=g, device=DEV)).to(torch.bfloat16),
                  w13=_pack4_groups(g, E, 2 * c, d), w3=_pack4_groups(g, E, d, c),
                  o=torch.empty((T, d), dtype=torch.bfloat16, device=DEV))
    else:
        b, m, n, R = case["batch"], case["m"], case["n"], case["tokens"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        grads = torch.empty((b, m, n), dtype=dt, device=DEV)
        for i in range(b):                     # a weight gradient is a sum of outer products; experts have 1, 1/2, 1/4, ... of the tokens
            r = max(1, R >> (i % 6))
            grads[i] = (torch.randn((m, r), generator=g, device=DEV) @ torch.randn((r, n), generator=g, device=DEV)) * (1e-3 / r)
        st.update(g=grads, out=torch.empty((b, m, n), dtype=torch.bfloat16, device=DEV))
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a program keeps across calls: descriptors, workspaces and the buffers between the steps."""
    from mixture_experts_layer_expert_gb300 import fs
    from mixture_experts_layer_expert_gb300.configs import LayerConfig
    case, op = st["case"], st["case"]["op"]
    empty = lambda n, dt=torch.uint8: torch.empty(n, dtype=dt, device=DEV)
    if op == "balance":
        st["desc"] = fs.make_balance(case["T"], case["E"], case["k"], case["gate"], case["seqs"], st["coef"])
        st["ws"] = empty(fs.fs_balance_ws_bytes(st["desc"]))
    elif op == "linear":
        st["q"] = fs.mx4_rows_empty(case["rows"], case["K"])
        st["ws"] = empty(fs.fs_linear_mx4_ws_bytes(case["rows"], case["N"], case["K"]))
    elif op == "moe":
        cfg = LayerConfig("routed", T=case["T"], d=case["d"], E=case["E"], k=case["k"], c=case["c"], n_shared=0, c_shared=0,
                          L=1, gate="softmax_renorm", dtype="mxfp4")
        st["desc"] = fs.make_desc(cfg)
        rows = fs.fs_dispatch_rows(st["desc"])
        st.update(ws=fs.alloc_workspace(st["desc"], 0), counts=empty(case["E"], torch.int32),
                  offsets=empty(case["E"] + 1, torch.int32), pos=empty(case["T"] * case["k"], torch.int32),
                  perm=empty(rows, torch.int32), xp=fs.mx4_rows_empty(rows, case["d"]),
                  yp=empty((rows, case["d"]), torch.bfloat16))
    else:
        st["desc"] = fs.make_orthogonalize(case["batch"], case["m"], case["n"], case["dtype"], scale=case["scale"],
                                           coefs=[COEFS] * 5, eps=EPS)
        st["ws"] = empty(fs.fs_orthogonalize_ws_bytes(st["desc"]))
    st["fs"] = fs


# ---------------------------------------------------------------- the operators

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    if "fs" not in st:
        _handles(st)
    fs, op = st["fs"], st["case"]["op"]
    if op == "balance":
        fs.fs_balance_loss(st["desc"], st["z"], st["idx"], st["counts"], st["tokens"], st["probs"], st["loss"], st["ws"],
                           bias=st["b"], cu=st["cu"], mask=st["mask"])
        fs.fs_balance_loss_backward(st["desc"], st["z"], st["counts"], st["tokens"], st["g"], st["dz"], bias=st["b"],
                                    cu=st["cu"], mask=st["mask"])
        return st["counts"], st["tokens"], st["probs"], st["loss"], st["dz"]
    if op == "linear":
        fs.fs_quantize_rows_mx4(st["x"].shape[0], st["x"].shape[1], st["x"], st["q"])
        fs.fs_linear_mx4(st["q"], st["w"], st["y"], st["case"]["K"], st["ws"])
        return st["y"]
    if op == "moe":
        fs.fs_dispatch(st["desc"], st["idx"], st["u"], st["counts"], st["offsets"], st["pos"], st["perm"], st["xp"], st["ws"])
        fs.fs_grouped_swiglu(st["desc"], st["xp"], st["offsets"], st["w13"], st["w3"], st["yp"], st["ws"])
        fs.fs_combine(st["desc"], st["yp"], st["pos"], st["tw"], st["o_prev"], None, None, st["o"])
        return st["o"]
    fs.fs_orthogonalize(st["desc"], st["g"], st["out"], st["ws"])
    return st["out"]


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "balance":
        return _plain_balance(st)
    if op == "linear":
        y = _round4(st["x"]) @ _values(st["w"], 1, case["N"], case["K"], torch.float32)[0].T
        return y.to(st["y"].dtype)
    if op == "moe":
        return _plain_moe(st)
    return _plain_ortho(st["g"], case["scale"])


def _scores(z, gate):
    if gate.startswith("softmax"):
        e = torch.exp(z - z.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), None
    p = 1 / (1 + torch.exp(-z))
    return p / p.sum(1, keepdim=True), 1 - p


def _plain_balance(st):
    case, cu = st["case"], st["cu"]
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    t = torch.arange(T, device=DEV)
    member = (t >= cu[:-1, None]) & (t < cu[1:, None])                                     # [S, T]
    if st["mask"] is not None:
        member = member & (st["mask"] != 0)
    member = member.float()
    s, rest = _scores(st["z"] if st["b"] is None else st["z"] + st["b"], case["gate"])
    chosen = torch.zeros((T, E), device=DEV).scatter_add_(1, st["idx"].long(), torch.ones((T, k), device=DEV))
    n, counts = member.sum(1), member @ chosen
    probs = (member @ s) / n.clamp(min=1)[:, None]
    f = counts * E / (k * n.clamp(min=1)[:, None])
    loss = st["coef"] / S * (f * probs).sum()
    weight = st["g"] * st["coef"] / (S * n.clamp(min=1))
    ft = member.T @ f
    dz = (member.T @ weight)[:, None] * s * (ft - (ft * s).sum(1, keepdim=True))
    if rest is not None:
        dz = dz * rest
    return counts.int(), n.int(), probs, loss[None], dz


def _round4(x):
    """The values that x's 4-bit blocks stand for, in 32 bits."""
    code, sf = _blocks4(x)
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    v = lut[(code & 7).int()] * (1 - 2 * (code >> 3).float())
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (sf.int() - 127)[..., None]).flatten(-2)


def _plain_moe(st):
    case = st["case"]
    T, d, c, E, k = (case[x] for x in ("T", "d", "c", "E", "k"))
    flat = st["idx"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    counts = (flat[None, :] == torch.arange(E, device=DEV)[:, None]).sum(1)
    start = torch.cumsum(counts, 0) - counts
    e = flat[order]
    slot = torch.arange(T * k, device=DEV) - start[e]                                      # place within its expert
    x = torch.zeros((E, int(counts.max()), d), device=DEV)
    x[e, slot] = _round4(st["u"])[order // k]
    gu = torch.bmm(x, _values(st["w13"], E, 2 * c, d, torch.float32).transpose(1, 2))
    gu = gu.unflatten(-1, (c // 64, 2, 64))                                                # 64 gate columns, 64 up columns, ...
    gate, up = gu[..., 0, :].flatten(-2), gu[..., 1, :].flatten(-2)
    h = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)                            # the hidden is stored in bf16's values
    y = torch.bmm(_round4(h), _values(st["w3"], E, d, c, torch.float32).transpose(1, 2)).to(torch.bfloat16)
    back = torch.empty((T * k, d), dtype=torch.bfloat16, device=DEV)
    back[order] = y[e, slot]
    r = (back.view(T, k, d).float() * st["tw"][..., None]).sum(1)
    return (st["o_prev"].float() + r).to(torch.bfloat16)


def _plain_ortho(g, scale):
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(5):
        a = x @ x.transpose(1, 2)
        x = COEFS[0] * x + (COEFS[1] * a + COEFS[2] * (a @ a)) @ x
    return ((x.transpose(1, 2) if tall else x) * scale).to(torch.bfloat16)


# ------------------------------------------------------------------ in 64 bits

def _nearest4(x):
    """Each block of 32 on the 4-bit grid, by distance (the even code of a tie), in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 6))
    e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e))
    s = torch.exp2(torch.where(top == 0, torch.zeros_like(e), e).clamp(-127, 127))
    grid = torch.tensor([0, 1, 2, 4, 6, 0.5, 1.5, 3], dtype=torch.float64, device=DEV)     # even codes first: a tie takes the first
    a, best, dist = (b / s).abs(), torch.zeros_like(b), torch.full_like(b, math.inf)
    for v in grid:
        d = (a - v).abs()
        best, dist = torch.where(d < dist, v, best), torch.minimum(d, dist)
    return (torch.copysign(best, b) * s).flatten(-2)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "balance":
        return _exact_balance(st)
    if op == "linear":
        w = _values(st["w"], 1, case["N"], case["K"], torch.float64)[0]
        return torch.cat([_nearest4(x) @ w.T for x in st["x"].split(4096)])
    if op == "moe":
        return _exact_moe(st)
    outs = []
    for m in st["g"]:
        x = m.double()
        x = x.T if x.shape[0] > x.shape[1] else x
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(5):
            a = x @ x.T
            x = torch.addmm(x, torch.addmm(a, a, a, beta=COEFS[1], alpha=COEFS[2]), x, beta=COEFS[0])
        outs.append((x.T if m.shape[0] > m.shape[1] else x) * case["scale"])
    return torch.stack(outs)


def _exact_balance(st):
    """Sequence by sequence, the gradient from the softmax's (or normalised sigmoid's) own derivative."""
    case, cu = st["case"], st["cu"].tolist()
    E, k, S = case["E"], case["k"], case["seqs"]
    z = st["z"].double() + (0 if st["b"] is None else st["b"].double())
    counts, tokens = torch.zeros((S, E), dtype=torch.int32, device=DEV), torch.zeros((S,), dtype=torch.int32, device=DEV)
    probs, dz = torch.zeros((S, E), dtype=torch.float64, device=DEV), torch.zeros_like(z)
    loss = torch.zeros((1,), dtype=torch.float64, device=DEV)
    for q in range(S):
        rows = torch.arange(cu[q], cu[q + 1], device=DEV)
        if st["mask"] is not None:
            rows = rows[st["mask"][rows] != 0]
        n = len(rows)
        tokens[q] = n
        if n == 0:
            continue
        counts[q] = torch.bincount(st["idx"][rows].flatten().long(), minlength=E).int()
        leaf = z[rows].requires_grad_()
        s = torch.softmax(leaf, 1) if case["gate"].startswith("softmax") else torch.sigmoid(leaf) / torch.sigmoid(leaf).sum(1, keepdim=True)
        p = s.mean(0)
        part = st["coef"] / S * (counts[q].double() * E / (k * n) * p).sum()
        part.backward()
        probs[q], dz[rows] = p.detach(), leaf.grad * st["g"].double()
        loss += part.detach()
    return counts, tokens, probs, loss, dz


def _exact_moe(st):
    case = st["case"]
    T, d, c, E, k = (case[x] for x in ("T", "d", "c", "E", "k"))
    x, r = _nearest4(st["u"]), torch.zeros((T, d), dtype=torch.float64, device=DEV)
    n13, n3 = st["w13"].numel() // E, st["w3"].numel() // E
    c13, c3 = (2 * c + 255) // 256 * ((d + 255) // 256) * 32768, (d + 255) // 256 * ((c + 255) // 256) * 32768
    for e in range(E):
        t, slot = torch.nonzero(st["idx"] == e, as_tuple=True)
        if len(t) == 0:
            continue
        def one(p, n, codes, rows, cols):                          # expert e's codes and scale chunks
            s = E * codes + e * (n - codes)
            return _values(torch.cat([p[e * codes:(e + 1) * codes], p[s:s + n - codes]]), 1, rows, cols, torch.float64)[0]
        gu = (x[t] @ one(st["w13"], n13, c13, 2 * c, d).T).unflatten(-1, (c // 64, 2, 64))
        gate, up = gu[..., 0, :].flatten(-2), gu[..., 1, :].flatten(-2)
        h = _nearest4((gate * torch.sigmoid(gate) * up).to(torch.bfloat16))
        y = (h @ one(st["w3"], n3, c3, d, c).T).to(torch.bfloat16).double()
        r.index_add_(0, t, y * st["tw"][t, slot].double()[:, None])
    return st["o_prev"].double() + r
