"""The 4-bit microscaled path (FS_MXFP4) against its 64-bit definition: codes and
scales bit for bit (quantised rows, packs, Dispatch), the dense product, the
routed and shared experts with the allowance for a hidden value on a rounding
border, and the stacks, which run the same steps, bit for bit."""
import math

import pytest
import torch

import mx4_ref as ref
from mixture_experts_layer_expert_gb300 import configs, fs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def no_error():
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)


def unpack(code_bytes):
    """[R, K / 2] bytes -> [R, K] codes."""
    c = code_bytes.cpu().long()
    return torch.stack([c & 15, c >> 4], -1).flatten(-2)


def scale_exps(chunks, rows, K):
    """[R / 128, K / 128, 512] -> [rows, K / 32] exponents."""
    c = chunks.cpu().long()
    r, b = torch.arange(rows)[:, None], torch.arange(K // 32)[None, :]
    return c[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] - 127


def matrix(q, rows, K):
    codes, chunks = fs.mx4_rows_split(q, rows, K)
    return unpack(codes)[:rows], scale_exps(chunks, rows, K)


def hard_rows(rows, K, seed):
    """bf16 rows over its whole range: ties, zeros, subnormals, largest values, signed zeros, one big value a block."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    x[0] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * (K // 8))
    if rows > 3:
        x[1] = 0.0
        x[1, ::2] = -0.0
        x[2] = torch.randn(K, generator=g) * 2.0 ** -130
        x[3] = torch.randn(K, generator=g).sign() * 3.38e38
        x[3, ::3] = 1e30
    if rows > 6:
        x[4, ::32] = 6.03125 * 4                         # a block's largest just above 6 2^e
        x[5, ::32] = 6.0 * 4
        x[6, 1:] = 0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("rows,K", [(1, 128), (7, 256), (128, 384), (129, 1408), (300, 2048), (1000, 128)])
def test_quantised_rows(rows, K):
    x = hard_rows(rows, K, rows + K)
    q = torch.full((fs.fs_mx4_rows_bytes(rows, K),), 0xAA, dtype=torch.uint8, device=DEV)
    fs.fs_quantize_rows_mx4(rows, K, x.to(DEV), q)
    no_error()
    codes, e = matrix(q, rows, K)
    want, we = ref.quantise(x)
    assert torch.equal(e, we)
    assert torch.equal(codes, want)
    tail, chunks = fs.mx4_rows_split(q, rows, K)
    r128 = tail.shape[0]
    assert not tail[rows:].any() and torch.equal(scale_exps(chunks, r128, K)[rows:], torch.zeros((r128 - rows, K // 32)).long())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_without_a_number_is_nan(bad):
    """Its scale is NaN, its row's products are NaN, other rows are what they were; so with a weight's column."""
    g = torch.Generator().manual_seed(3)
    rows, N, K = 130, 264, 256
    x, w = torch.randn((rows, K), generator=g).to(torch.bfloat16), torch.randn((N, K), generator=g).to(torch.bfloat16)
    clean, _ = linear(x, w, torch.float32)
    x2 = x.clone()
    x2[77, 40] = bad
    y, q = linear(x2, w, torch.float32)
    assert scale_exps(fs.mx4_rows_split(q, rows, K)[1], rows, K)[77, 1] == 128
    assert y[77].isnan().all()
    keep = torch.arange(rows) != 77
    assert torch.equal(y[keep], clean[keep])
    w2 = w.clone()
    w2[259, 255] = bad
    y, _ = linear(x, w2, torch.float32)
    assert y[:, 259].isnan().all()
    keep = torch.arange(N) != 259
    assert torch.equal(y[:, keep], clean[:, keep])


def linear(x, w, dtype, pad=0, stream=None):
    (rows, K), N = x.shape, w.shape[0]
    q = fs.mx4_rows_empty(rows, K)
    fs.fs_quantize_rows_mx4(rows, K, x.to(DEV), q)
    wp = fs.pack_linear_mx4(w.to(DEV))
    full = torch.full((rows, N + pad), 7.0, dtype=dtype, device=DEV)
    y = full[:, :N]
    ws = torch.empty(fs.fs_linear_mx4_ws_bytes(rows, N, K), dtype=torch.uint8, device=DEV)
    fs.fs_linear_mx4(q, wp, y, K, ws)
    no_error()
    assert (full[:, N:] == 7.0).all()
    return y.cpu(), q


SIZES = [(1, 8, 128), (1, 7168, 2048), (3, 264, 384), (17, 2048, 1408), (64, 1000, 7168), (127, 256, 256), (128, 40, 640),
         (129, 2112, 512), (300, 1032, 2048), (1025, 328, 128), (5, 16384, 256), (2, 512, 16384), (511, 64, 256), (512, 64, 256),
         (600, 264, 384), (641, 520, 1408), (1500, 72, 7168), (770, 3008, 640)]


@pytest.mark.parametrize("rows,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(rows, N, K, dtype):
    g = torch.Generator().manual_seed(rows + N + K)
    x = (torch.randn((rows, K), generator=g) * torch.exp(torch.randn((rows, 1), generator=g))).to(torch.bfloat16)
    w = (torch.randn((N, K), generator=g) / math.sqrt(K)).to(torch.bfloat16)
    y, _ = linear(x, w, dtype, pad=8 * (N % 3))
    a, b = ref.rounded(x).to(DEV), ref.rounded(w).to(DEV)
    want, room = (a @ b.T).cpu(), (a.abs() @ b.abs().T).cpu() * K * 2.0 ** -23
    if dtype is torch.bfloat16:
        room = room + (want.abs() + room) * ref.BF16_HALF
    off = (y.double() - want).abs()
    assert (off <= room).all(), "%.3e over its bound" % float((off - room).max())


def test_linear_identity_returns_the_quantised_rows():
    """With the unit matrix as weight (exact in 4 bits) the product is the value of each code."""
    rows, K = 70, 512
    x = torch.randn((rows, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    y, _ = linear(x, torch.eye(K).to(torch.bfloat16), torch.float32)
    assert torch.equal(y.double(), ref.rounded(x))


def test_linear_of_scales_at_both_ends():
    """Blocks whose scales differ by 2^200 inside a row, and tiny times huge."""
    g = torch.Generator().manual_seed(5)
    rows, N, K = 33, 72, 384
    ex = torch.randint(-100, 100, (rows, K // 32, 1), generator=g).float()
    x = (torch.randn((rows, K // 32, 32), generator=g) * torch.exp2(ex)).flatten(1).to(torch.bfloat16)
    w = (torch.randn((N, K // 32, 32), generator=g) * torch.exp2(-ex[:1] / 2)).flatten(1).to(torch.bfloat16)
    y, _ = linear(x, w, torch.float32)
    a, b = ref.rounded(x), ref.rounded(w)
    want, mass = a @ b.T, a.abs() @ b.abs().T
    top = torch.finfo(torch.float32).max
    # rows whose scales sum to more than 2^127 pass fp32's largest number: infinite, or NaN where partial sums of both
    # signs pass it
    fits = mass < top
    assert fits.any() and ((y.double() - want).abs() <= mass * K * 2.0 ** -23)[fits].all()
    over = want.abs() > top + mass * K * 2.0 ** -23
    assert over.any() and not y[over].isfinite().any()


def layer(**kw):
    base = dict(name="mx4", T=300, d=256, E=8, k=2, c=256, n_shared=1, c_shared=128, L=1, gate="softmax_renorm",
                dtype="mxfp4")
    base.update(kw)
    return configs.LayerConfig(**base)


def weights(buf, G, N, K):
    """Codes [G, N, K] and exponents of a pack."""
    NB, KB = (N + 255) // 256, (K + 255) // 256
    n = G * NB * KB * 32768
    c = buf[:n].view(G, NB, KB, 256, 128).permute(0, 1, 3, 2, 4).reshape(G * NB * 256, KB * 128)
    s = buf[n:].view(G, NB, K // 128, 2, 512).permute(0, 1, 3, 2, 4).reshape(G * NB * 2, K // 128, 512)
    codes = unpack(c).view(G, NB * 256, KB * 256)
    return codes, scale_exps(s, G * NB * 256, K).view(G, NB * 256, K // 32)


@pytest.mark.parametrize("kw", [dict(E=3, c=384, d=640), dict(E=2, c=128, d=128, n_shared=3, c_shared=128)])
def test_packs(kw):
    cfg = layer(**kw)
    w = synth.make_block_weights(cfg, 0)
    p = fs.pack_block(cfg, {k: v.to(DEV) if v is not None else None for k, v in w.items()})
    E, c, d, cw = cfg.E, cfg.c, cfg.d, cfg.n_shared * cfg.c_shared

    def interleave(up, gate):                              # [G, c, d] each -> [G, 2c, d]
        return torch.stack([gate.unflatten(1, (-1, 64)), up.unflatten(1, (-1, 64))], 2).flatten(1, 3)
    shared3 = w["w3s"].permute(1, 0, 2).reshape(1, d, cw)
    for buf, rows in ((p["w13"], interleave(w["w1"], w["w2"])), (p["w3"], w["w3"]),
                      (p["w13_shared"], interleave(w["w1s"].reshape(1, cw, d), w["w2s"].reshape(1, cw, d))),
                      (p["w3_shared"], shared3)):
        G, N, K = rows.shape
        codes, e = weights(buf, G, N, K)
        want, we = ref.quantise(rows)
        assert torch.equal(codes[:, :N, :K], want) and torch.equal(e[:, :N], we)
        assert not codes[:, N:].any() and not codes[:, :, K:].any() and not e[:, N:].any()


def route(cfg, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((cfg.T, cfg.E), generator=g) + skew * torch.randn((1, cfg.E), generator=g)
    top = torch.topk(z, cfg.k, dim=1)
    return top.indices.int(), torch.softmax(top.values, 1)


def dispatch(cfg, desc, idx, u, ws):
    rows = fs.fs_dispatch_rows(desc)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    counts, offsets, pos, perm = i32(cfg.E), i32(cfg.E + 1), i32(cfg.T * cfg.k), i32(rows)
    xp = fs.mx4_rows_empty(rows, cfg.d)
    fs.fs_dispatch(desc, idx, u, counts, offsets, pos, perm, xp, ws)
    return counts, offsets, pos, perm, xp


LAYERS = [dict(), dict(T=1, k=1, E=1), dict(T=61, E=64, k=6, c=128), dict(T=300, d=384, c=640), dict(T=513, E=4, k=4, c=128),
          dict(T=130, E=16, k=8, d=128, c=384), dict(T=700, E=2, k=2, d=384, c=640), dict(T=1100, E=3, k=2, d=128, c=128),
          dict(T=640, E=1, k=1, d=640, c=384)]


@pytest.mark.parametrize("kw", LAYERS)
def test_dispatch_and_routed_experts(kw):
    cfg = layer(**kw)
    desc, ws = fs.make_desc(cfg), None
    ws = fs.alloc_workspace(desc, 0)
    w = synth.make_block_weights(cfg, 0)
    p = fs.pack_block(cfg, {k: v.to(DEV) if v is not None else None for k, v in w.items()})
    u = synth.make_x(cfg)
    idx, tw = route(cfg, 7, skew=1.0)
    counts, offsets, pos, perm, xp = dispatch(cfg, desc, idx.to(DEV), u.to(DEV), ws)
    rows = fs.fs_dispatch_rows(desc)
    yp = torch.empty((rows, cfg.d), dtype=torch.bfloat16, device=DEV)
    fs.fs_grouped_swiglu(desc, xp, offsets, p["w13"], p["w3"], yp, ws)
    no_error()
    want_counts = torch.bincount(idx.flatten().long(), minlength=cfg.E)
    assert torch.equal(counts.cpu().long(), want_counts)
    assert torch.equal(offsets.cpu().long()[1:], torch.cumsum((want_counts + 127) // 128 * 128, 0))
    codes, e = matrix(xp, rows, cfg.d)
    uc, ue = ref.quantise(u)
    at = pos.cpu().long().view(cfg.T, cfg.k)
    assert torch.equal(codes[at], uc[:, None].expand(-1, cfg.k, -1)) and torch.equal(e[at], ue[:, None].expand(-1, cfg.k, -1))
    uq = ref.value(uc, ue)
    for x in range(cfg.E):
        t, s = torch.nonzero(idx == x, as_tuple=True)
        if len(t) == 0:
            continue
        y, room = ref.expert(uq[t], w["w1"][x], w["w2"][x], w["w3"][x])
        off = (yp.cpu().double()[at[t, s]] - y).abs()
        room = room + (y.abs() + room) * ref.BF16_HALF
        assert (off <= room).all(), "expert %d: %.3e over its bound" % (x, float((off - room).max()))
        assert float(room.norm()) < 0.1 * float(y.norm()) * math.sqrt(cfg.c)     # the allowance stays small


@pytest.mark.parametrize("T", [200, 700])
def test_shared_expert(T):
    cfg = layer(T=T, n_shared=2, c_shared=128, d=384)
    desc = fs.make_desc(cfg)
    ws = fs.alloc_workspace(desc, 0)
    w = synth.make_block_weights(cfg, 0)
    p = fs.pack_block(cfg, {k: v.to(DEV) if v is not None else None for k, v in w.items()})
    u = synth.make_x(cfg)
    s = torch.empty((cfg.T, cfg.d), dtype=torch.float32, device=DEV)
    fs.fs_shared_expert(desc, u.to(DEV), p["w13_shared"], p["w3_shared"], s, ws)
    no_error()
    cw = cfg.n_shared * cfg.c_shared
    y, room = ref.expert(ref.rounded(u), w["w1s"].reshape(cw, -1), w["w2s"].reshape(cw, -1),
                         w["w3s"].permute(1, 0, 2).reshape(cfg.d, cw))
    assert ((s.cpu().double() - y).abs() <= room).all()


@pytest.mark.parametrize("wiring", ["partial", "outdated", "disabled"])
def test_stack_runs_the_single_steps(wiring):
    """Two blocks of fs_farskip_stack, the two-stream form and its graph, and the steps one by one, bit for bit."""
    cfg = layer(T=260, L=2, wiring=wiring, E=6, k=3)
    prob = synth.make_problem(cfg, device=DEV)
    stack = fs.FarSkipStack(cfg, prob["blocks"])
    o, star = (t.clone() for t in stack.forward(prob["x"]))
    desc, ws = stack.desc, fs.alloc_workspace(stack.desc, 0)
    u = o_prev = prob["x"]
    for b, bw in enumerate(stack.blocks):
        last = b == cfg.L - 1
        idx = torch.empty((cfg.T, cfg.k), dtype=torch.int32, device=DEV)
        tw = torch.empty((cfg.T, cfg.k), device=DEV)
        fs.fs_router_topk(desc, u, bw["w_r"], bw["bias"], idx, tw, None, ws)
        _, offsets, pos, _, xp = dispatch(cfg, desc, idx, u, ws)
        yp = torch.empty((fs.fs_dispatch_rows(desc), cfg.d), dtype=torch.bfloat16, device=DEV)
        fs.fs_grouped_swiglu(desc, xp, offsets, bw["w13"], bw["w3"], yp, ws)
        s = torch.empty((cfg.T, cfg.d), device=DEV)
        fs.fs_shared_expert(desc, u, bw["w13_shared"], bw["w3_shared"], s, ws)
        dt = torch.bfloat16 if last else torch.float32
        part, full = (torch.empty((cfg.T, cfg.d), dtype=dt, device=DEV) for _ in range(2))
        nxt = None if last else torch.empty((cfg.T, cfg.d), dtype=torch.bfloat16, device=DEV)
        fs.fs_combine(desc, yp, pos, tw, o_prev, s, part, full, nxt, wiring)
        u, o_prev = nxt, full
    no_error()
    assert torch.equal(o, full) and torch.equal(star, part)
    if wiring != "disabled":
        o2, _ = stack.forward_overlap(prob["x"])
        no_error()
        assert torch.equal(o, o2)
    o.zero_()
    want = full.clone()
    stack.capture(prob["x"])
    stack.o_full.zero_()
    stack.replay()
    no_error()
    assert torch.equal(stack.o_full, want)


def test_attention_wiring_runs():
    cfg = layer(T=128, wiring="attn_farskip", L=2)
    prob = synth.make_problem(cfg, device=DEV)
    blocks = [dict(b, w_att=(torch.randn((cfg.d, cfg.d), device=DEV) / math.sqrt(cfg.d)).to(torch.bfloat16))
              for b in prob["blocks"]]
    stack = fs.FarSkipStack(cfg, blocks, wiring="attn_farskip")
    o, _ = stack.forward(prob["x"])
    no_error()
    assert o.isfinite().all()


def test_dispatch_without_workspace_and_repeats():
    cfg = layer(T=300)
    desc = fs.make_desc(cfg)
    ws = fs.alloc_workspace(desc, 0)
    idx, _ = route(cfg, 3)
    u = synth.make_x(cfg).to(DEV)
    _, offsets, pos, _, xp = dispatch(cfg, desc, idx.to(DEV), u, ws)
    rows = fs.fs_dispatch_rows(desc)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    c2, o2, p2, s2, x2 = i32(cfg.E), i32(cfg.E + 1), i32(cfg.T * cfg.k), i32(rows), fs.mx4_rows_empty(rows, cfg.d)
    fs.fs_dispatch_noalloc(desc, idx.to(DEV), u, c2, o2, p2, s2, x2)
    no_error()
    assert torch.equal(offsets, o2) and torch.equal(pos, p2)
    at = pos.cpu().long()
    for a, b in zip(matrix(xp, rows, cfg.d), matrix(x2, rows, cfg.d)):
        assert torch.equal(a[at], b[at])


def test_linear_on_another_stream_and_replayed():
    g = torch.Generator().manual_seed(9)
    rows, N, K = 200, 512, 1024
    x = torch.randn((rows, K), generator=g).to(torch.bfloat16)
    w = torch.randn((N, K), generator=g).to(torch.bfloat16)
    want, _ = linear(x, w, torch.bfloat16)
    xd, wp, q = x.to(DEV), fs.pack_linear_mx4(w.to(DEV)), fs.mx4_rows_empty(rows, K)
    ws = torch.empty(fs.fs_linear_mx4_ws_bytes(rows, N, K), dtype=torch.uint8, device=DEV)
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fs.fs_quantize_rows_mx4(rows, K, xd, q, stream=side)
    fs.fs_linear_mx4(q, wp, y, K, ws, stream=side)
    side.synchronize()
    assert torch.equal(y.cpu(), want)
    y.zero_()
    q.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fs_quantize_rows_mx4(rows, K, xd, q)
        fs.fs_linear_mx4(q, wp, y, K, ws)
    for _ in range(2):
        y.zero_()
        graph.replay()
        no_error()
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("T", [60, 1200])
def test_inconsistent_offsets_are_reported(T):
    """Offsets that decrease, are negative or pass the rows: code 2, no rows written (both GEMM forms)."""
    cfg = layer(T=T, E=4, k=2)
    desc = fs.make_desc(cfg)
    ws = fs.alloc_workspace(desc, 0)
    w = synth.make_block_weights(cfg, 0)
    p = fs.pack_block(cfg, {k: v.to(DEV) if v is not None else None for k, v in w.items()})
    idx, _ = route(cfg, 1)
    _, offsets, _, _, xp = dispatch(cfg, desc, idx.to(DEV), synth.make_x(cfg).to(DEV), ws)
    rows = fs.fs_dispatch_rows(desc)
    no_error()
    for at, value in ((2, -128), (1, rows + 128), (3, 0), (4, 2 ** 31 - 1)):
        bad = offsets.clone()
        bad[at] = value
        yp = torch.full((rows, cfg.d), 3.0, dtype=torch.bfloat16, device=DEV)
        fs.fs_grouped_swiglu(desc, xp, bad, p["w13"], p["w3"], yp, ws)
        torch.cuda.synchronize()
        assert fs.fs_get_error() == (5, 2)
        assert (yp == 3.0).all()
