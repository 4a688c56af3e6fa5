"""Orthogonalised updates against the exact Newton-Schulz steps, with tolerances
from the documented roundings (ortho_ref)."""
import math

import pytest
import torch

import ortho_ref as ref
from mixture_experts_layer_expert_gb300 import configs, fs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def no_error():
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)


def run(g, scale=1.0, coefs=ref.USUAL, eps=1e-7, out=None, stream=None):
    b, m, n = g.shape
    desc = fs.make_orthogonalize(b, m, n, "f32" if g.dtype == torch.float32 else "bf16", scale, coefs, eps)
    ws = torch.full((fs.fs_orthogonalize_ws_bytes(desc),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((b, m, n), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    fs.fs_orthogonalize(desc, g, out, ws, stream)
    no_error()
    return out


def check(out, g, **kw):
    for o, x in zip(out, g):
        want, room = ref.tolerance(x.to(DEV), **kw)
        off = float((o.double() - want).norm())
        assert off <= room + 1e-30, "%.2e off, %.2e allowed (norm %.2e)" % (off, room, float(want.norm()))
        # roundings average out over many elements only: of one element bf16's alone may be 2^-8 = 0.39%
        if kw.get("coefs", ref.USUAL) == ref.USUAL and min(x.shape) >= 32:
            assert off <= 3e-3 * float(want.norm())


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 5, 1), (4, 8, 128), (1, 64, 2048), (2, 63, 65), (3, 127, 129), (2, 128, 128), (5, 333, 1001),
          (2, 257, 300), (8, 256, 128), (2, 1000, 64), (3, 512, 512), (1, 700, 2500), (2, 2049, 130), (1, 1408, 2048), (17, 40, 24)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rank", ["full", "few"])
def test_against_exact(shape, dtype, rank):
    b, m, n = shape
    r = min(m, n)
    g = torch.stack([ref.gradient(m, n, 2 * r if rank == "full" else max(1, r // (4 + i)), i + m + n) for i in range(b)])
    g = g.to(dtype).to(DEV)
    check(run(g, scale=0.2 * math.sqrt(max(m, n))), g, scale=0.2 * math.sqrt(max(m, n)))


def test_decaying_singular_values():
    """Singular values over six decades."""
    gen = torch.Generator().manual_seed(0)
    u = torch.linalg.qr(torch.randn((300, 300), generator=gen))[0]
    v = torch.linalg.qr(torch.randn((400, 300), generator=gen))[0]
    g = ((u * torch.logspace(0, -6, 300)) @ v.T)[None].to(DEV)
    check(run(g), g)


@pytest.mark.parametrize("coefs", [[(1.5, -0.5, 0.0)], [(1.875, -1.25, 0.375)] * 8, [(4.0, -6.0, 2.5), (3.0, -3.5, 1.2), (1.5, -0.5, 0.0)],
                                   [(0.5, 0.0, 0.0)] * 16, [(2.0, 0.0, 0.0)] * 3])
def test_other_coefficients(coefs):
    g = torch.stack([ref.gradient(96, 200, 300, 1), ref.gradient(96, 200, 10, 2)]).to(DEV)
    check(run(g, coefs=coefs), g, coefs=coefs)


def test_orthogonal_after_converging_steps():
    """Steps that converge to 1 leave nearly orthonormal rows: within 1% of the unit matrix (fp16's 2^-11 twice, times the rows)."""
    g = torch.linalg.qr(torch.randn((256, 128), generator=torch.Generator().manual_seed(3)))[0].T.contiguous()[None].to(DEV)
    out = run(g, coefs=[(1.875, -1.25, 0.375)] * 12)[0].double()
    assert float((out @ out.T - torch.eye(128, device=DEV)).abs().max()) < 1e-2


@pytest.mark.parametrize("power", [-140, -100, -60, 0, 60, 110])
def test_norm_over_the_whole_range(power):
    """The result does not depend on the gradient's scale, from subnormal numbers to the largest (eps 0)."""
    g = ref.gradient(40, 70, 60, 4)
    g = g / g.abs().max()
    big = torch.ldexp(g.double(), torch.tensor(power)).float()           # subnormal below 2^-126: rounded to 2^-149
    check(run(big[None].to(DEV), eps=0.0), big[None], eps=0.0)


def test_zero_matrices_and_eps():
    g = torch.zeros((3, 50, 80), device=DEV)
    g[1] = ref.gradient(50, 80, 50, 5).to(DEV)
    for eps in (0.0, 1e-7):
        out = run(g, eps=eps)
        assert not out[0].any() and not out[2].any()
        check(out[1:2], g[1:2], eps=eps)
    check(run(g[1:2], eps=0.5), g[1:2], eps=0.5)                           # eps as large as the norm counts


def test_nan_and_infinity_stay_in_their_matrix():
    g = torch.stack([ref.gradient(100, 60, 60, i) for i in range(4)]).to(DEV)
    clean = run(g)
    g[1, 99, 59] = math.nan
    g[2, 0, 0] = math.inf
    out = run(g)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert out[1].isnan().all() and out[2].isnan().all()


@pytest.mark.parametrize("m,n", [(65, 130), (200, 90)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_offsets(m, n, dtype):
    """Views with odd strides and offsets, in and out; what lies between is left."""
    b = 3
    g = torch.stack([ref.gradient(m, n, 30, i) for i in range(b)]).to(dtype).to(DEV)
    want = run(g)
    for pad_r, pad_m, off in ((1, 3, 1), (8, 0, 8), (6, 2, 4)):
        def view(fill, dt):
            base = torch.full((off + b * ((m + pad_m) * (n + pad_r)),), fill, dtype=dt, device=DEV)
            return base, base[off:].view(b, m + pad_m, n + pad_r)[:, :m, :n]
        gb, gv = view(math.nan, dtype)
        gv.copy_(g)
        ob, ov = view(5.0, torch.bfloat16)
        run(gv, out=ov)
        assert torch.equal(ov, want)
        ov.fill_(5.0)
        assert (ob == 5.0).all()


def test_batches_in_groups_match_single_matrices():
    """More matrices than the workspace holds at once: each as by itself."""
    desc = fs.make_orthogonalize(90, 1024, 2048, "bf16")
    assert fs.fs_orthogonalize_ws_bytes(desc) <= 2 ** 31 + 2 ** 20
    gen = torch.Generator(device=DEV).manual_seed(1)
    g = torch.randn((300, 1024, 1024), generator=gen, device=DEV).to(torch.bfloat16)
    out = run(g)
    for i in (0, 150, 299):
        assert torch.equal(run(g[i:i + 1])[0], out[i])
    check(out[299:], g[299:])


def test_repeats_replays_and_streams():
    g = torch.stack([ref.gradient(150, 300, 40, i) for i in range(3)]).to(DEV)
    want = run(g)
    assert torch.equal(run(g), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(run(g, stream=side), want)
    desc = fs.make_orthogonalize(3, 150, 300)
    ws = torch.empty(fs.fs_orthogonalize_ws_bytes(desc), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fs_orthogonalize(desc, g, out, ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        no_error()
        assert torch.equal(out, want)


def test_trainers_updates():
    """A training step's expert and router gradients through FarSkipTrainer.orthogonalized; an expert without tokens
    has a zero gradient and gets a zero update."""
    cfg = configs.LayerConfig("ortho", T=200, d=256, E=6, k=2, c=128, n_shared=1, c_shared=128, L=2, gate="softmax", dtype="bf16")
    prob = synth.make_problem(cfg, device=DEV)
    for b in prob["blocks"]:
        b["bias"] = torch.zeros(cfg.E, device=DEV)
        b["bias"][4] = -1e4                                                # nobody's expert
    tr = fs.FarSkipTrainer(cfg, prob["blocks"])
    tr.forward(prob["x"])
    tr.backward(torch.randn((cfg.T, cfg.d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    upd = tr.orthogonalized(("dW1", "dW2", "dW3", "dW1s", "dW_R"))
    no_error()
    for blk in range(cfg.L):
        for name, u in upd[blk].items():
            g = tr.grads[blk][name]
            assert u.shape == g.shape
            check(u if g.dim() == 3 else u[None], g if g.dim() == 3 else g[None])
        assert not upd[blk]["dW1"][4].any() and upd[blk]["dW1"][0].any()


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 1, 2), (2, 1, 300), (2, 2, 2), (5, 3, 257), (2, 4000, 1), (1, 16, 16), (160, 16, 40),
                                   (2, 513, 16), (20, 11, 2000), (1, 7, 8192), (1, 4097, 16)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_rows(shape, dtype):
    """Up to 16 rows nothing is rounded below fp32.  A step's sums (at most 16 x 2 + 13 + 16 + 17 terms) and products are
    within 2^-24 each of their size, 80 x 2^-24 of the norm, and later steps multiply by at most 3.4445 each:
    (3.4445^5 - 1) / 2.4445 x 80 x 2^-24 = 9.5e-4 of the norm at worst, beside half a step of bf16 for each element."""
    b, m, n = shape
    g = torch.stack([ref.gradient(m, n, min(m, n) + i, 3 * i + m + n) for i in range(b)]).to(dtype).to(DEV)
    out = run(g, scale=0.3)
    for o, x in zip(out, g):
        want = ref.exact(x, scale=0.3)
        off = (o.double() - want).abs() - want.abs() * 2.0 ** -8
        assert float(off.clamp_min(0).norm()) <= 9.5e-4 * float(want.norm())


def test_few_rows_strided_and_apart():
    """Row and matrix strides, a NaN in one matrix, zeros in another; what lies between rows stays."""
    for m, n in ((5, 700), (700, 5)):
        base = torch.stack([ref.gradient(m, n + 3, 9, i) for i in range(4)]).to(DEV)
        g, full = base[:, :, 1:n + 1], torch.full((4, m, n + 2), 7.0, dtype=torch.bfloat16, device=DEV)
        g[1] = 0.0
        g[2, m // 2, n // 2] = math.nan
        out = run(g, out=full[:, :, :n])
        assert (full[:, :, n:] == 7).all() and not out[1].any() and out[2].isnan().all()
        for i in (0, 3):
            assert torch.equal(out[i], run(g[i:i + 1].contiguous())[0])
            assert float((out[i].double() - ref.exact(g[i])).norm()) <= (2.0 ** -8 + 9.5e-4) * float(ref.exact(g[i]).norm())
