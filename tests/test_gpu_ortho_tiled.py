"""Orthogonalised updates of matrices that the tiled kernels take (shorter side above 128, or longer side above
4,096): edges of norm, loaders, strides and stores, which these kernels have of their own, against the exact steps with
tolerances from the roundings of the kernels (ortho_carry)."""
import math

import pytest
import torch

import ortho_carry as carry
import ortho_ref as ref
from mixture_experts_layer_expert_gb300 import fs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(g, scale=1.0, coefs=ref.USUAL, eps=1e-7, out=None):
    b, m, n = g.shape
    assert carry.kernel(m, n) == "tiled"
    desc = fs.make_orthogonalize(b, m, n, "f32" if g.dtype == torch.float32 else "bf16", scale, coefs, eps)
    ws = torch.full((fs.fs_orthogonalize_ws_bytes(desc),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((b, m, n), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    fs.fs_orthogonalize(desc, g, out, ws)
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)
    return out


def check(out, g, **kw):
    for o, x in zip(out, g):
        want, room = carry.tolerance(x.to(DEV), **kw)
        off = float((o.double() - want).norm())
        assert off <= room + 1e-30, "%.2e off, %.2e allowed (norm %.2e)" % (off, room, float(want.norm()))
        if kw.get("coefs", ref.USUAL) == ref.USUAL and min(x.shape) >= 32:
            assert off <= 3e-3 * float(want.norm())


SHAPES = [(2, 129, 129), (1, 129, 260), (2, 200, 333), (2, 333, 200), (1, 64, 5000), (2, 5000, 100), (1, 128, 4097),
          (2, 4100, 33), (1, 17, 4097), (1, 10, 9000), (1, 9000, 10), (1, 1, 16384), (2, 16384, 1), (1, 2, 8193)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rank", ["full", "few"])
def test_against_exact(shape, dtype, rank):
    """Long matrices of few rows among them: most of a tile of 256 rows is then past the matrix's end."""
    b, m, n = shape
    r = min(m, n)
    g = torch.stack([ref.gradient(m, n, 2 * r if rank == "full" else max(1, r // (4 + i)), i + m + n) for i in range(b)])
    g = g.to(dtype).to(DEV)
    check(run(g, scale=0.2 * math.sqrt(max(m, n))), g, scale=0.2 * math.sqrt(max(m, n)))


@pytest.mark.parametrize("m,n", [(200, 333), (333, 200), (40, 4100)])
@pytest.mark.parametrize("power", [-140, -100, -60, 0, 60, 110])
def test_norm_over_the_whole_range(m, n, power):
    """The result does not depend on the gradient's scale, from subnormal numbers to the largest (eps 0)."""
    g = ref.gradient(m, n, 60, 4)
    g = g / g.abs().max()
    big = torch.ldexp(g.double(), torch.tensor(power)).float()           # subnormal below 2^-126: rounded to 2^-149
    check(run(big[None].to(DEV), eps=0.0), big[None], eps=0.0)


@pytest.mark.parametrize("m,n", [(200, 333), (333, 200), (4100, 40)])
def test_magnitudes_of_every_range_in_one_matrix(m, n):
    """Rows (columns) of 2^-70, 1 and 2^45 times the rest: each third of the norm's three sums counts, and the largest decides."""
    g = ref.gradient(m, n, 60, 5)
    for lo, hi in ((-70, 0), (0, 45), (-70, 45)):
        x = g.clone()
        x[: m // 2] = torch.ldexp(x[: m // 2], torch.tensor(lo))
        x[m // 2:] = torch.ldexp(x[m // 2:], torch.tensor(hi))
        check(run(x[None].to(DEV), eps=0.0), x[None], eps=0.0)


@pytest.mark.parametrize("m,n", [(200, 333), (336, 200), (20, 4100)])
def test_zero_matrices_and_eps(m, n):
    g = torch.zeros((3, m, n), device=DEV)
    g[1] = ref.gradient(m, n, 50, 5).to(DEV)
    for eps in (0.0, 1e-7):
        out = run(g, eps=eps)
        assert not out[0].any() and not out[2].any()
        check(out[1:2], g[1:2], eps=eps)
    check(run(g[1:2], eps=0.5), g[1:2], eps=0.5)                           # eps as large as the norm counts


@pytest.mark.parametrize("m,n", [(200, 333), (333, 200), (5000, 24), (24, 5000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_infinity_stay_in_their_matrix(m, n, dtype):
    g = torch.stack([ref.gradient(m, n, 60, i) for i in range(5)]).to(dtype).to(DEV)
    clean = run(g)
    g[1, m - 1, n - 1] = math.nan
    g[2, 0, 0] = math.inf
    g[3, m // 2, n // 2] = -math.inf
    out = run(g)
    assert torch.equal(out[0], clean[0]) and torch.equal(out[4], clean[4])
    assert out[1:4].isnan().all()


@pytest.mark.parametrize("m,n", [(200, 333), (333, 200), (136, 264), (264, 136), (9, 8200), (8200, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_offsets(m, n, dtype):
    """Views with odd and even strides and offsets, in and out: the stores by TMA and by lanes; what lies between is left."""
    b = 3
    g = torch.stack([ref.gradient(m, n, 30, i) for i in range(b)]).to(dtype).to(DEV)
    want = run(g)
    for pad_r, pad_m, off in ((1, 3, 1), (8, 0, 8), (6, 2, 4), (0, 1, 0)):
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


@pytest.mark.parametrize("coefs", [[(1.5, -0.5, 0.0)], [(1.875, -1.25, 0.375)] * 8, [(4.0, -6.0, 2.5), (3.0, -3.5, 1.2), (1.5, -0.5, 0.0)],
                                   [(0.5, 0.0, 0.0)] * 16, [(2.0, 0.0, 0.0)] * 3, [(3.4445, -4.7750, 2.0315)] * 9])
@pytest.mark.parametrize("m,n", [(160, 300), (300, 160)])
def test_other_coefficients(coefs, m, n):
    g = torch.stack([ref.gradient(m, n, 300, 1), ref.gradient(m, n, 10, 2)]).to(DEV)
    check(run(g, coefs=coefs), g, coefs=coefs)


@pytest.mark.parametrize("m,n", [(160, 300), (5000, 20)])
def test_a_batchs_order_does_not_matter(m, n):
    g = torch.stack([ref.gradient(m, n, 40 + i, i) for i in range(7)]).to(DEV)
    out = run(g)
    back = run(g.flip(0).contiguous()).flip(0)
    assert torch.equal(out, back)
    assert all(torch.equal(run(g[i:i + 1])[0], out[i]) for i in (0, 3, 6))


@pytest.mark.parametrize("m,n", [(301, 2600), (2600, 301)])
def test_stores_by_lanes_match_stores_by_tma(m, n):
    """Many pieces through each warp's two buffers, which take a piece's inputs by TMA after the last one's result left by lanes."""
    g = torch.stack([ref.gradient(m, n, 40, i) for i in range(4)]).to(DEV)
    width = (n + 7) // 8 * 8
    whole = torch.full((4, m, width), 5.0, dtype=torch.bfloat16, device=DEV)
    want = run(g, out=whole[:, :, :n])
    for _ in range(5):
        odd = torch.full((4, m, n + 1 + n % 2), 5.0, dtype=torch.bfloat16, device=DEV)
        assert odd.stride(1) % 8
        assert torch.equal(run(g, out=odd[:, :, :n]), want)
        assert (odd[:, :, n:] == 5).all()
