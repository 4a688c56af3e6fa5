"""Dispatch's order around the size where one launch sorts all pairs (1,024 tokens): counts, offsets, positions, sources and
rows against a plain stable sort, indices out of range and a token that names an expert twice."""
import pytest
import torch

from mixture_experts_layer_expert_gb300 import configs, fs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(T, E, k, dtype, idx, noalloc=False):
    cfg = configs.LayerConfig("chunk", T=T, d=128, E=E, k=k, c=128, n_shared=0, c_shared=0, L=1, gate="softmax", dtype=dtype)
    desc = fs.make_desc(cfg, T)
    rows = fs.fs_dispatch_rows(desc)
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device=DEV)
    counts, offsets, pos, perm = i32(E), i32(E + 1), i32(T * k), i32(rows)
    u = torch.randn((T, 128), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(DEV)
    xp = torch.zeros((rows, 128), dtype=torch.bfloat16, device=DEV) if dtype == "bf16" else fs.mx4_rows_empty(rows, 128)
    if noalloc:
        fs.fs_dispatch_noalloc(desc, idx.to(DEV), u, counts, offsets, pos, perm, xp)
    else:
        fs.fs_dispatch(desc, idx.to(DEV), u, counts, offsets, pos, perm, xp, fs.alloc_workspace(desc, 0))
    torch.cuda.synchronize()
    return counts.cpu(), offsets.cpu(), pos.cpu().view(T, k), perm.cpu(), xp, u


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 16), (31, 8, 2), (33, 7, 7), (1000, 512, 16), (1024, 40, 8), (1025, 40, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp4"])
@pytest.mark.parametrize("noalloc", [False, True])
def test_stable_order(T, E, k, dtype, noalloc):
    g = torch.Generator().manual_seed(E + k)
    idx = torch.argsort(torch.rand((T, E), generator=g) + (torch.arange(E) % 3 == 1) * 0.5, 1)[:, :k].int()
    counts, offsets, pos, perm, xp, u = run(T, E, k, dtype, idx, noalloc)
    assert fs.fs_get_error() == (0, 0)
    want = torch.bincount(idx.flatten().long(), minlength=E)
    seg = want if dtype == "bf16" else (want + 127) // 128 * 128
    first = torch.cat([torch.zeros(1, dtype=torch.long), seg.cumsum(0)])
    assert torch.equal(counts.long(), want) and torch.equal(offsets.long(), first)
    order = torch.sort(idx.flatten().long(), stable=True).indices            # pairs by expert, then token
    e = idx.flatten().long()[order]
    before = torch.cat([torch.zeros(1, dtype=torch.long), want.cumsum(0)])
    where = torch.empty(T * k, dtype=torch.long)
    where[order] = first[e] + torch.arange(T * k) - before[e]
    assert torch.equal(pos.flatten().long(), where)
    assert torch.equal(perm[where].long(), torch.arange(T).repeat_interleave(k))
    if dtype == "bf16":
        assert torch.equal(xp[where.to(DEV)], u.repeat_interleave(k, 0))


@pytest.mark.parametrize("T", [64, 1500])
def test_bad_and_repeated_indices(T):
    idx = torch.stack([torch.arange(T) % 5, (torch.arange(T) + 1) % 5], 1).int()
    idx[3, 1], idx[T - 1, 0] = 5, -1
    counts, offsets, pos, perm, xp, u = run(T, 5, 2, "bf16", idx)
    assert fs.fs_get_error()[1] == 1
    assert pos[3, 1] == -1 and pos[T - 1, 0] == -1 and int((pos < 0).sum()) == 2
    assert int(counts.sum()) == 2 * T - 2 and offsets[-1] == 2 * T - 2
    idx = torch.zeros((T, 2), dtype=torch.int32)                                # every token names expert 0 twice
    counts, offsets, pos, perm, xp, u = run(T, 5, 2, "bf16", idx)
    assert fs.fs_get_error() == (0, 0) and counts[0] == 2 * T and (offsets[1:] == 2 * T).all()
    assert (pos >= 0).all() and (pos < 2 * T).all()
