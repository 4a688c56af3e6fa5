"""Argument checks and sizes of the 4-bit microscaled entry points without a GPU,
and the 64-bit definition that the GPU tests use against brute force."""
import ctypes

import pytest
import torch

import mx4_ref as ref
from mixture_experts_layer_expert_gb300 import build, fs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
V = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = fs.lib()
    before = fs.fs_launch_count()
    yield lib
    assert fs.fs_launch_count() == before


def test_sizes(L):
    assert fs.fs_mx4_rows_bytes(1, 128) == 128 * 64 + 512
    assert fs.fs_mx4_rows_bytes(129, 1408) == 256 * 704 + 2 * 11 * 512
    for bad in ((0, 128), (1, 0), (1, 64), (-1, 128)):
        assert fs.fs_mx4_rows_bytes(*bad) == 0
    assert fs.fs_packed_bytes(1, 8, 128, fs.FS_MXFP4) == 32768 + 1024
    assert fs.fs_packed_bytes(3, 264, 384, fs.FS_MXFP4) == 3 * 2 * (2 * 32768 + 3 * 1024)
    for bad in ((1, 4, 128), (1, 8, 64), (0, 8, 128)):
        assert fs.fs_packed_bytes(*bad, fs.FS_MXFP4) == 0
    d = fs.LayerDesc(300, 256, 8, 2, 256, 1, 128, fs.FS_MXFP4, 1)
    assert fs.fs_dispatch_rows(d) == (600 + 127 * 8 + 127) // 128 * 128
    assert 0 < fs.fs_workspace_bytes(d, 2) < fs.fs_workspace_bytes(fs.LayerDesc(300, 256, 8, 2, 256, 1, 128, fs.FS_MXFP8, 1), 2)
    assert fs.fs_train_saved_bytes(d, 1) == 0
    for bad in (dict(d=192), dict(c=64), dict(c_shared=64)):
        e = fs.LayerDesc(300, 256, 8, 2, 256, 1, 128, fs.FS_MXFP4, 1)
        for k, v in bad.items():
            setattr(e, k, v)
        assert fs.fs_workspace_bytes(e, 1) == 0


def test_refusals(L):
    f = L.fs_quantize_rows_mx4
    assert f(0, 128, V, V, None) == INVALID and f(1, 0, V, V, None) == INVALID
    assert f(1, 64, V, V, None) == UNSUPPORTED and f(2 ** 31, 128, V, V, None) == UNSUPPORTED
    assert f(1, 128, None, V, None) == INVALID and f(1, 128, V, MIS, None) == UNSUPPORTED
    g = L.fs_linear_mx4
    ok = dict(rows=5, N=264, K=384, q=V, w=V, y=V, y_dtype=0, y_row=264, ws=V, ws_bytes=1 << 30, stream=None)
    def call(want, **kw):
        a = dict(ok)
        a.update(kw)
        assert g(*a.values()) == want, kw
    for k in ("rows", "N", "K"):
        call(INVALID, **{k: 0})
    call(UNSUPPORTED, N=260, y_row=264)
    call(UNSUPPORTED, K=64)
    call(UNSUPPORTED, rows=2 ** 31)
    call(UNSUPPORTED, rows=2 ** 31 - 2048, N=2 ** 31 - 8, y_row=2 ** 31)
    call(INVALID, y_dtype=2)
    call(INVALID, y_row=256)
    call(UNSUPPORTED, y_row=268)
    call(UNSUPPORTED, y_row=2 ** 36 + 8)
    for k in ("q", "w", "y"):
        call(INVALID, **{k: None})
        call(UNSUPPORTED, **{k: MIS})
    call(INVALID, ws=None)
    call(WORKSPACE, ws=MIS)
    call(WORKSPACE, ws_bytes=0)
    assert fs.fs_linear_mx4_ws_bytes(5, 264, 384) > 0 and fs.fs_linear_mx4_ws_bytes(5, 260, 384) == 0
    assert L.fs_pack_w3(1, 12, 128, fs.FS_MXFP4, V, V, None) == UNSUPPORTED
    assert L.fs_pack_w13(1, 64, 128, fs.FS_MXFP4, V, V, V, None) == UNSUPPORTED
    d = ctypes.byref(fs.LayerDesc(300, 256, 8, 2, 256, 1, 128, fs.FS_MXFP4, 1))
    assert L.fs_grouped_swiglu_gather(d, V, V, V, V, V, V, ctypes.c_void_p(0x100000), 1 << 40, None) == UNSUPPORTED


def test_definition():
    """The exponent against a search, the codes against every grid value, midpoints to even codes."""
    for a, e in ((6.0, 0), (6.01, 1), (3.0, -1), (3.01, 0), (0.0, 0), (1e-45, -127), (3.3e38, 126)):
        assert ref.block_exp(torch.tensor([a], dtype=torch.float64)).item() == e
    x = torch.zeros(32)
    x[:8] = ref.GRID.float()
    codes, _ = ref.quantise(x)
    assert codes[:8].tolist() == list(range(8))
    x[:8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    codes, _ = ref.quantise(x)
    assert codes[:8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    y = torch.randn((4, 64), generator=torch.Generator().manual_seed(0))
    v = ref.rounded(y)
    b = y.double().unflatten(-1, (-1, 32))
    s = torch.exp2(ref.block_exp(b.abs().amax(-1)))[..., None]
    full = torch.cat([ref.GRID, -ref.GRID])
    best = ((b / s)[..., None] - full).abs().amin(-1) * s
    assert torch.equal((v.unflatten(-1, (-1, 32)) - b).abs(), best)
