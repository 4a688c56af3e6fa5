"""Argument checks of the attention entry points without a GPU: every refusal
comes before any CUDA call."""
import ctypes

import pytest

from mixture_experts_layer_expert_gb300 import build, fs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
V = ctypes.c_void_p(0x10000)            # 16-byte aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)          # 4-byte aligned only
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = fs.lib()
    before = fs.fs_launch_count()
    yield lib
    assert fs.fs_launch_count() == before


def rows(p=0x10000, row=128 * 576, head=576):
    return ctypes.byref(fs.Rows(p, row, head))


def call(f, args, want, **change):
    a = dict(args)
    a.update(change)
    assert f(*a.values()) == want, change


def test_rope_refusals(L):
    rope = lambda **kw: ctypes.byref(fs.make_rope(**dict(dict(d_rot=64), **kw)))
    args = dict(rope=rope(), T=4, H=2, dtype=0, pos=V, x=V, x_row=128, x_head=64, y=V, y_row=128, y_head=64, inverse=0,
                stream=None)
    f = L.fs_rope
    call(f, args, INVALID, rope=None)
    for bad in (dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(mscale=0.0), dict(d_rot=0),
                dict(factor=4.0, orig_len=0.0), dict(factor=4.0, orig_len=4096.0, beta_fast=1.0, beta_slow=2.0),
                dict(base=float("inf")), dict(d_rot=-16)):
        call(f, args, INVALID, rope=rope(**bad))
    call(f, args, INVALID, rope=ctypes.byref(fs.RopeDesc(64, 2, 1e4, 1, 0, 32, 1, 1)))
    for bad in (24, 272):
        call(f, args, UNSUPPORTED, rope=rope(d_rot=bad))
    for k in ("T", "H"):
        call(f, args, INVALID, **{k: 0})
    call(f, args, INVALID, dtype=9)
    call(f, args, UNSUPPORTED, dtype=2)
    for k in ("pos", "x", "y"):
        call(f, args, INVALID, **{k: None})
        call(f, args, UNSUPPORTED, **{k: ODD})
    call(f, args, UNSUPPORTED, x=MIS)
    call(f, args, UNSUPPORTED, x_row=124)
    call(f, args, UNSUPPORTED, x_head=0)                 # broadcast heads
    call(f, args, INVALID, x_row=-128)
    call(f, args, INVALID, y_row=64)                     # rows overlap
    call(f, args, INVALID, y_head=32)                    # heads overlap


def test_cache_sizes_and_refusals(L):
    assert fs.fs_latent_cache_bytes(fs.make_latent_cache(3, 5, "bf16")) == 15 * 1152
    assert fs.fs_latent_cache_bytes(fs.make_latent_cache(3, 5, "fp8")) == 15 * 656
    assert fs.fs_latent_cache_bytes(fs.make_latent_cache(2 ** 31 - 1, 64, "bf16")) == (2 ** 31 - 1) * 64 * 1152
    for bad in (fs.make_latent_cache(0, 5), fs.make_latent_cache(3, 0), fs.make_latent_cache(3, 5, "f32"),
                fs.make_latent_cache(3, 5, "mxfp8"), fs.make_latent_cache(2 ** 31, 5), fs.LatentCache(3, 5, 9)):
        assert fs.fs_latent_cache_bytes(bad) == 0
    desc = ctypes.byref(fs.make_latent_cache(3, 5))
    rope = ctypes.byref(fs.make_rope(64))
    w = dict(desc=desc, T=4, c=V, c_row=512, kr=V, kr_row=64, rope=rope, pos=V, slots=V, cache=V, stream=None)
    f = L.fs_latent_cache_write
    call(f, w, INVALID, desc=None)
    call(f, w, UNSUPPORTED, desc=ctypes.byref(fs.make_latent_cache(3, 5, "f32")))
    call(f, w, INVALID, T=0)
    call(f, w, INVALID, pos=None)
    call(f, w, UNSUPPORTED, rope=ctypes.byref(fs.make_rope(32)))
    for k in ("c", "kr", "slots", "cache"):
        call(f, w, INVALID, **{k: None})
        call(f, w, UNSUPPORTED, **{k: MIS})
    call(f, w, UNSUPPORTED, c_row=0)
    call(f, w, UNSUPPORTED, kr_row=68)
    r = dict(desc=desc, cache=V, T=4, slots=V, c=V, c_row=512, kr=V, kr_row=64, stream=None)
    f = L.fs_latent_cache_read
    call(f, r, INVALID, T=0)
    call(f, r, INVALID, c_row=504)                       # output rows overlap
    call(f, r, INVALID, kr_row=56)
    for k in ("c", "kr", "slots", "cache"):
        call(f, r, INVALID, **{k: None})
        call(f, r, UNSUPPORTED, **{k: MIS})


def test_decode_refusals(L):
    ws = fs.fs_latent_decode_ws_bytes(128, 4, 2)
    assert ws > 0
    for bad in ((0, 4, 1), (129, 4, 1), (16, 0, 1), (16, 4, 0), (16, 4, 17), (128, 2 ** 25, 1)):
        assert fs.fs_latent_decode_ws_bytes(*bad) == 0
    W = ctypes.c_void_p(0x1000000)
    args = dict(desc=ctypes.byref(fs.make_latent_cache(9, 64)), H=128, B=4, n_q=2, ql=rows(), qr=rows(), cache=V,
                table=V, max_pages=8, table_row=8, lens=V, scale=0.1, out=rows(), lse=None, ws=W, ws_bytes=ws,
                stream=None)
    f = L.fs_latent_decode
    for k in ("desc", "ql", "qr", "cache", "table", "lens", "out", "ws"):
        call(f, args, INVALID, **{k: None})
    for k in ("ql", "qr", "out"):
        call(f, args, INVALID, **{k: rows(p=None)})
        call(f, args, UNSUPPORTED, **{k: rows(p=0x10008)})
        call(f, args, UNSUPPORTED, **{k: rows(row=128 * 576 + 4)})
        call(f, args, INVALID, **{k: rows(row=-8)})
    call(f, args, UNSUPPORTED, ql=rows(head=0))
    call(f, args, INVALID, out=rows(head=504))           # heads overlap
    call(f, args, UNSUPPORTED, H=129)
    call(f, args, UNSUPPORTED, n_q=17)
    call(f, args, INVALID, B=0)
    call(f, args, INVALID, max_pages=0)
    call(f, args, INVALID, table_row=7)
    call(f, args, INVALID, scale=float("inf"))
    call(f, args, UNSUPPORTED, lse=ODD)
    call(f, args, UNSUPPORTED, lens=ODD)
    call(f, args, WORKSPACE, ws_bytes=ws - 1)
    call(f, args, WORKSPACE, ws=ctypes.c_void_p(0x1000010))


def test_prefill_refusals(L):
    d = lambda **kw: ctypes.byref(fs.LatentPrefillDesc(*dict(dict(heads=4, n_seqs=2, Tq=64, Tk=96, causal=1,
                                                                  scale=0.1), **kw).values()))
    r = lambda **kw: rows(**dict(dict(row=4 * 192, head=192), **kw))
    fwd = dict(desc=d(), q=r(), kn=r(), kr=r(), v=r(), cu_q=V, cu_k=V, out=r(), lse=V, stream=None)
    W = ctypes.c_void_p(0x1000000)
    n = fs.fs_latent_prefill_backward_ws_bytes(4, 64, 96)
    assert n > 0 and fs.fs_latent_prefill_backward_ws_bytes(129, 64, 96) == 0
    assert fs.fs_latent_prefill_backward_ws_bytes(4, 0, 96) == 0
    bwd = dict(desc=d(), q=r(), kn=r(), kr=r(), v=r(), cu_q=V, cu_k=V, out=r(), lse=V, do=r(), dq=r(), dkn=r(),
               dkr=r(), dv=r(), ws=W, ws_bytes=n, stream=None)
    for f, args, outs in ((L.fs_latent_prefill, fwd, ("out",)),
                          (L.fs_latent_prefill_backward, bwd, ("dq", "dkn", "dv"))):
        for k in args:
            if k not in ("stream", "ws_bytes"):
                call(f, args, INVALID, **{k: None})
        for bad in (dict(heads=0), dict(n_seqs=0), dict(Tq=0), dict(Tk=0), dict(scale=float("nan"))):
            call(f, args, INVALID, desc=d(**bad))
        call(f, args, UNSUPPORTED, desc=d(heads=129))
        for k in ("q", "kn", "v"):
            call(f, args, UNSUPPORTED, **{k: r(p=0x10008)})
            call(f, args, UNSUPPORTED, **{k: r(head=0)})
            call(f, args, UNSUPPORTED, **{k: r(row=4 * 192 + 2)})
            call(f, args, INVALID, **{k: r(head=-192)})
        call(f, args, UNSUPPORTED, kr=r(row=0))
        for k in outs:
            call(f, args, INVALID, **{k: r(head=64)})    # heads overlap
            call(f, args, INVALID, **{k: r(row=192)})    # rows overlap
        call(f, args, UNSUPPORTED, cu_q=ODD)
    call(L.fs_latent_prefill_backward, bwd, INVALID, dkr=r(row=32))
    call(L.fs_latent_prefill_backward, bwd, WORKSPACE, ws_bytes=n - 1)
    call(L.fs_latent_prefill_backward, bwd, WORKSPACE, ws=ctypes.c_void_p(0x1000080))


def test_binding_refuses_what_the_pointers_hide():
    """Shapes, types and devices are checked before a pointer is taken."""
    import torch
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(fs.FsError):
        fs.fs_rope(fs.make_rope(64), torch.zeros(2, dtype=torch.int64), x, x)
    with pytest.raises(fs.FsError):
        fs.fs_rope(fs.make_rope(64), torch.zeros(3, dtype=torch.int32), x, x)
    with pytest.raises(fs.FsError):
        fs.fs_rope(fs.make_rope(32), torch.zeros(2, dtype=torch.int32), x, x)
    with pytest.raises(fs.FsError):
        fs.fs_rope(fs.make_rope(64), torch.zeros(2, dtype=torch.int32), x, x)          # not on the GPU
