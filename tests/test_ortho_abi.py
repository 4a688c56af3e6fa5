"""Argument checks of the orthogonalised update without a GPU, and the rounding
model of its tolerances against the claim it stands for."""
import ctypes

import pytest
import torch

import ortho_ref as ref
from mixture_experts_layer_expert_gb300 import build, fs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
V = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = fs.lib()
    before = fs.fs_launch_count()
    yield lib
    assert fs.fs_launch_count() == before


def desc(**kw):
    a = dict(batch=3, m=40, n=70, dtype="f32", scale=1.0, coefs=ref.USUAL, eps=1e-7)
    a.update(kw)
    return fs.make_orthogonalize(**a)


def test_refusals(L):
    f = L.fs_orthogonalize
    args = dict(desc=desc(), g=V, g_row=70, g_mat=2800, out=V, out_row=70, out_mat=2800, ws=V, ws_bytes=1 << 40, stream=None)

    def call(want, **change):
        a = dict(args)
        a.update(change)
        assert f(*a.values()) == want, change
    call(INVALID, desc=None)
    nan, inf = float("nan"), float("inf")
    for kw, want in [(dict(batch=0), INVALID), (dict(m=0), INVALID), (dict(n=-1), INVALID), (dict(coefs=[]), INVALID),
                     (dict(scale=nan), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=nan), INVALID), (dict(eps=inf), INVALID),
                     (dict(coefs=[(nan, 0, 0)]), INVALID), (dict(coefs=[(1, inf, 0)]), INVALID),
                     (dict(m=16385), UNSUPPORTED), (dict(n=16385), UNSUPPORTED), (dict(dtype="fp8"), UNSUPPORTED),
                     (dict(coefs=[(9.0, 0, 0)]), UNSUPPORTED), (dict(coefs=[(3.0, 3.0, 3.0)] * 4), UNSUPPORTED),
                     (dict(coefs=[(2.0, 0, 0)] * 4), UNSUPPORTED), (dict(coefs=[(1.0, 2000.0, -2000.0)]), UNSUPPORTED)]:
        assert fs.fs_orthogonalize_ws_bytes(desc(**kw)) == 0
        call(want, desc=desc(**kw), g_row=1 << 20, out_row=1 << 20, g_mat=1 << 35, out_mat=1 << 35)
    d = desc()
    d.steps = 17
    call(UNSUPPORTED, desc=d)
    d = desc()
    d.dtype = 9
    call(INVALID, desc=d)
    for k in ("g", "out"):
        call(INVALID, **{k: None})
        call(UNSUPPORTED, **{k: ODD})
    call(UNSUPPORTED, g=ctypes.c_void_p(0x10002))
    for k in ("g", "out"):
        call(INVALID, **{k + "_row": 69})
        call(INVALID, **{k + "_mat": 2799})
        call(UNSUPPORTED, **{k + "_mat": 2 ** 36 + 1})
    call(INVALID, ws=None)
    call(WORKSPACE, ws=ctypes.c_void_p(0x10080))
    call(WORKSPACE, ws_bytes=fs.fs_orthogonalize_ws_bytes(desc()) - 1)
    with pytest.raises(fs.FsError):
        fs.make_orthogonalize(1, 2, 2, coefs=[(1, 0, 0)] * 17)
    with pytest.raises(fs.FsError):
        fs.make_orthogonalize(1, 2, 2, coefs=[(1, 0)])


def test_workspace_stays_bounded(L):
    one = fs.fs_orthogonalize_ws_bytes(desc(batch=1, m=16384, n=16384))
    assert one == fs.fs_orthogonalize_ws_bytes(desc(batch=100, m=16384, n=16384)) > 2 ** 31
    for b, m, n in ((256, 2048, 7168), (10 ** 6, 1, 1), (128, 768, 2048)):
        assert 0 < fs.fs_orthogonalize_ws_bytes(desc(batch=b, m=m, n=n)) < 2 ** 31 + 2 ** 20


def test_rounding_model():
    """Five usual steps in the documented roundings stay within the documented 0.3%, bf16's rounding included,
    while X in a single fp16 or bf16 number would not for a gradient of few tokens."""
    for m, n, r in ((128, 128, 300), (128, 200, 8), (96, 500, 24)):
        g = ref.gradient(m, n, r, m + r)
        want = ref.exact(g)
        got = ref.rounded(g).to(torch.bfloat16).double()
        assert float((got - want).norm() / want.norm()) < 3e-3
    x = ref.start(g, 1e-7).half().double()
    for a, b, c in ref.USUAL:
        s = x @ x.T
        x = (a * x + (b * s + c * (s @ s)) @ x)
        x = ref.half(x, 13)
    assert float((x - want).norm() / want.norm()) > 1e-2
