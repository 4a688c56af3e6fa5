"""Argument checks of the balance loss and of the stack's backward with an extra
logit gradient, without a GPU: every refusal comes before any CUDA call."""
import ctypes

import pytest

from mixture_experts_layer_expert_gb300 import build, fs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
V = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10004)
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = fs.lib()
    before = fs.fs_launch_count()
    yield lib
    assert fs.fs_launch_count() == before


def desc(**kw):
    a = dict(T=100, E=16, k=4, gate="softmax", n_seqs=3, coef=0.1)
    a.update(kw)
    return fs.make_balance(**a)


def call(f, args, want, **change):
    a = dict(args)
    a.update(change)
    assert f(*a.values()) == want, change


BAD = [(dict(T=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(n_seqs=0), INVALID),
       (dict(coef=float("nan")), INVALID), (dict(coef=float("inf")), INVALID), (dict(E=513), UNSUPPORTED),
       (dict(E=64, k=17), UNSUPPORTED), (dict(T=2 ** 31 - 8), UNSUPPORTED), (dict(n_seqs=65536), UNSUPPORTED)]


def test_forward_refusals(L):
    f = L.fs_balance_loss
    args = dict(desc=desc(), z=V, row=16, bias=V, idx=V, cu=V, mask=V, counts=V, tokens=V, probs=V, loss=V, ws=V,
                ws_bytes=1 << 30, stream=None)
    call(f, args, INVALID, desc=None)
    for kw, want in BAD:
        assert fs.fs_balance_ws_bytes(desc(**kw)) == 0
        call(f, args, want, desc=desc(**kw), row=1 << 20)
    d = desc()
    d.gate = 4
    call(f, args, INVALID, desc=d)
    for k in ("z", "idx", "counts", "tokens", "probs", "loss"):
        call(f, args, INVALID, **{k: None})
        call(f, args, UNSUPPORTED, **{k: ODD})
    for k in ("bias", "cu"):
        call(f, args, UNSUPPORTED, **{k: ODD})
    call(f, args, INVALID, cu=None)                       # three sequences need their borders
    call(f, args, INVALID, row=15)
    call(f, args, UNSUPPORTED, row=2 ** 36 + 1)
    call(f, args, INVALID, ws=None)
    call(f, args, WORKSPACE, ws=MIS)
    call(f, args, WORKSPACE, ws_bytes=fs.fs_balance_ws_bytes(desc()) - 1)


def test_backward_refusals(L):
    f = L.fs_balance_loss_backward
    args = dict(desc=desc(), z=V, row=16, bias=V, cu=V, mask=V, counts=V, tokens=V, d_loss=V, dz=V, d_row=16, stream=None)
    for kw, want in BAD:
        call(f, args, want, desc=desc(**kw), row=1 << 20, d_row=1 << 20)
    for k in ("z", "counts", "tokens", "dz"):
        call(f, args, INVALID, **{k: None})
        call(f, args, UNSUPPORTED, **{k: ODD})
    call(f, args, UNSUPPORTED, d_loss=ODD)
    call(f, args, INVALID, d_row=8)
    call(f, args, INVALID, cu=None)


def test_largest_sizes_have_a_workspace(L):
    assert 0 < fs.fs_balance_ws_bytes(desc(T=2 ** 31 - 8193, E=512, k=16, n_seqs=65535)) < 2 ** 31


def test_stack_backward_aux_and_saved_routing(L):
    d = fs.LayerDesc(300, 256, 8, 2, 256, 0, 0, fs.FS_BF16, 1)
    dref = ctypes.byref(d)
    z, i = ctypes.c_void_p(), ctypes.c_void_p()
    f = L.fs_train_saved_routing
    assert f(dref, 2, 1, ctypes.c_void_p(0x100000), ctypes.byref(z), ctypes.byref(i)) == 0
    size = fs.fs_train_saved_bytes(d, 2)
    assert 0x100000 + size // 2 <= z.value < i.value < 0x100000 + size
    for a in ((2, 2), (2, -1), (0, 0)):
        assert f(dref, *a, V, ctypes.byref(z), ctypes.byref(i)) == INVALID
    assert f(dref, 2, 0, None, ctypes.byref(z), ctypes.byref(i)) == INVALID
    assert f(dref, 2, 0, V, None, ctypes.byref(i)) == INVALID
    d8 = fs.LayerDesc(300, 256, 8, 2, 256, 0, 0, fs.FS_MXFP8, 1)
    assert f(ctypes.byref(d8), 1, 0, V, ctypes.byref(z), ctypes.byref(i)) == UNSUPPORTED
    g = L.fs_farskip_stack_backward_aux
    args = dict(desc=dref, L=1, wiring=0, blocks=(fs.BlockWeights * 1)(), blocks_t=(fs.BlockWeightsT * 1)(), saved=V,
                saved_bytes=1 << 40, d_o=V, d_os=None, d_logits=(ctypes.c_void_p * 1)(None), dx=V,
                grads=(fs.BlockGrads * 1)(), ws=V, ws_bytes=1 << 40, stream=None)
    call(g, args, INVALID, d_logits=None)
    call(g, args, UNSUPPORTED, d_logits=(ctypes.c_void_p * 1)(0x10002))
    call(g, args, INVALID)                                # the blocks' packs are null
    call(g, args, INVALID, L=0)
