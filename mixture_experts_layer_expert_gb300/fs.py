"""Thin Python binding of libfs (the C ABI in include/fs.h).

Argument marshalling only: every function passes tensor data pointers, sizes
and the current CUDA stream to the library entry point of the same name.  The
library is loaded from the in-tree build (``_build/libfs.so``); if it is
missing, ``lib()`` raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from .configs import LayerConfig

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfs.so")
_lib = None

FS_BF16, FS_F32, FS_FP8, FS_MXFP8, FS_MXFP4 = 0, 1, 2, 3, 4
DTYPES = {"bf16": FS_BF16, "f32": FS_F32, "fp8": FS_FP8, "mxfp8": FS_MXFP8, "mxfp4": FS_MXFP4}
GATES = {"softmax": 0, "softmax_renorm": 1, "sigmoid": 2, "sigmoid_norm": 3}
WIRINGS = {"partial": 0, "outdated": 1, "disabled": 2, "attn_farskip": 3, "attn_plain": 4}
STATUS = {0: "FS_OK", 1: "FS_ERR_INVALID_ARG", 2: "FS_ERR_UNSUPPORTED", 3: "FS_ERR_WORKSPACE",
          4: "FS_ERR_CUDA", 5: "FS_ERR_DEVICE_STATE"}


class FsError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__("%s failed: %s%s" % (what, STATUS.get(status, status), (" (%s)" % detail) if detail else ""))


class LayerDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "E", "k", "c", "n_shared", "c_shared", "dtype", "gate")]


class BlockWeights(ctypes.Structure):
    _fields_ = [("w_r", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("w13", ctypes.c_void_p),
                ("w3", ctypes.c_void_p), ("w13_shared", ctypes.c_void_p), ("w3_shared", ctypes.c_void_p),
                ("w_att", ctypes.c_void_p)]


class BlockWeightsT(ctypes.Structure):
    _fields_ = [("w13t", ctypes.c_void_p), ("w3t", ctypes.c_void_p), ("w13t_shared", ctypes.c_void_p),
                ("w3t_shared", ctypes.c_void_p), ("w_rt", ctypes.c_void_p)]


class BlockGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dw_r", "dw1", "dw2", "dw3", "dw1_shared", "dw2_shared", "dw3_shared")]


class RopeDesc(ctypes.Structure):
    _fields_ = [("d_rot", ctypes.c_int32), ("layout", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "orig_len", "beta_fast", "beta_slow", "mscale")]


class BalanceDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "k", "gate", "n_seqs")] + [("coef", ctypes.c_float)]


class OrthogonalizeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "m", "n", "dtype", "steps")] + [
        ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("coefs", ctypes.c_float * 48)]


class LatentCache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class LatentPrefillDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "n_seqs", "Tq", "Tk", "causal")] + [("scale", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


_VP, _I32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_I64, _RP = ctypes.c_int64, ctypes.POINTER(Rows)
_SIGS = {
    "fs_workspace_bytes": (_SZ, [ctypes.POINTER(LayerDesc), ctypes.c_int]),
    "fs_pack_w13": (_I32, [_I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP]),
    "fs_pack_w3_shared": (_I32, [_I32, _I32, _I32, _I32, _VP, _VP, _VP]),
    "fs_pack_w3": (_I32, [_I32, _I32, _I32, _I32, _VP, _VP, _VP]),
    "fs_packed_bytes": (_SZ, [_I32, _I32, _I32, _I32]),
    "fs_router_topk": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_dispatch": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_dispatch_noalloc": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "fs_grouped_swiglu": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_grouped_swiglu_gather": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_shared_expert": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_combine": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _I32,
                          _VP, _VP]),
    "fs_attn_standin": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fs_shared_expert_combine": (_I32, [ctypes.POINTER(LayerDesc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP,
                                        _I32, _VP, _I32, _VP, _SZ, _VP]),
    "fs_farskip_stack": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, ctypes.POINTER(BlockWeights), _VP, _VP,
                                _VP, _VP, _SZ, _VP]),
    "fs_farskip_stack_overlap": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, ctypes.POINTER(BlockWeights), _VP,
                                        _VP, _VP, _VP, _SZ, _VP, _VP]),
    "fs_workspace_bytes_overlap": (_SZ, [ctypes.POINTER(LayerDesc), ctypes.c_int]),
    "fs_workspace_bytes_attn": (_SZ, [ctypes.POINTER(LayerDesc), ctypes.c_int]),
    "fs_fp8_rows_bytes": (_SZ, [ctypes.c_int64, _I32]),
    "fs_pack_w13t": (_I32, [_I32, _I32, _I32, _VP, _VP, _VP, _VP]),
    "fs_pack_w3t": (_I32, [_I32, _I32, _I32, _VP, _VP, _VP]),
    "fs_pack_w3t_shared": (_I32, [_I32, _I32, _I32, _VP, _VP, _VP]),
    "fs_pack_wrt": (_I32, [_I32, _I32, _VP, _VP, _VP]),
    "fs_train_saved_bytes": (_SZ, [ctypes.POINTER(LayerDesc), ctypes.c_int]),
    "fs_workspace_bytes_backward": (_SZ, [ctypes.POINTER(LayerDesc), ctypes.c_int]),
    "fs_farskip_stack_train": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, ctypes.POINTER(BlockWeights), _VP, _VP,
                                      _VP, _VP, _SZ, _VP, _SZ, _VP]),
    "fs_farskip_stack_backward": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, ctypes.POINTER(BlockWeights),
                                         ctypes.POINTER(BlockWeightsT), _VP, _SZ, _VP, _VP, _VP,
                                         ctypes.POINTER(BlockGrads), _VP, _SZ, _VP]),
    "fs_farskip_stack_backward_aux": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, ctypes.POINTER(BlockWeights),
                                             ctypes.POINTER(BlockWeightsT), _VP, _SZ, _VP, _VP, ctypes.POINTER(_VP),
                                             _VP, ctypes.POINTER(BlockGrads), _VP, _SZ, _VP]),
    "fs_train_saved_routing": (_I32, [ctypes.POINTER(LayerDesc), _I32, _I32, _VP, ctypes.POINTER(_VP),
                                      ctypes.POINTER(_VP)]),
    "fs_orthogonalize_ws_bytes": (_SZ, [ctypes.POINTER(OrthogonalizeDesc)]),
    "fs_orthogonalize": (_I32, [ctypes.POINTER(OrthogonalizeDesc), _VP, _I64, _I64, _VP, _I64, _I64, _VP, _SZ, _VP]),
    "fs_balance_ws_bytes": (_SZ, [ctypes.POINTER(BalanceDesc)]),
    "fs_balance_loss": (_I32, [ctypes.POINTER(BalanceDesc), _VP, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                               _SZ, _VP]),
    "fs_balance_loss_backward": (_I32, [ctypes.POINTER(BalanceDesc), _VP, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                        _I64, _VP]),
    "fs_quantize_rows_fp8": (_I32, [ctypes.c_int64, _I32, _VP, _VP, _VP]),
    "fs_mx_rows_bytes": (_SZ, [ctypes.c_int64, _I32]),
    "fs_quantize_rows_mx": (_I32, [ctypes.c_int64, _I32, _VP, _VP, _VP]),
    "fs_mx4_rows_bytes": (_SZ, [ctypes.c_int64, _I32]),
    "fs_quantize_rows_mx4": (_I32, [ctypes.c_int64, _I32, _VP, _VP, _VP]),
    "fs_linear_mx4_ws_bytes": (_SZ, [ctypes.c_int64, _I32, _I32]),
    "fs_linear_mx4": (_I32, [ctypes.c_int64, _I32, _I32, _VP, _VP, _VP, _I32, _I64, _VP, _SZ, _VP]),
    "fs_dispatch_rows": (ctypes.c_int64, [ctypes.POINTER(LayerDesc)]),
    "fs_rope": (_I32, [ctypes.POINTER(RopeDesc), _I64, _I32, _I32, _VP, _VP, _I64, _I64, _VP, _I64, _I64, _I32, _VP]),
    "fs_latent_cache_bytes": (_SZ, [ctypes.POINTER(LatentCache)]),
    "fs_latent_cache_write": (_I32, [ctypes.POINTER(LatentCache), _I64, _VP, _I64, _VP, _I64, ctypes.POINTER(RopeDesc),
                                     _VP, _VP, _VP, _VP]),
    "fs_latent_cache_read": (_I32, [ctypes.POINTER(LatentCache), _VP, _I64, _VP, _VP, _I64, _VP, _I64, _VP]),
    "fs_latent_decode_ws_bytes": (_SZ, [_I32, _I32, _I32]),
    "fs_latent_decode": (_I32, [ctypes.POINTER(LatentCache), _I32, _I32, _I32, _RP, _RP, _VP, _VP, _I32, _I64, _VP,
                                ctypes.c_float, _RP, _VP, _VP, _SZ, _VP]),
    "fs_latent_prefill": (_I32, [ctypes.POINTER(LatentPrefillDesc), _RP, _RP, _RP, _RP, _VP, _VP, _RP, _VP, _VP]),
    "fs_latent_prefill_backward_ws_bytes": (_SZ, [_I32, _I32, _I32]),
    "fs_latent_prefill_backward": (_I32, [ctypes.POINTER(LatentPrefillDesc), _RP, _RP, _RP, _RP, _VP, _VP, _RP, _VP,
                                          _RP, _RP, _RP, _RP, _RP, _VP, _SZ, _VP]),
    "fs_get_error": (_I32, [ctypes.POINTER(ctypes.c_int32)]),
    "fs_launch_count": (ctypes.c_uint64, []),
    "fs_selftest_wait_timeout": (_I32, [_I32, _VP]),
    "fs_last_cuda_error": (ctypes.c_char_p, []),
    "fs_status_string": (ctypes.c_char_p, [_I32]),
}


def lib():
    """Load libfs.so (built in-tree).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfs.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        detail = ""
        if status in (3, 4):
            detail = (lib().fs_last_cuda_error() or b"").decode()
        raise FsError(status, what, detail)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The raw stream of a call, without building a Stream object when none is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def make_desc(cfg: LayerConfig, T: int | None = None) -> LayerDesc:
    return LayerDesc(cfg.T if T is None else T, cfg.d, cfg.E, cfg.k, cfg.c, cfg.n_shared, cfg.c_shared,
                     DTYPES[cfg.dtype], GATES[cfg.gate])


# ----------------------------------------------------------------- entry points

def fs_workspace_bytes(desc: LayerDesc, L: int = 0) -> int:
    return int(lib().fs_workspace_bytes(ctypes.byref(desc), L))


def fs_pack_w13(G, c, d, dtype, w1, w2, w13, stream=None):
    _check(lib().fs_pack_w13(G, c, d, dtype, _p(w1), _p(w2), _p(w13), _stream(stream)), "fs_pack_w13")


def fs_packed_bytes(G, N, K, dtype) -> int:
    return int(lib().fs_packed_bytes(G, N, K, dtype))


def fs_pack_w3(G, d, c, dtype, w3, w3p, stream=None):
    _check(lib().fs_pack_w3(G, d, c, dtype, _p(w3), _p(w3p), _stream(stream)), "fs_pack_w3")


def fs_pack_w3_shared(n_shared, c_shared, d, dtype, w3s, w3cat, stream=None):
    _check(lib().fs_pack_w3_shared(n_shared, c_shared, d, dtype, _p(w3s), _p(w3cat), _stream(stream)),
           "fs_pack_w3_shared")


def fs_fp8_rows_bytes(rows: int, cols: int) -> int:
    return int(lib().fs_fp8_rows_bytes(rows, cols))


def fs_quantize_rows_fp8(rows, cols, x, q, stream=None):
    _check(lib().fs_quantize_rows_fp8(rows, cols, _p(x), _p(q), _stream(stream)), "fs_quantize_rows_fp8")


def fs_mx_rows_bytes(rows: int, cols: int) -> int:
    return int(lib().fs_mx_rows_bytes(rows, cols))


def fs_quantize_rows_mx(rows, cols, x, q, stream=None):
    _check(lib().fs_quantize_rows_mx(rows, cols, _p(x), _p(q), _stream(stream)), "fs_quantize_rows_mx")


def fs_mx4_rows_bytes(rows: int, cols: int) -> int:
    return int(lib().fs_mx4_rows_bytes(rows, cols))


def mx4_rows_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A byte buffer for a 4-bit MX matrix [rows, cols] (codes, then block-scale chunks)."""
    n = fs_mx4_rows_bytes(rows, cols)
    if n == 0:
        raise FsError(1, "fs_mx4_rows_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def mx4_rows_split(buf: torch.Tensor, rows: int, cols: int):
    """Views (code bytes [rows128, cols / 2], scale bytes [rows128 / 128, cols / 128, 512]) of a 4-bit MX matrix."""
    r128 = (rows + 127) // 128 * 128
    off = (r128 * cols // 2 + 255) // 256 * 256
    return (buf[:r128 * cols // 2].view(r128, cols // 2),
            buf[off:off + r128 // 128 * cols // 128 * 512].view(r128 // 128, cols // 128, 512))


def _mx4_bytes(rows, cols):
    """fs_mx4_rows_bytes of valid sizes (other sizes the entry points refuse), without a call into the library."""
    r128 = (rows + 127) // 128
    return (r128 * 64 * cols + 255) // 256 * 256 + r128 * (cols // 128) * 512


def fs_quantize_rows_mx4(rows, cols, x, q, stream=None):
    """Quantise bf16 rows x [rows, cols] into q, a 4-bit MX matrix (mx4_rows_empty)."""
    dev, st = _here(stream)
    what = "fs_quantize_rows_mx4"
    xp, qp = _ptrs(what, dev, (("x", x, (rows, cols), torch.bfloat16), ("q", q, (_mx4_bytes(rows, cols),), torch.uint8)))
    _check(lib().fs_quantize_rows_mx4(rows, cols, xp, qp, st), what)


def pack_linear_mx4(w: torch.Tensor, stream=None) -> torch.Tensor:
    """The FS_MXFP4 pack of a bf16 weight [N, K] for fs_linear_mx4."""
    N, K = w.shape
    dev, _ = _here(stream)
    _operand("pack_linear_mx4 w", w, (N, K), dev, strided=False)
    with _allocating(stream):
        out = _packed(1, N, K, FS_MXFP4, w)
    fs_pack_w3(1, N, K, FS_MXFP4, w, out, stream)
    return out


def fs_linear_mx4_ws_bytes(rows: int, N: int, K: int) -> int:
    return int(lib().fs_linear_mx4_ws_bytes(rows, N, K))


def fs_linear_mx4(q, w, y, K, ws, stream=None):
    """y [rows, N] (bf16 or fp32, any row stride of 16-byte multiples) = the product of the 4-bit MX matrix q [rows, K]
    with the pack w of a weight [N, K]; ws: fs_linear_mx4_ws_bytes(rows, N, K) bytes."""
    dev, st = _here(stream)
    what, (rows, N), u8 = "fs_linear_mx4", y.shape, torch.uint8
    f32 = y.dtype is torch.float32
    yp, ys = _operand("fs_linear_mx4 y", y, (rows, N), dev, torch.float32 if f32 else torch.bfloat16)
    tiles = (N + 255) // 256
    qp, wp, sp = _ptrs(what, dev, (("q", q, (_mx4_bytes(rows, K),), u8),
                                   ("w", w, (tiles * ((K + 255) // 256 * 32768 + K // 128 * 1024),), u8),
                                   ("ws", ws, ws.shape, u8)))
    _check(lib().fs_linear_mx4(rows, N, K, qp, wp, yp, FS_F32 if f32 else FS_BF16, ys[0] if rows > 1 else max(ys[0], N),
                               sp, ws.numel(), st), what)


def fs_dispatch_rows(desc) -> int:
    return int(lib().fs_dispatch_rows(ctypes.byref(desc)))


def mx_rows_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A byte buffer for an MX matrix [rows, cols] (codes, then block-scale chunks)."""
    return torch.empty(fs_mx_rows_bytes(rows, cols), dtype=torch.uint8, device=device)


def mx_rows_split(buf: torch.Tensor, rows: int, cols: int):
    """Views (codes [rows128, cols] uint8, scale bytes [rows128 / 128, cols / 128, 512]) of an MX matrix."""
    r128 = (rows + 127) // 128 * 128
    off = (r128 * cols + 255) // 256 * 256
    return (buf[:r128 * cols].view(r128, cols),
            buf[off:off + r128 // 128 * cols // 128 * 512].view(r128 // 128, cols // 128, 512))


def fp8_rows_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A byte buffer for an FP8 row-scaled matrix [rows, cols] (codes, then scales)."""
    return torch.empty(fs_fp8_rows_bytes(rows, cols), dtype=torch.uint8, device=device)


def fp8_rows_split(buf: torch.Tensor, rows: int, cols: int):
    """Views (codes [rows, cols] uint8, scales [rows] fp32) of an FP8 row-scaled matrix."""
    off = (rows * cols + 255) // 256 * 256
    return buf[:rows * cols].view(rows, cols), buf[off:off + 4 * rows].view(torch.float32)


def fs_router_topk(desc, u, w_r, bias, topk_idx, topk_w, logits, ws, stream=None):
    _check(lib().fs_router_topk(ctypes.byref(desc), _p(u), _p(w_r), _p(bias), _p(topk_idx), _p(topk_w),
                                _p(logits), _p(ws), _nbytes(ws), _stream(stream)), "fs_router_topk")


def fs_dispatch(desc, topk_idx, u, counts, offsets, pos, perm_src, x_perm, ws, stream=None):
    _check(lib().fs_dispatch(ctypes.byref(desc), _p(topk_idx), _p(u), _p(counts), _p(offsets), _p(pos),
                             _p(perm_src), _p(x_perm), _p(ws), _nbytes(ws), _stream(stream)), "fs_dispatch")


def fs_dispatch_noalloc(desc, topk_idx, u, counts, offsets, pos, perm_src, x_perm, stream=None):
    """fs_dispatch with the library's fixed static scratch instead of a workspace
    (for callers that cannot provide device scratch memory)."""
    _check(lib().fs_dispatch_noalloc(ctypes.byref(desc), _p(topk_idx), _p(u), _p(counts), _p(offsets), _p(pos),
                                     _p(perm_src), _p(x_perm), _stream(stream)), "fs_dispatch_noalloc")


def fs_grouped_swiglu(desc, x_perm, offsets, w13, w3, y_perm, ws, stream=None):
    _check(lib().fs_grouped_swiglu(ctypes.byref(desc), _p(x_perm), _p(offsets), _p(w13), _p(w3), _p(y_perm),
                                   _p(ws), _nbytes(ws), _stream(stream)), "fs_grouped_swiglu")


def fs_grouped_swiglu_gather(desc, u, perm_src, offsets, w13, w3, y_perm, ws, stream=None):
    _check(lib().fs_grouped_swiglu_gather(ctypes.byref(desc), _p(u), _p(perm_src), _p(offsets), _p(w13), _p(w3),
                                          _p(y_perm), _p(ws), _nbytes(ws), _stream(stream)),
           "fs_grouped_swiglu_gather")


def fs_shared_expert(desc, u, w13_shared, w3_shared, s_out, ws, stream=None):
    _check(lib().fs_shared_expert(ctypes.byref(desc), _p(u), _p(w13_shared), _p(w3_shared), _p(s_out), _p(ws),
                                  _nbytes(ws), _stream(stream)), "fs_shared_expert")


def _dtype_code(t):
    return FS_BF16 if t.dtype == torch.bfloat16 else FS_F32


def fs_combine(desc, y_perm, pos, topk_w, o_prev, shared_out, o_partial, o_full, u_next=None, wiring="partial",
               extra=None, u_full=None, stream=None):
    """Residual dtypes (bf16 or fp32) are taken from the o_prev and o_full tensors."""
    if o_partial is not None:
        assert o_partial.dtype == o_full.dtype
    w = WIRINGS[wiring] if isinstance(wiring, str) else int(wiring)
    _check(lib().fs_combine(ctypes.byref(desc), _p(y_perm), _p(pos), _p(topk_w), _p(o_prev), _dtype_code(o_prev),
                            _p(shared_out), _p(extra), _p(o_partial), _p(o_full), _dtype_code(o_full), _p(u_next), w,
                            _p(u_full), _stream(stream)), "fs_combine")


def fs_shared_expert_combine(desc, u, w13_shared, w3_shared, y_perm, pos, topk_w, o_prev, o_partial, o_full,
                             u_next=None, wiring="partial", ws=None, stream=None):
    """fs_shared_expert + fs_combine in one pass; residual dtypes from o_prev and o_full."""
    if o_partial is not None:
        assert o_partial.dtype == o_full.dtype
    w = WIRINGS[wiring] if isinstance(wiring, str) else int(wiring)
    _check(lib().fs_shared_expert_combine(ctypes.byref(desc), _p(u), _p(w13_shared), _p(w3_shared), _p(y_perm),
                                          _p(pos), _p(topk_w), _p(o_prev), _dtype_code(o_prev), _p(o_partial),
                                          _p(o_full), _dtype_code(o_full), _p(u_next), w, _p(ws), _nbytes(ws),
                                          _stream(stream)), "fs_shared_expert_combine")


def fs_attn_standin(desc, a, w_att, out, ws, stream=None):
    _check(lib().fs_attn_standin(ctypes.byref(desc), _p(a), _p(w_att), _p(out), _p(ws), _nbytes(ws),
                                 _stream(stream)), "fs_attn_standin")


def block_struct(packed: dict) -> BlockWeights:
    return BlockWeights(_p(packed["w_r"]), _p(packed.get("bias")), _p(packed["w13"]), _p(packed["w3"]),
                        _p(packed.get("w13_shared")), _p(packed.get("w3_shared")), _p(packed.get("w_att")))


def fs_farskip_stack(desc, L, wiring, blocks, x, o_full, o_partial, ws, stream=None):
    """`blocks`: list of L packed-weight dicts (see pack_block)."""
    arr = (BlockWeights * L)(*[block_struct(b) for b in blocks])
    w = WIRINGS[wiring] if isinstance(wiring, str) else int(wiring)
    _check(lib().fs_farskip_stack(ctypes.byref(desc), L, w, arr, _p(x), _p(o_full), _p(o_partial), _p(ws),
                                  _nbytes(ws), _stream(stream)), "fs_farskip_stack")


def fs_workspace_bytes_overlap(desc: LayerDesc, L: int) -> int:
    return int(lib().fs_workspace_bytes_overlap(ctypes.byref(desc), L))


def fs_farskip_stack_overlap(desc, L, wiring, blocks, x, o_full, o_partial, ws, stream=None, stream2=None):
    """Two-stream stack: `stream2` (a torch.cuda.Stream) runs router/dispatch/shared."""
    arr = (BlockWeights * L)(*[block_struct(b) for b in blocks])
    w = WIRINGS[wiring] if isinstance(wiring, str) else int(wiring)
    _check(lib().fs_farskip_stack_overlap(ctypes.byref(desc), L, w, arr, _p(x), _p(o_full), _p(o_partial), _p(ws),
                                          _nbytes(ws), _stream(stream), _stream(stream2)),
           "fs_farskip_stack_overlap")


def fs_get_error():
    code = ctypes.c_int32(0)
    st = lib().fs_get_error(ctypes.byref(code))
    return int(st), int(code.value)


def fs_selftest_wait_timeout(limit_us: int, stream=None):
    _check(lib().fs_selftest_wait_timeout(limit_us, _stream(stream)), "fs_selftest_wait_timeout")


def fs_launch_count() -> int:
    return int(lib().fs_launch_count())


# -------------------------------------------------------------- conveniences

def fs_workspace_bytes_attn(desc: LayerDesc, L: int) -> int:
    return int(lib().fs_workspace_bytes_attn(ctypes.byref(desc), L))


def alloc_workspace(desc: LayerDesc, L: int, device="cuda", attn: bool = False) -> torch.Tensor:
    n = fs_workspace_bytes_attn(desc, L) if attn else fs_workspace_bytes(desc, L)
    if n == 0:
        raise FsError(1, "fs_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _packed(G, N, K, dt, like):
    n = fs_packed_bytes(G, N, K, dt)
    if n == 0:
        raise FsError(1, "fs_packed_bytes")
    if dt in (FS_FP8, FS_MXFP8, FS_MXFP4):
        return torch.empty(n, dtype=torch.uint8, device=like.device)
    return torch.empty(n // like.element_size(), dtype=like.dtype, device=like.device)


def pack_block(cfg: LayerConfig, w: dict, stream=None) -> dict:
    """Repack one block's page-layout weights (on the GPU) into the library layout
    (FP8: quantised from the bf16 weights)."""
    with _allocating(stream):               # copies of strided weights live and die in the order of the packs
        dt = DTYPES[cfg.dtype]
        E, c, d = cfg.E, cfg.c, cfg.d
        out = {"w_r": w["w_r"].contiguous(), "bias": None if w.get("bias") is None else w["bias"].contiguous().float()}
        out["w13"] = _packed(E, 2 * c, d, dt, w["w1"])
        fs_pack_w13(E, c, d, dt, w["w1"].contiguous(), w["w2"].contiguous(), out["w13"], stream)
        out["w3"] = _packed(E, d, c, dt, w["w3"])
        fs_pack_w3(E, d, c, dt, w["w3"].contiguous(), out["w3"], stream)
        if w.get("w_att") is not None:
            out["w_att"] = w["w_att"].contiguous()
        if cfg.n_shared:
            cw = cfg.n_shared * cfg.c_shared
            out["w13_shared"] = _packed(1, 2 * cw, d, dt, w["w1s"])
            fs_pack_w13(1, cw, d, dt, w["w1s"].contiguous(), w["w2s"].contiguous(), out["w13_shared"], stream)
            out["w3_shared"] = _packed(1, d, cw, dt, w["w3s"])
            fs_pack_w3_shared(cfg.n_shared, cfg.c_shared, d, dt, w["w3s"].contiguous(), out["w3_shared"], stream)
    return out


class FarSkipStack:
    """L FarSkip MoE blocks on one GPU: packed weights + workspace, one
    fs_farskip_stack call per forward."""

    def __init__(self, cfg: LayerConfig, raw_blocks: list, wiring: str | None = None, T: int | None = None,
                 device="cuda"):
        self.cfg = cfg
        self.T = cfg.T if T is None else T
        self.wiring = wiring or cfg.wiring
        self.desc = make_desc(cfg, self.T)
        self.blocks = [pack_block(cfg, b) for b in raw_blocks]
        self.ws = alloc_workspace(self.desc, len(self.blocks), device, attn=self.wiring.startswith("attn"))
        dt = torch.float32 if cfg.dtype == "f32" else torch.bfloat16
        self.o_full = torch.empty((self.T, cfg.d), dtype=dt, device=device)
        self.o_partial = torch.empty((self.T, cfg.d), dtype=dt, device=device)

    def forward(self, x: torch.Tensor, stream=None):
        fs_farskip_stack(self.desc, len(self.blocks), self.wiring, self.blocks, x, self.o_full, self.o_partial,
                         self.ws, stream)
        return self.o_full, self.o_partial

    def capture(self, x: torch.Tensor, overlap: bool = False):
        """Record one forward (the library's launches for all L blocks, reading x and
        writing o_full, o_partial) into a CUDA graph; replay() re-runs it.  Warm the
        stack up (one eager forward) first so that one-time setup happens outside
        the capture."""
        self.graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream(device=self.o_full.device)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(self.graph, stream=s):
                if overlap:
                    self.forward_overlap(x, stream=s)
                else:
                    self.forward(x, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        return self.graph

    def replay(self):
        """Re-run the captured forward (same x buffer, same outputs)."""
        self.graph.replay()
        return self.o_full, self.o_partial

    def forward_overlap(self, x: torch.Tensor, stream=None):
        """Two-stream FarSkip schedule (partial/outdated wiring)."""
        if not hasattr(self, "ws_overlap"):
            n = fs_workspace_bytes_overlap(self.desc, len(self.blocks))
            self.ws_overlap = torch.empty(n, dtype=torch.uint8, device=self.o_full.device)
            self.stream2 = torch.cuda.Stream(device=self.o_full.device)
        fs_farskip_stack_overlap(self.desc, len(self.blocks), self.wiring, self.blocks, x, self.o_full,
                                 self.o_partial, self.ws_overlap, stream, self.stream2)
        return self.o_full, self.o_partial


# ------------------------------------------------------------------ training

def fs_train_saved_bytes(desc: LayerDesc, L: int) -> int:
    return int(lib().fs_train_saved_bytes(ctypes.byref(desc), L))


def fs_workspace_bytes_backward(desc: LayerDesc, L: int) -> int:
    return int(lib().fs_workspace_bytes_backward(ctypes.byref(desc), L))


def fs_pack_w13t(G, c, d, w1, w2, out, stream=None):
    _check(lib().fs_pack_w13t(G, c, d, _p(w1), _p(w2), _p(out), _stream(stream)), "fs_pack_w13t")


def fs_pack_w3t(G, d, c, w3, out, stream=None):
    _check(lib().fs_pack_w3t(G, d, c, _p(w3), _p(out), _stream(stream)), "fs_pack_w3t")


def fs_pack_w3t_shared(n_shared, c_shared, d, w3s, out, stream=None):
    _check(lib().fs_pack_w3t_shared(n_shared, c_shared, d, _p(w3s), _p(out), _stream(stream)), "fs_pack_w3t_shared")


def fs_pack_wrt(E, d, w_r, out, stream=None):
    _check(lib().fs_pack_wrt(E, d, _p(w_r), _p(out), _stream(stream)), "fs_pack_wrt")


def pack_block_t(cfg: LayerConfig, w: dict, stream=None) -> dict:
    """Transposed packs of one block's bf16 weights for the input-gradient GEMMs."""
    with _allocating(stream):               # copies of strided weights live and die in the order of the packs
        E, c, d = cfg.E, cfg.c, cfg.d
        epad = (E + 63) // 64 * 64
        out = {"w13t": _packed(E, d, 2 * c, FS_BF16, w["w1"]), "w3t": _packed(E, c, d, FS_BF16, w["w3"]),
               "w_rt": _packed(1, d, epad, FS_BF16, w["w_r"])}
        fs_pack_w13t(E, c, d, w["w1"].contiguous(), w["w2"].contiguous(), out["w13t"], stream)
        fs_pack_w3t(E, d, c, w["w3"].contiguous(), out["w3t"], stream)
        fs_pack_wrt(E, d, w["w_r"].contiguous(), out["w_rt"], stream)
        if cfg.n_shared:
            cw = cfg.n_shared * cfg.c_shared
            out["w13t_shared"] = _packed(1, d, 2 * cw, FS_BF16, w["w1s"])
            out["w3t_shared"] = _packed(1, cw, d, FS_BF16, w["w3s"])
            fs_pack_w13t(1, cw, d, w["w1s"].contiguous(), w["w2s"].contiguous(), out["w13t_shared"], stream)
            fs_pack_w3t_shared(cfg.n_shared, cfg.c_shared, d, w["w3s"].contiguous(), out["w3t_shared"], stream)
    return out


def _block_t_struct(p: dict) -> BlockWeightsT:
    return BlockWeightsT(_p(p["w13t"]), _p(p["w3t"]), _p(p.get("w13t_shared")), _p(p.get("w3t_shared")),
                         _p(p["w_rt"]))


def _grads_struct(g: dict) -> BlockGrads:
    return BlockGrads(*[_p(g.get(k)) for k in ("dW_R", "dW1", "dW2", "dW3", "dW1s", "dW2s", "dW3s")])


def make_balance(T: int, E: int, k: int, gate: str, n_seqs: int = 1, coef: float = 1.0) -> BalanceDesc:
    return BalanceDesc(T, E, k, GATES[gate], n_seqs, coef)


def _balance_shapes(d):
    """Shapes of logits, indices, borders, mask, bias, counts, tokens, from the fields as they are now: the library
    reads these, and they may have changed since the descriptor was made."""
    T, E, S = d.T, d.E, d.n_seqs
    return (T, E), (T, d.k), (S + 1,), (T,), (E,), (S, E), (S,)


def fs_balance_ws_bytes(desc: BalanceDesc) -> int:
    return int(lib().fs_balance_ws_bytes(ctypes.byref(desc)))


def _logit_rows(what, t, shape, dev):
    """(pointer, row stride) of a [T, E] fp32 operand with any row stride."""
    p, st = _operand(what, t, shape, dev, torch.float32)
    return p, st[0] if shape[0] > 1 else max(st[0], shape[1])


def fs_balance_loss(desc: BalanceDesc, logits, topk_idx, counts, tokens, probs, loss, ws, bias=None, cu=None, mask=None,
                    stream=None):
    """Balance loss of router logits [T, E] (fp32, any row stride) and top-k indices [T, k] int32: counts [S, E] and
    tokens [S] int32, probs [S, E] and loss [1] fp32; cu [S + 1] int32 borders and mask [T] uint8 optional;
    ws: fs_balance_ws_bytes(desc) bytes."""
    dev, st = _here(stream)
    what, f32, i32, u8 = "fs_balance_loss", torch.float32, torch.int32, torch.uint8
    te, tk, s1, t1, e1, se, s = _balance_shapes(desc)
    zp, zr = _logit_rows("fs_balance_loss logits", logits, te, dev)
    bp, ip, cp, mp, np_, tp, pp, lp, wp = _ptrs(what, dev, (
        ("bias", bias, e1, f32), ("topk_idx", topk_idx, tk, i32), ("cu", cu, s1, i32), ("mask", mask, t1, u8),
        ("counts", counts, se, i32), ("tokens", tokens, s, i32), ("probs", probs, se, f32), ("loss", loss, _ONE, f32),
        ("ws", ws, ws.shape, u8)))
    _check(lib().fs_balance_loss(desc, zp, zr, bp, ip, cp, mp, np_, tp, pp, lp, wp, ws.numel(), st), what)


def fs_balance_loss_backward(desc: BalanceDesc, logits, counts, tokens, d_loss, d_logits, bias=None, cu=None, mask=None,
                             stream=None):
    """d_logits [T, E] fp32 from fs_balance_loss's counts and tokens and d_loss [1] (None: 1)."""
    dev, st = _here(stream)
    what, f32, i32 = "fs_balance_loss_backward", torch.float32, torch.int32
    te, _, s1, t1, e1, se, s = _balance_shapes(desc)
    zp, zr = _logit_rows("fs_balance_loss_backward logits", logits, te, dev)
    dp, dr = _logit_rows("fs_balance_loss_backward d_logits", d_logits, te, dev)
    bp, cp, mp, np_, tp, gp = _ptrs(what, dev, (
        ("bias", bias, e1, f32), ("cu", cu, s1, i32), ("mask", mask, t1, torch.uint8), ("counts", counts, se, i32),
        ("tokens", tokens, s, i32), ("d_loss", d_loss, _ONE, f32)))
    _check(lib().fs_balance_loss_backward(desc, zp, zr, bp, cp, mp, np_, tp, gp, dp, dr, st), what)


NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5      # coefficients (a, b, c) of the usual five steps


def make_orthogonalize(batch: int, m: int, n: int, dtype: str = "f32", scale: float = 1.0, coefs=NEWTON_SCHULZ,
                       eps: float = 1e-7) -> OrthogonalizeDesc:
    """Steps of (a, b, c) on a batch of [m, n] matrices of type dtype ("f32" or "bf16")."""
    flat = [float(x) for abc in coefs for x in abc]
    if len(flat) > 48 or len(flat) != 3 * len(coefs):
        raise FsError(1, "make_orthogonalize", "%d steps, at most 16 of three coefficients" % len(coefs))
    return OrthogonalizeDesc(batch, m, n, DTYPES[dtype], len(coefs), eps, scale, (ctypes.c_float * 48)(*flat))


def fs_orthogonalize_ws_bytes(desc: OrthogonalizeDesc) -> int:
    return int(lib().fs_orthogonalize_ws_bytes(ctypes.byref(desc)))


def fs_orthogonalize(desc: OrthogonalizeDesc, g, out, ws, stream=None):
    """out [batch, m, n] bf16 = the orthogonalised g [batch, m, n] (fp32 or bf16 as desc says; any row and matrix
    strides); ws: fs_orthogonalize_ws_bytes(desc) bytes."""
    dev, st = _here(stream)
    what, shape = "fs_orthogonalize", (desc.batch, desc.m, desc.n)
    gp, gs = _operand(what + " g", g, shape, dev, torch.float32 if desc.dtype == FS_F32 else torch.bfloat16)
    op, os_ = _operand(what + " out", out, shape, dev)
    wp, _ = _operand(what + " ws", ws, ws.shape, dev, torch.uint8, False)
    row = lambda s: s[1] if desc.m > 1 else max(s[1], desc.n)
    _check(lib().fs_orthogonalize(desc, gp, row(gs), gs[0], op, row(os_), os_[0], wp, ws.numel(), st), what)


class FarSkipTrainer:
    """Forward (keeping what the backward reads) and backward of an L-block
    FarSkip MoE stack on one GPU (bf16, MoE wirings): two library calls."""

    def __init__(self, cfg: LayerConfig, raw_blocks: list, wiring: str | None = None, T: int | None = None,
                 device="cuda"):
        self.cfg = cfg
        self.T = cfg.T if T is None else T
        self.wiring = wiring or cfg.wiring
        self.desc = make_desc(cfg, self.T)
        L = len(raw_blocks)
        self.L = L
        self.blocks = [pack_block(cfg, b) for b in raw_blocks]
        self.blocks_t = [pack_block_t(cfg, b) for b in raw_blocks]
        self.saved = torch.empty(fs_train_saved_bytes(self.desc, L), dtype=torch.uint8, device=device)
        self.ws = alloc_workspace(self.desc, L, device)
        self.ws_b = torch.empty(fs_workspace_bytes_backward(self.desc, L), dtype=torch.uint8, device=device)
        E, c, d, ns, cs = cfg.E, cfg.c, cfg.d, cfg.n_shared, cfg.c_shared
        f32 = dict(dtype=torch.float32, device=device)
        self.grads = []
        for _ in range(L):
            g = {"dW_R": torch.empty((E, d), **f32), "dW1": torch.empty((E, c, d), **f32),
                 "dW2": torch.empty((E, c, d), **f32), "dW3": torch.empty((E, d, c), **f32)}
            if ns:
                g.update(dW1s=torch.empty((ns, cs, d), **f32), dW2s=torch.empty((ns, cs, d), **f32),
                         dW3s=torch.empty((ns, d, cs), **f32))
            self.grads.append(g)
        self.o_full = torch.empty((self.T, d), dtype=torch.bfloat16, device=device)
        self.o_partial = torch.empty((self.T, d), dtype=torch.bfloat16, device=device)
        self.dx = torch.empty((self.T, d), **f32)

    def forward(self, x: torch.Tensor, stream=None):
        self.bal_ready = False              # the balance loss belongs to one forward
        arr = (BlockWeights * self.L)(*[block_struct(b) for b in self.blocks])
        _check(lib().fs_farskip_stack_train(ctypes.byref(self.desc), self.L, WIRINGS[self.wiring], arr, _p(x),
                                            _p(self.o_full), _p(self.o_partial), _p(self.saved), _nbytes(self.saved),
                                            _p(self.ws), _nbytes(self.ws), _stream(stream)), "fs_farskip_stack_train")
        return self.o_full, self.o_partial

    def balance_loss(self, coef: float, cu: torch.Tensor | None = None, mask: torch.Tensor | None = None, stream=None):
        """Balance loss of every block's router in the last forward: loss [L, 1] fp32 and counts [L, S, E] int32 (also
        kept for backward's d_balance).  cu [S + 1] int32: sequence borders; mask [T] uint8: 0 leaves a token out."""
        cfg, S, dev = self.cfg, 1 if cu is None else cu.shape[0] - 1, self.o_full.device
        desc = make_balance(self.T, cfg.E, cfg.k, cfg.gate, S, coef)
        n = fs_balance_ws_bytes(desc)
        if n == 0:
            raise FsError(1, "fs_balance_ws_bytes")
        self.bal_ready = False
        cur, st = _here(stream)
        cp = None if cu is None else _operand("balance_loss cu", cu, (S + 1,), cur, torch.int32, False)[0]
        mp = None if mask is None else _operand("balance_loss mask", mask, (self.T,), cur, torch.uint8, False)[0]
        b = getattr(self, "bal", None)
        if b is None or b["counts"].shape[1] != S:
            i32, f32 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.float32, device=dev)
            with _allocating(stream):
                b = {"counts": torch.empty((self.L, S, cfg.E), **i32), "tokens": torch.empty((self.L, S), **i32),
                     "probs": torch.empty((self.L, S, cfg.E), **f32), "loss": torch.empty((self.L, 1), **f32),
                     "d_logits": torch.empty((self.L, self.T, cfg.E), **f32),
                     "ws": torch.empty(n, dtype=torch.uint8, device=dev)}
        b.update(desc=desc, cu=cu, mask=mask)
        self.bal = b
        for blk in range(self.L):
            z, idx = self._routing(blk)
            _check(lib().fs_balance_loss(desc, z, cfg.E, _p(self.blocks[blk]["bias"]), idx, cp, mp,
                                         _p(b["counts"][blk]), _p(b["tokens"][blk]), _p(b["probs"][blk]),
                                         _p(b["loss"][blk]), _p(b["ws"]), n, st), "fs_balance_loss")
        self.bal_ready = True
        return b["loss"], b["counts"]

    def _routing(self, blk: int):
        z, idx = _VP(), _VP()
        _check(lib().fs_train_saved_routing(ctypes.byref(self.desc), self.L, blk, _p(self.saved), ctypes.byref(z),
                                            ctypes.byref(idx)), "fs_train_saved_routing")
        return z, idx

    def backward(self, d_o: torch.Tensor, d_os: torch.Tensor | None = None, stream=None,
                 dx: torch.Tensor | None = None, d_balance: torch.Tensor | None = None):
        """Gradients for the last forward: dx (into `dx` when given, else self.dx)
        and the weight gradients (self.grads).  d_balance [1] fp32 on the device: the gradient of the loss with
        respect to the sum of balance_loss's losses, which then goes into the routers' gradients."""
        out = self.dx if dx is None else dx
        arr = (BlockWeights * self.L)(*[block_struct(b) for b in self.blocks])
        arr_t = (BlockWeightsT * self.L)(*[_block_t_struct(b) for b in self.blocks_t])
        gr = (BlockGrads * self.L)(*[_grads_struct(g) for g in self.grads])
        head = (ctypes.byref(self.desc), self.L, WIRINGS[self.wiring], arr, arr_t, _p(self.saved), _nbytes(self.saved),
                _p(d_o), _p(d_os))
        tail = (_p(out), gr, _p(self.ws_b), _nbytes(self.ws_b), _stream(stream))
        if d_balance is None:
            _check(lib().fs_farskip_stack_backward(*head, *tail), "fs_farskip_stack_backward")
            return out, self.grads
        if not getattr(self, "bal_ready", False):
            raise FsError(1, "backward", "d_balance without a balance_loss of the last forward")
        b = self.bal
        cur, st = _here(stream)
        gp, _ = _operand("backward d_balance", d_balance, (1,), cur, torch.float32, False)
        if b["cu"] is not None:             # rows outside every sequence are not written, and may have been inside one
            with _allocating(stream):
                b["d_logits"].zero_()
        extra = (_VP * self.L)()
        for blk in range(self.L):
            z, _ = self._routing(blk)
            extra[blk] = b["d_logits"][blk].data_ptr()
            _check(lib().fs_balance_loss_backward(b["desc"], z, self.cfg.E, _p(self.blocks[blk]["bias"]), _p(b["cu"]),
                                                  _p(b["mask"]), _p(b["counts"][blk]), _p(b["tokens"][blk]), gp,
                                                  extra[blk], self.cfg.E, st), "fs_balance_loss_backward")
        _check(lib().fs_farskip_stack_backward_aux(*head, extra, *tail), "fs_farskip_stack_backward_aux")
        return out, self.grads

    def orthogonalized(self, names=("dW1", "dW2", "dW3"), scale: float = 1.0, coefs=NEWTON_SCHULZ, eps: float = 1e-7,
                       stream=None):
        """The orthogonalised updates (bf16) of every block's weight gradients of these names: a list of dicts like
        self.grads.  Each expert's matrix is one of a batch."""
        updates = []
        for blk in range(self.L):
            upd = {}
            for name in names:
                g = self.grads[blk][name]
                g3 = g if g.dim() == 3 else g[None]
                desc = make_orthogonalize(*g3.shape, "f32", scale, coefs, eps)
                need = fs_orthogonalize_ws_bytes(desc)
                if need == 0:
                    raise FsError(1, "fs_orthogonalize_ws_bytes")
                with _allocating(stream):
                    if getattr(self, "ws_o", None) is None or self.ws_o.numel() < need:
                        self.ws_o = torch.empty(need, dtype=torch.uint8, device=g.device)
                    upd[name] = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
                fs_orthogonalize(desc, g3, upd[name].view(g3.shape), self.ws_o, stream)
            updates.append(upd)
        return updates


# ----------------------------------------------------------------- attention

ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
LATENT, ROPE_DIM, NOPE_DIM, V_DIM = 512, 64, 128, 128      # widths of the latent-attention operators
LATENT_RECORD = {"bf16": 2 * (LATENT + ROPE_DIM), "fp8": LATENT + 2 * ROPE_DIM + 16}      # bytes per cached token


def _here(stream):
    """(current device, raw stream) of a call, without building a Stream object when none is given."""
    try:
        dev = torch.cuda.current_device()
    except (RuntimeError, AssertionError) as e:
        raise FsError(4, "current device", str(e)) from None
    if stream is not None and stream.device_index != dev:
        raise FsError(1, "stream", "of cuda:%d, not of the current device" % stream.device_index)
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _allocating(stream):
    """Context in which torch allocates, fills and recycles memory in the order of the call's stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _operand(what: str, t: torch.Tensor, shape, dev: int, dtype=torch.bfloat16, strided=True):
    """Refuse a tensor whose shape, type, inner stride or device the call could not take: the C entry sees only a
    pointer.  Returns (pointer, strides)."""
    st = t.stride()
    if t.shape != shape or t.dtype is not dtype:
        raise FsError(1, what, "got %s %s, expected %s %s" % (tuple(t.shape), t.dtype, tuple(shape), dtype))
    if (st[-1] != 1 and shape[-1] > 1) or not (strided or t.is_contiguous()):
        raise FsError(1, what, "strides %s" % (st,))
    if t.get_device() != dev:
        raise FsError(1, what, "tensor on %s, not on the current device" % t.device)
    return t.data_ptr(), st


_ONE = (1,)


def _ptrs(what: str, dev: int, specs):
    """Pointers of contiguous operands (name, tensor or None, shape, type), refused as by _operand."""
    out = []
    for name, t, shape, dtype in specs:
        if t is None:
            out.append(None)
        elif t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev:
            out.append(t.data_ptr())
        else:
            out.append(_operand("%s %s" % (what, name), t, shape, dev, dtype, False)[0])
    return out


def _rows(ptr_strides) -> Rows:
    """(pointer, strides) of [rows, heads, width] or [rows, width] -> (pointer, row stride, head stride)."""
    p, st = ptr_strides
    return Rows(p, st[0], st[1] if len(st) == 3 else 0)


def make_rope(d_rot: int, layout: str = "interleaved", base: float = 10000.0, factor: float = 1.0,
              orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, mscale: float = 1.0) -> RopeDesc:
    return RopeDesc(d_rot, ROPE_LAYOUTS[layout], base, factor, orig_len, beta_fast, beta_slow, mscale)


def fs_rope(rope: RopeDesc, pos, x, y, inverse: bool = False, stream=None):
    """Rotate x [T, H, d_rot] (a view of the rotated part of each head) into y (which may be x)."""
    dev, st = _here(stream)
    T, H, _ = x.shape
    f32 = x.dtype is torch.float32
    dt = torch.float32 if f32 else torch.bfloat16
    xp, xs = _operand("fs_rope x", x, (T, H, rope.d_rot), dev, dt)
    yp, ys = _operand("fs_rope y", y, (T, H, rope.d_rot), dev, dt)
    pp, _ = _operand("fs_rope pos", pos, (T,), dev, torch.int32)
    _check(lib().fs_rope(rope, T, H, FS_F32 if f32 else FS_BF16, pp, xp, xs[0], xs[1], yp, ys[0], ys[1], inverse,
                         st), "fs_rope")


def make_latent_cache(n_pages: int, page_size: int, dtype: str = "bf16") -> LatentCache:
    return LatentCache(n_pages, page_size, DTYPES[dtype])


def fs_latent_cache_bytes(desc: LatentCache) -> int:
    return int(lib().fs_latent_cache_bytes(ctypes.byref(desc)))


def latent_cache_empty(desc: LatentCache, device="cuda") -> torch.Tensor:
    """A cache tensor: [n_pages, page_size, 576] bf16, or [n_pages, page_size, 656] bytes for FP8."""
    if fs_latent_cache_bytes(desc) == 0:
        raise FsError(1, "fs_latent_cache_bytes")
    if desc.dtype == FS_BF16:
        return torch.empty((desc.n_pages, desc.page_size, LATENT + ROPE_DIM), dtype=torch.bfloat16, device=device)
    return torch.empty((desc.n_pages, desc.page_size, LATENT_RECORD["fp8"]), dtype=torch.uint8, device=device)


def _cache_operand(what, desc, cache, dev):
    if desc.dtype == FS_FP8:
        return _operand(what, cache, (desc.n_pages, desc.page_size, LATENT_RECORD["fp8"]), dev, torch.uint8, False)[0]
    return _operand(what, cache, (desc.n_pages, desc.page_size, LATENT + ROPE_DIM), dev, torch.bfloat16, False)[0]


def fs_latent_cache_write(desc: LatentCache, c, k_rope, slots, cache, rope: RopeDesc | None = None, pos=None,
                          stream=None):
    """Write c [T, 512], k_rope [T, 64] (rotated by rope at pos when given) to the slots [T] (int64; negative: skipped)."""
    dev, st = _here(stream)
    T, what = c.shape[0], "fs_latent_cache_write"
    cp, cs = _operand("fs_latent_cache_write c", c, (T, LATENT), dev)
    kp, ks = _operand("fs_latent_cache_write k_rope", k_rope, (T, ROPE_DIM), dev)
    sp, _ = _operand("fs_latent_cache_write slots", slots, (T,), dev, torch.int64)
    pp = None if pos is None else _operand("fs_latent_cache_write pos", pos, (T,), dev, torch.int32)[0]
    _check(lib().fs_latent_cache_write(desc, T, cp, cs[0], kp, ks[0], rope, pp, sp,
                                       _cache_operand("fs_latent_cache_write cache", desc, cache, dev),
                                       st), what)


def fs_latent_cache_read(desc: LatentCache, cache, slots, c, k_rope, stream=None):
    """Read the records of slots [T] back into c [T, 512], k_rope [T, 64] (rows with a negative slot are left)."""
    dev, st = _here(stream)
    T, what = slots.shape[0], "fs_latent_cache_read"
    sp, _ = _operand("fs_latent_cache_read slots", slots, (T,), dev, torch.int64)
    cp, cs = _operand("fs_latent_cache_read c", c, (T, LATENT), dev)
    kp, ks = _operand("fs_latent_cache_read k_rope", k_rope, (T, ROPE_DIM), dev)
    _check(lib().fs_latent_cache_read(desc, _cache_operand("fs_latent_cache_read cache", desc, cache, dev), T, sp, cp, cs[0],
                                      kp, ks[0], st), what)


def fs_latent_decode_ws_bytes(heads: int, B: int, n_q: int = 1) -> int:
    return int(lib().fs_latent_decode_ws_bytes(heads, B, n_q))


def fs_latent_decode(desc: LatentCache, q_latent, q_rope, cache, block_table, seq_lens, scale, out, lse, ws,
                     stream=None):
    """Absorbed attention of the newest n_q tokens of B sequences: q_latent [B n_q, H, 512], q_rope [B n_q, H, 64],
    block_table [B, max_pages] int32, seq_lens [B] int32 -> out [B n_q, H, 512], lse [B n_q, H] (or None);
    ws: fs_latent_decode_ws_bytes(H, B, n_q) bytes."""
    dev, st = _here(stream)
    rows, H, _ = q_latent.shape
    B, max_pages = block_table.shape
    n_q = rows // max(B, 1)
    rows = B * n_q
    ql = _rows(_operand("fs_latent_decode q_latent", q_latent, (rows, H, LATENT), dev))
    qr = _rows(_operand("fs_latent_decode q_rope", q_rope, (rows, H, ROPE_DIM), dev))
    op = _rows(_operand("fs_latent_decode out", out, (rows, H, LATENT), dev))
    tp, ts = _operand("fs_latent_decode block_table", block_table, (B, max_pages), dev, torch.int32)
    lp, _ = _operand("fs_latent_decode seq_lens", seq_lens, (B,), dev, torch.int32)
    ep = None if lse is None else _operand("fs_latent_decode lse", lse, (rows, H), dev, torch.float32, False)[0]
    wp, _ = _operand("fs_latent_decode ws", ws, ws.shape, dev, torch.uint8, False)
    _check(lib().fs_latent_decode(desc, H, B, n_q, ql, qr, _cache_operand("fs_latent_decode cache", desc, cache, dev), tp,
                                  max_pages, ts[0], lp, scale, op, ep, wp, ws.numel(), st),
           "fs_latent_decode")


def _prefill_operands(what, dev, q, k_nope, k_rope, v, cu_q, cu_k, causal, scale):
    """The descriptor and the operands that the forward and the backward share."""
    (Tq, H, _), Tk, B = q.shape, k_rope.shape[0], cu_q.shape[0] - 1
    return (LatentPrefillDesc(H, B, Tq, Tk, bool(causal), scale),
            _rows(_operand(what, q, (Tq, H, NOPE_DIM + ROPE_DIM), dev)), _rows(_operand(what, k_nope, (Tk, H, NOPE_DIM), dev)),
            _rows(_operand(what, k_rope, (Tk, ROPE_DIM), dev)), _rows(_operand(what, v, (Tk, H, V_DIM), dev)),
            _operand(what, cu_q, (B + 1,), dev, torch.int32)[0], _operand(what, cu_k, (B + 1,), dev, torch.int32)[0])


def fs_latent_prefill(q, k_nope, k_rope, v, cu_q, cu_k, causal, scale, out, lse, stream=None):
    """Expanded attention over packed sequences: q [Tq, H, 192], k_nope and v [Tk, H, 128], k_rope [Tk, 64],
    cu_q and cu_k [B + 1] int32 -> out [Tq, H, 128], lse [H, Tq] fp32."""
    what = "fs_latent_prefill"
    dev, st = _here(stream)
    ops = _prefill_operands(what, dev, q, k_nope, k_rope, v, cu_q, cu_k, causal, scale)
    Tq, H, _ = q.shape
    _check(lib().fs_latent_prefill(*ops, _rows(_operand(what, out, (Tq, H, V_DIM), dev)),
                                   _operand(what, lse, (H, Tq), dev, torch.float32, False)[0], st), what)


def fs_latent_prefill_backward_ws_bytes(heads: int, Tq: int, Tk: int) -> int:
    return int(lib().fs_latent_prefill_backward_ws_bytes(heads, Tq, Tk))


def fs_latent_prefill_backward(q, k_nope, k_rope, v, cu_q, cu_k, causal, scale, out, lse, d_out, dq, dk_nope, dk_rope,
                               dv, ws, stream=None):
    """Gradient of fs_latent_prefill from its out and lse: dq, dk_nope, dk_rope (summed over the heads), dv in the
    inputs' shapes; ws: fs_latent_prefill_backward_ws_bytes(H, Tq, Tk) bytes."""
    what = "fs_latent_prefill_backward"
    dev, st = _here(stream)
    ops = _prefill_operands(what, dev, q, k_nope, k_rope, v, cu_q, cu_k, causal, scale)
    Tq, H, _ = q.shape
    grads = [_rows(_operand(what, g, like.shape, dev)) for g, like in ((dq, q), (dk_nope, k_nope), (dk_rope, k_rope), (dv, v))]
    wp, _ = _operand(what, ws, ws.shape, dev, torch.uint8, False)
    _check(lib().fs_latent_prefill_backward(*ops, _rows(_operand(what, out, (Tq, H, V_DIM), dev)),
                                            _operand(what, lse, (H, Tq), dev, torch.float32, False)[0],
                                            _rows(_operand(what, d_out, (Tq, H, V_DIM), dev)), *grads, wp, ws.numel(),
                                            st), what)
