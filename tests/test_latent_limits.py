"""Limits of the attention entry points at the ends of their integer and floating-point ranges, without a GPU: every
refusal comes before any CUDA call."""
import ctypes

import pytest

from mixture_experts_layer_expert_gb300 import build, fs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
V = ctypes.c_void_p(0x10000)            # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = fs.lib()
    before = fs.fs_launch_count()
    yield lib
    assert fs.fs_launch_count() == before


def test_cache_whose_bytes_pass_64_bits(L):
    """(2^31 - 1)^2 records have no byte count: the size is 0 and the calls refuse, not a size modulo 2^64."""
    top = 2 ** 31 - 1
    for dtype, rec in (("bf16", 1152), ("fp8", 656)):
        most = (2 ** 63 - 1) // rec // top                        # pages of 2^31 - 1 records that 63 bits still count
        assert fs.fs_latent_cache_bytes(fs.make_latent_cache(most, top, dtype)) == most * top * rec
        for pages in (most + 1, top):
            big = fs.make_latent_cache(pages, top, dtype)
            assert fs.fs_latent_cache_bytes(big) == 0
            d = ctypes.byref(big)
            assert L.fs_latent_cache_write(d, 4, V, 512, V, 64, None, None, V, V, None) == UNSUPPORTED
            assert L.fs_latent_cache_read(d, V, 4, V, V, 512, V, 64, None) == UNSUPPORTED


def test_rope_mscale_outside_fp32(L):
    """mscale multiplies in fp32: one that would become 0, subnormal or infinite there is refused, one at the range's ends is not
    refused for its value (the misaligned operand behind it is)."""
    def call(mscale, pos):
        rope = ctypes.byref(fs.make_rope(64, mscale=mscale))
        return L.fs_rope(rope, 4, 2, 0, pos, V, 128, 64, V, 128, 64, 0, None)
    for bad in (1e39, 1e300, 1e-40, 1e-46, 5e-324, float("inf"), float("nan"), -1.0):
        assert call(bad, ODD) == INVALID, bad
    for good in (3.4e38, 1.0, 1e-37):
        assert call(good, ODD) == UNSUPPORTED                     # the misaligned pos, checked after the table


def test_prefill_rows_past_the_kernels_index_range(L):
    """Row and key indexes of a packed batch, their differences and tile ends are int32 in the kernels: 2^29 rows of
    queries or keys leave room for all of them, more are refused (one head's rows would pass the card's memory)."""
    top = 2 ** 29
    r = ctypes.byref(fs.Rows(0x10000, 192, 192))
    W = ctypes.c_void_p(0x1000000)
    for Tq, Tk in ((top + 1, 96), (64, top + 1), (2 ** 31 - 1, 2 ** 31 - 1), (top, top)):
        want = UNSUPPORTED if max(Tq, Tk) > top else INVALID
        d = ctypes.byref(fs.LatentPrefillDesc(1, 2, Tq, Tk, 0, 0.1))
        # past the limit refused as such; at it, the missing cu_q is what is refused
        assert L.fs_latent_prefill(d, r, r, r, r, None, V, r, V, None) == want
        assert L.fs_latent_prefill_backward(d, r, r, r, r, None, V, r, V, r, r, r, r, r, W, 1 << 40, None) == want
        assert (fs.fs_latent_prefill_backward_ws_bytes(1, Tq, Tk) == 0) == (want == UNSUPPORTED)
