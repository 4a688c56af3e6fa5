"""Weights packed on a stream that is not the current one: buffers and the copies of strided weights belong to that
stream, so that memory which the current stream recycles meanwhile is none that a pack still reads or writes."""
import pytest
import torch

from mixture_experts_layer_expert_gb300 import configs, fs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def strided(block):
    """The same weights with rows that are not dense."""
    def wide(t):
        if t is None or t.dim() < 2:
            return t
        big = torch.full((*t.shape[:-1], t.shape[-1] + 8), 3.0, dtype=t.dtype, device=t.device)
        big[..., :t.shape[-1]] = t
        return big[..., :t.shape[-1]]
    return {k: wide(v) for k, v in block.items()}


def on_a_late_stream(pack):
    """pack(stream) behind work that holds the stream up, while the current stream takes and fills whatever was freed."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = pack(side)
    keep = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22) for _ in range(8)]
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0) and len(keep) == 32
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "mxfp8", "mxfp4"])
def test_blocks(dtype):
    cfg = configs.LayerConfig("packs", T=64, d=256, E=6, k=2, c=128, n_shared=2, c_shared=128, L=1, gate="softmax", dtype=dtype)
    block = strided(synth.make_problem(cfg, device=DEV)["blocks"][0])
    forms = [fs.pack_block] + ([fs.pack_block_t] if dtype == "bf16" else [])
    for form in forms:
        want = form(cfg, block)
        got = on_a_late_stream(lambda s: form(cfg, block, s))
        for k, v in want.items():
            assert (v is None and got[k] is None) or torch.equal(got[k].view(torch.uint8), v.view(torch.uint8)), k


def test_buffers_come_from_the_calls_stream(monkeypatch):
    cfg = configs.LayerConfig("packs", T=64, d=256, E=6, k=2, c=128, n_shared=1, c_shared=128, L=1, gate="softmax", dtype="bf16")
    block = synth.make_problem(cfg, device=DEV)["blocks"][0]
    packed, at = fs._packed, []
    monkeypatch.setattr(fs, "_packed", lambda *a: at.append(torch.cuda.current_stream()) or packed(*a))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w = torch.randn((264, 384), device=DEV).to(torch.bfloat16)
    torch.cuda.synchronize()
    for call in (lambda s: fs.pack_linear_mx4(w, s), lambda s: fs.pack_block(cfg, block, s), lambda s: fs.pack_block_t(cfg, block, s)):
        for stream, want in ((side, side), (None, torch.cuda.current_stream())):
            at.clear()
            call(stream)
            assert at and all(s == want for s in at)
    torch.cuda.synchronize()


def test_dense_weight():
    w = torch.randn((1000, 1408), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    want = fs.pack_linear_mx4(w)
    assert torch.equal(on_a_late_stream(lambda s: fs.pack_linear_mx4(w, s)), want)
