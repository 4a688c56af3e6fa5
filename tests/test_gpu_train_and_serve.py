"""The balance loss, orthogonalised updates and 4-bit experts as one program: training steps whose gradients take the
balance term, updates by orthogonalised gradients, the updated layer served in 4 bits."""
import dataclasses

import pytest
import torch

import mx4_ref
import ortho_ref
from mixture_experts_layer_expert_gb300 import configs, fs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("dW1", "dW2", "dW3", "dW_R")
WEIGHT = {"dW1": "w1", "dW2": "w2", "dW3": "w3", "dW_R": "w_r"}


def problem():
    cfg = configs.LayerConfig("together", T=192, d=256, E=10, k=3, c=128, n_shared=1, c_shared=128, L=2, gate="sigmoid_norm",
                              dtype="bf16")
    return cfg, synth.make_problem(cfg, device=DEV)


def step(tr, x, d_o, cu, mask, g, stream=None):
    """One step's losses, counts, gradients and updates, in buffers of their own."""
    tr.forward(x, stream=stream)
    loss, counts = tr.balance_loss(0.01, cu=cu, mask=mask, stream=stream)
    dx, grads = tr.backward(d_o, d_balance=g, stream=stream)
    upd = tr.orthogonalized(NAMES, scale=0.2, stream=stream)
    return [loss, counts, dx] + [gr[n] for gr in grads for n in sorted(gr)] + [u[n] for u in upd for n in NAMES], upd


def test_steps_then_four_bits():
    cfg, prob = problem()
    cu = torch.tensor([0, 50, 50, 180], dtype=torch.int32, device=DEV)     # the last rows are padding
    mask = (torch.arange(cfg.T, device=DEV) % 7 != 3).to(torch.uint8)
    g = torch.tensor([30.0], device=DEV)
    d_o = torch.randn((cfg.T, cfg.d), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    blocks, side = prob["blocks"], torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(2):
        tr = fs.FarSkipTrainer(cfg, blocks)
        torch.cuda.synchronize()
        out, upd = step(tr, prob["x"], d_o, cu, mask, g)
        torch.cuda.synchronize()
        assert fs.fs_get_error() == (0, 0)
        want = [t.clone() for t in out]
        counted = int(((mask != 0) & (torch.arange(cfg.T, device=DEV) < 180)).sum())
        assert (out[1].sum((1, 2)) == counted * cfg.k).all() and (out[0] > 0).all()
        # on another stream, and from a graph with its inputs' buffers: the same bits
        with torch.cuda.stream(side):
            again, _ = step(tr, prob["x"], d_o, cu, mask, g, side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held, _ = step(tr, prob["x"], d_o, cu, mask, g)
        for t in held:
            t.fill_(3)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert fs.fs_get_error() == (0, 0)
        new = []
        for blk, b in enumerate(blocks):
            b = dict(b)
            for n in NAMES:
                grad, u = tr.grads[blk][n], upd[blk][n]
                for gm, um in zip(grad if grad.dim() == 3 else grad[None], u if u.dim() == 3 else u[None]):
                    exact, room = ortho_ref.tolerance(gm, scale=0.2)
                    assert float((um.double() - exact).norm()) <= room + 1e-30
                w = b[WEIGHT[n]]
                b[WEIGHT[n]] = (w.float() - 0.1 * u.float()).to(w.dtype)
            new.append(b)
        blocks = new
    assert all(not torch.equal(a["w1"], b["w1"]) for a, b in zip(blocks, prob["blocks"]))

    # served: the updated layer in 4 bits is the bf16 layer up to the rounding of the experts' operands to E2M1
    cfg4 = dataclasses.replace(cfg, dtype="mxfp4")
    o = fs.FarSkipStack(cfg, blocks).forward(prob["x"])[0].clone()
    stack = fs.FarSkipStack(cfg4, blocks)
    o4 = stack.forward(prob["x"])[0].clone()
    stack.capture(prob["x"])
    stack.o_full.zero_()
    stack.replay()
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0) and torch.equal(stack.o_full, o4)
    # three products of operands off by at most a fifth of themselves each (a quarter step below 4 / 6 of a block's largest),
    # with random signs: well under their sum
    assert 0 < float((o4.double() - o.double()).norm()) < 0.6 * float(o.double().norm())

    # and its output projection in 4 bits
    w = blocks[0]["w_r"].to(torch.bfloat16)[:8].contiguous()
    q, y = fs.mx4_rows_empty(cfg.T, cfg.d), torch.empty((cfg.T, 8), device=DEV)
    fs.fs_quantize_rows_mx4(cfg.T, cfg.d, o4, q)
    fs.fs_linear_mx4(q, fs.pack_linear_mx4(w), y, cfg.d, torch.empty(fs.fs_linear_mx4_ws_bytes(cfg.T, 8, cfg.d), dtype=torch.uint8,
                                                                     device=DEV))
    torch.cuda.synchronize()
    a, b = mx4_ref.rounded(o4.cpu().double()), mx4_ref.rounded(w.cpu().double())
    room = (a.abs() @ b.abs().T) * cfg.d * 2.0 ** -23
    assert ((y.cpu().double() - a @ b.T).abs() <= room).all()
