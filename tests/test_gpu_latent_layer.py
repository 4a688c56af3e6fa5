"""The attention operators inside a block, as they are used: projections, rotary positions, the paged cache, expanded
attention for the prompts and absorbed attention for the tokens after them, the output projection, and its result as
fs_combine's fp32 `extra` beside the routed and shared experts.  Every step of ours is checked against its 64-bit
definition on its own inputs; the decode step also as a captured graph with new inputs."""
import math

import pytest
import torch

import latent_ref as ref
import parity
from mixture_experts_layer_expert_gb300 import configs, fs, synth
from test_gpu_latent import DEV, SCALE, SCALED, _no_dev_error, gen, ints

pytestmark = pytest.mark.gpu
H, D, PAGE = 16, 256, 48


@pytest.fixture(autouse=True, scope="module")
def _loaded():
    fs.lib()


class Block:
    def __init__(self, cache):
        g = gen(31)
        w = lambda *s: torch.randn(s, generator=g, device=DEV) / math.sqrt(s[-2])
        self.wq, self.wc, self.wk = w(D, H * 192), w(D, 512), w(D, 64)
        self.w_uk, self.w_uv = (torch.randn((H, 128, 512), generator=g, device=DEV) / math.sqrt(512) for _ in range(2))
        self.wo = w(H * 128, D)
        self.cfg = lambda T: configs.LayerConfig("block", T=T, d=D, E=8, k=2, c=128, n_shared=1, c_shared=128, L=1,
                                                 gate="softmax_renorm", dtype="bf16")
        self.moe = fs.pack_block(self.cfg(1), synth.make_block_weights(self.cfg(1), 0, DEV))
        self.rope = fs.make_rope(64, "interleaved", **SCALED)
        self.desc = fs.make_latent_cache(24, PAGE, cache)
        self.cache = fs.latent_cache_empty(self.desc)
        self.cache.view(torch.uint8).fill_(0x7F)                       # NaN where nothing has been written

    def project(self, x, pos, slots):
        """q with its rotary part turned, the new tokens' records written."""
        T = x.shape[0]
        q = (x.float() @ self.wq).to(torch.bfloat16).view(T, H, 192)
        c, kr = (x.float() @ self.wc).to(torch.bfloat16), (x.float() @ self.wk).to(torch.bfloat16)
        fs.fs_rope(self.rope, pos, q[..., 128:], q[..., 128:])
        fs.fs_latent_cache_write(self.desc, c, kr, slots, self.cache, rope=self.rope, pos=pos)
        return q

    def moe_with(self, run, x, extra):
        """Router, routed and shared experts on x, combined with x and the attention's result."""
        T = x.shape[0]
        fs.fs_router_topk(run.desc, x, self.moe["w_r"], self.moe.get("bias"), run.idx, run.w, None, run.ws)
        fs.fs_dispatch(run.desc, run.idx, x, run.counts, run.offsets, run.pos, run.perm, run.x_perm, run.ws)
        fs.fs_grouped_swiglu(run.desc, run.x_perm, run.offsets, self.moe["w13"], self.moe["w3"], run.y_perm, run.ws)
        fs.fs_shared_expert(run.desc, x, self.moe["w13_shared"], self.moe["w3_shared"], run.s, run.ws)
        o_star, o = (torch.empty((T, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        fs.fs_combine(run.desc, run.y_perm, run.pos, run.w, x, run.s, o_star, o, None, "partial", extra=extra)
        return o_star, o

    def check_block(self, run, x, extra, o_star, o):
        """o* = x + S + A and o = o* + R: fp32 sums of at most six terms, rounded once to bf16."""
        T = x.shape[0]
        y = run.y_perm.double()[run.pos.long().view(T, 2)] * run.w.double()[..., None]
        terms = [x.double(), run.s.double(), extra.double()]
        for got, extra_terms in ((o_star, []), (o, list(y.unbind(1)))):
            t = torch.stack(terms + extra_terms)
            want = t.sum(0)
            ref.within(got, want, ref.HALF * want.abs() + 8 * ref.ULP32 * t.abs().sum(0), "block output")


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_block_prompts_then_tokens(cache):
    blk, g = Block(cache), gen(32)
    lens, pages = [150, 1, 333], [0, 6, 8]                               # prompts; first page of each sequence
    B, T = len(lens), sum(lens)
    seq = torch.cat([torch.full((n,), b, device=DEV) for b, n in enumerate(lens)])
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device=DEV) for n in lens])
    slots = (ints(pages, torch.int64)[seq] * PAGE + pos).contiguous()
    cu = ints([0, 150, 151, 484])

    # the prompts: expanded attention over what the cache gives back
    x = torch.randn((T, D), generator=g, device=DEV).to(torch.bfloat16)
    q = blk.project(x, pos, slots)
    cb = torch.empty((T, 512), dtype=torch.bfloat16, device=DEV)
    kb = torch.empty((T, 64), dtype=torch.bfloat16, device=DEV)
    fs.fs_latent_cache_read(blk.desc, blk.cache, slots, cb, kb)
    kn = torch.einsum("hnl,tl->thn", blk.w_uk, cb.float()).to(torch.bfloat16)
    v = torch.einsum("hnl,tl->thn", blk.w_uv, cb.float()).to(torch.bfloat16)
    out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((H, T), device=DEV)
    fs.fs_latent_prefill(q, kn, kb, v, cu, cu, True, SCALE, out, lse)
    extra = out.view(T, H * 128).float() @ blk.wo
    run = parity.GpuBlockRunner(blk.cfg(T), T, DEV)
    o_star, o = blk.moe_with(run, x, extra)
    _no_dev_error()
    for b in range(B):
        s = slice(int(cu[b]), int(cu[b + 1]))
        for h in range(H):
            want, wl, tol, tl = ref.attend(q[s, h], torch.cat([kn[s, h], kb[s]], -1), v[s, h], SCALE,
                                           ref.visible(lens[b], lens[b], True, DEV))
            ref.within(out[s, h], want, tol, "prompt out")
            ref.within(lse[h, s], wl, tl, "prompt lse")
    blk.check_block(run, x, extra, o_star, o)

    # one token more for each sequence, three times: eager, then captured, then replayed with new inputs
    table = torch.zeros((B, 8), dtype=torch.int32, device=DEV)
    for b in range(B):
        table[b] = pages[b] + torch.arange(8, device=DEV)
    now = ints(lens)
    step_x = torch.empty((B, D), dtype=torch.bfloat16, device=DEV)
    step_pos, step_slots, step_len = torch.empty_like(now), torch.empty((B,), dtype=torch.int64, device=DEV), torch.empty_like(now)
    ws = torch.empty(fs.fs_latent_decode_ws_bytes(H, B, 1), dtype=torch.uint8, device=DEV)
    run1 = parity.GpuBlockRunner(blk.cfg(B), B, DEV)

    def step():
        q1 = blk.project(step_x, step_pos, step_slots)
        ql = torch.einsum("thn,hnl->thl", q1[..., :128].float(), blk.w_uk).to(torch.bfloat16)
        ol = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV)
        l1 = torch.empty((B, H), device=DEV)
        fs.fs_latent_decode(blk.desc, ql, q1[..., 128:], blk.cache, table, step_len, SCALE, ol, l1, ws)
        att = torch.einsum("hnl,thl->thn", blk.w_uv, ol.float()).reshape(B, H * 128) @ blk.wo
        return (ql, q1, ol, l1, att) + blk.moe_with(run1, step_x, att)

    def inputs(i):
        step_x.copy_(torch.randn((B, D), generator=gen(40 + i), device=DEV))
        step_pos.copy_(now + i)
        step_slots.copy_(ints(pages, torch.int64) * PAGE + now + i)
        step_len.copy_(now + i + 1)

    def check(i, got):
        ql, q1, ol, l1, att, o_star, o = got
        for b in range(B):
            n = lens[b] + i + 1
            sl = pages[b] * PAGE + torch.arange(n, device=DEV)
            c, kr = torch.empty((n, 512), dtype=torch.bfloat16, device=DEV), torch.empty((n, 64), dtype=torch.bfloat16, device=DEV)
            fs.fs_latent_cache_read(blk.desc, blk.cache, sl, c, kr)
            assert torch.equal(c[:lens[b]], cb[cu[b]:cu[b + 1]]) and torch.equal(kr[:lens[b]], kb[cu[b]:cu[b + 1]])
            want, wl, tol, tl = ref.attend(torch.cat([ql[b], q1[b, :, 128:]], -1), torch.cat([c, kr], -1), c, SCALE,
                                           torch.ones((H, n), dtype=torch.bool, device=DEV))
            ref.within(ol[b], want, tol, "token out")
            ref.within(l1[b], wl, tl, "token lse")
        blk.check_block(run1, step_x, att, o_star, o)

    inputs(0)
    eager = step()
    _no_dev_error()
    check(0, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    _no_dev_error()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    for i in (1, 2):
        inputs(i)
        graph.replay()
        _no_dev_error()
        check(i, got)
