"""A process whose first call of each attention operator is under stream capture: nothing that a first call sets up
(kernel attributes, the error word's address, tensor-map encoding) may break the capture or be missing in the graph."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import math, sys
import torch
sys.path[:0] = [%r, %r]
from mixture_experts_layer_expert_gb300 import fs

dev, bf = "cuda", torch.bfloat16
g = torch.Generator(device=dev).manual_seed(1)
rn = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
T, H, n = 200, 4, 40
pos = torch.arange(T, dtype=torch.int32, device=dev)
x, y = rn(T, H, 64), torch.zeros((T, H, 64), dtype=bf, device=dev)
c, kr = rn(T, 512), rn(T, 64)
slots = torch.arange(T, device=dev)
desc = {k: fs.make_latent_cache(5, n, k) for k in ("bf16", "fp8")}
cache = {k: fs.latent_cache_empty(d) for k, d in desc.items()}
for t in cache.values():
    t.zero_()
back = {k: (torch.zeros_like(c), torch.zeros_like(kr)) for k in desc}
table = i32([[0, 1, 2, 3, 4]])
dec = {(k, h): (rn(1, h, 512), rn(1, h, 64), torch.zeros((1, h, 512), dtype=bf, device=dev), torch.zeros((1, h), device=dev),
                torch.zeros(fs.fs_latent_decode_ws_bytes(h, 1, 1), dtype=torch.uint8, device=dev))
       for k in desc for h in (16, 32, 64, 128)}
q, kn, v, do = rn(T, H, 192), rn(T, H, 128), rn(T, H, 128), rn(T, H, 128)
out, lse = torch.zeros_like(v), torch.zeros((H, T), device=dev)
dq, dkn, dkr, dv = (torch.zeros_like(t) for t in (q, kn, kr, v))
ws = torch.zeros(fs.fs_latent_prefill_backward_ws_bytes(H, T, T), dtype=torch.uint8, device=dev)
cu, scale, rope, ln = i32([0, 77, T]), 1 / math.sqrt(192), fs.make_rope(64), i32([T])


def everything():
    fs.fs_rope(rope, pos, x, y)
    for k, d in desc.items():
        fs.fs_latent_cache_write(d, c, kr, slots, cache[k], rope=rope, pos=pos)
        fs.fs_latent_cache_read(d, cache[k], slots, *back[k])
    for (k, h), (ql, qr, o, l, w) in dec.items():
        fs.fs_latent_decode(desc[k], ql, qr, cache[k], table, ln, scale, o, l, w)
    fs.fs_latent_prefill(q, kn, kr, v, cu, cu, True, scale, out, lse)
    fs.fs_latent_prefill_backward(q, kn, kr, v, cu, cu, True, scale, out, lse, do, dq, dkn, dkr, dv, ws)


results = [y, out, lse, dq, dkn, dkr, dv] + [t for b in back.values() for t in b] + [t for d in dec.values() for t in d[2:4]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    everything()
graph.replay()
torch.cuda.synchronize()
assert fs.fs_get_error() == (0, 0)
first = [t.clone() for t in results]
assert all(t.isfinite().all() and t.abs().max() > 0 for t in first)
for t in results:
    t.zero_()
everything()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, results))
slots[3] = 5 * n                              # past the cache: the captured calls report it
graph.replay()
torch.cuda.synchronize()
assert fs.fs_get_error() == (5, 5) and fs.fs_get_error() == (0, 0)
print("first calls under capture: ok")
"""


def test_first_calls_under_capture():
    r = subprocess.run([sys.executable, "-c", CHILD % (ROOT, os.path.join(ROOT, "tests"))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "first calls under capture: ok" in r.stdout, r.stdout + r.stderr
