"""Balance loss, 4-bit products and orthogonalised updates in graphs: a process whose first call of each is under
capture, and two graphs that share their workspaces."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
import torch
sys.path[:0] = [%r]
from mixture_experts_layer_expert_gb300 import configs, fs, synth

dev, bf, f32, i32, u8 = "cuda", torch.bfloat16, torch.float32, torch.int32, torch.uint8
SHAPES = [("f32", 2, 7, 300), ("bf16", 3, 12, 16), ("f32", 2, 64, 300), ("bf16", 1, 100, 2100), ("f32", 3, 40, 100),
          ("f32", 2, 150, 300), ("bf16", 1, 301, 140)]


class Ops:
    # one set of inputs and results; workspaces are the caller's
    def __init__(self, seed, ws):
        g = torch.Generator(device=dev).manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device=dev)
        self.ws = ws
        self.bal = []
        for T, E, k, gate, cu in ((300, 12, 2, "softmax", None), (3000, 40, 4, "sigmoid_norm", [0, 700, 700, 2900])):
            z = rn(T, E)
            S = 1 if cu is None else len(cu) - 1
            d = fs.make_balance(T, E, k, gate, S, 0.5)
            self.bal.append((d, z, torch.topk(z, k, 1).indices.int(), torch.zeros((S, E), dtype=i32, device=dev),
                             torch.zeros(S, dtype=i32, device=dev), torch.zeros((S, E), device=dev), torch.zeros(1, device=dev),
                             torch.zeros((T, E), device=dev), None if cu is None else torch.tensor(cu, dtype=i32, device=dev)))
        self.lin = []
        for rows, N, K, dt in ((1, 264, 384, bf), (40, 5000, 1408, f32), (600, 512, 256, bf)):
            x, w = rn(rows, K).to(bf), fs_pack[(N, K)]
            self.lin.append((rows, N, K, x, fs.mx4_rows_empty(rows, K), w, torch.zeros((rows, N), dtype=dt, device=dev)))
        self.orth = []
        for dt, b, m, n in SHAPES:
            x = rn(b, m, n).to(bf if dt == "bf16" else f32)
            self.orth.append((fs.make_orthogonalize(b, m, n, dt), x, torch.zeros((b, m, n), dtype=bf, device=dev)))

    def run(self):
        for d, z, idx, counts, tokens, probs, loss, dz, cu in self.bal:
            fs.fs_balance_loss(d, z, idx, counts, tokens, probs, loss, self.ws, cu=cu)
            fs.fs_balance_loss_backward(d, z, counts, tokens, None, dz, cu=cu)
        for rows, N, K, x, q, w, y in self.lin:
            fs.fs_quantize_rows_mx4(rows, K, x, q)
            fs.fs_linear_mx4(q, w, y, K, self.ws)
        for d, x, out in self.orth:
            fs.fs_orthogonalize(d, x, out, self.ws)

    def results(self):
        return [t for b in self.bal for t in b[3:8]] + [l[6] for l in self.lin] + [o[2] for o in self.orth]


# packs are made on the host's side of the story, before: weights laid out once
gw = torch.Generator(device=dev).manual_seed(9)
raw = {s: torch.randn(s, generator=gw, device=dev).to(bf) for s in ((264, 384), (5000, 1408), (512, 256))}
fs_pack = {s: torch.zeros(fs.fs_packed_bytes(1, *s, fs.FS_MXFP4), dtype=u8, device=dev) for s in raw}
need = max([fs.fs_orthogonalize_ws_bytes(fs.make_orthogonalize(b, m, n, dt)) for dt, b, m, n in SHAPES] + [1 << 22])
ws = torch.full((need,), 0xFF, dtype=u8, device=dev)
one, two = Ops(1, ws), Ops(2, ws)
torch.cuda.synchronize()


def record(ops, packs):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if packs:
            for s, w in raw.items():
                fs.fs_pack_w3(1, *s, fs.FS_MXFP4, w, fs_pack[s])
        ops.run()
    return graph


first, second = record(one, True), record(two, False)
first.replay()
torch.cuda.synchronize()
assert fs.fs_get_error() == (0, 0)
for _ in range(2):
    for graph in (second, first, first, second):
        graph.replay()
torch.cuda.synchronize()
assert fs.fs_get_error() == (0, 0)
replayed = [[t.clone() for t in o.results()] for o in (one, two)]
for o, was in zip((one, two), replayed):
    for t in o.results():
        t.zero_()
    o.ws = torch.full((need,), 0xA5, dtype=u8, device=dev)
    o.run()
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)
    for i, (a, b) in enumerate(zip(o.results(), was)):
        assert torch.equal(a, b) and a.any(), i
    assert len(was) == 20
print("same")
""" % ROOT


def test_first_calls_under_capture_and_graphs_that_share_a_workspace():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
