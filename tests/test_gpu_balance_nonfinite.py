"""Infinities and NaN in the router logits, for every gate."""
import math

import pytest
import torch

from mixture_experts_layer_expert_gb300 import fs

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -16        # of a score, as derived in test_gpu_balance


def call(z, idx, gate, cu):
    T, E = z.shape
    S = len(cu) - 1
    desc = fs.make_balance(T, E, idx.shape[1], gate, S, 1.0)
    new = lambda *s, dt=torch.float32: torch.full(s, 77, dtype=dt, device=DEV)
    counts, tokens, probs, loss, dz = new(S, E, dt=torch.int32), new(S, dt=torch.int32), new(S, E), new(1), new(T, E)
    ws = new(fs.fs_balance_ws_bytes(desc), dt=torch.uint8)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    fs.fs_balance_loss(desc, z.to(DEV), idx.to(DEV), counts, tokens, probs, loss, ws, cu=cud)
    fs.fs_balance_loss_backward(desc, z.to(DEV), counts, tokens, None, dz, cu=cud)
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)
    return [t.cpu() for t in (counts, tokens, probs, loss, dz)]


@pytest.mark.parametrize("gate", ["softmax", "softmax_renorm", "sigmoid", "sigmoid_norm"])
@pytest.mark.parametrize("T,E", [(64, 16), (3000, 33)])
@pytest.mark.parametrize("what", ["nan", "+inf", "all +inf"])
def test_what_reaches_how_far(gate, T, E, what):
    """A NaN makes its row and its sequence's means NaN for every gate.  +infinity does so for a softmax; a sigmoid of it
    is one, so that row is finite, and its gradient there zero.  Other rows and sequences keep their bits."""
    g = torch.Generator().manual_seed(T)
    z = torch.randn((T, E), generator=g)
    idx = torch.topk(z, 2, 1).indices.int()
    cu, t = [0, T // 2, T], T // 2 + 9
    clean = call(z, idx, gate, cu)
    if what == "nan":
        z[t, 3] = math.nan
    else:
        z[t, 3 if what == "+inf" else slice(None)] = math.inf
    got = call(z, idx, gate, cu)
    others = torch.arange(T) != t
    assert torch.equal(got[2][0], clean[2][0]) and torch.equal(got[4][others], clean[4][others])
    if what == "nan" or gate.startswith("softmax"):
        assert got[2][1].isnan().all() and got[3].isnan().all() and got[4][t].isnan().all()
        return
    assert all(x.isfinite().all() for x in got[2:])
    sig = torch.sigmoid(z[t].double())
    s = sig / sig.sum()
    n = T - T // 2
    f = got[0][1].double() * E / (2 * n)
    want = 1.0 / (2 * n) * s * (f - (f * s).sum()) * (1 - sig)
    assert (got[4][t][z[t] == math.inf] == 0).all()
    assert ((got[4][t].double() - want).abs() <= s / (2 * n) * f.max() * 4 * REL + 1e-44).all()
