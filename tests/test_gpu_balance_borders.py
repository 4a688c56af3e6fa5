"""Borders of the balance loss that decrease or leave the batch: reported, and no sequence's results then depend on
which of two sequences that share rows was worked on first, or on what the workspace held."""
import pytest
import torch

from mixture_experts_layer_expert_gb300 import fs

pytestmark = pytest.mark.gpu
DEV = "cuda"

BAD = [
    (50, [0, 30, 20, 50]), (50, [0, 60, 60]), (50, [-3, 20, 50]), (50, [0, 30, 20]), (50, [0, 10, 2 ** 31 - 1]),
    (50, [0, 51]), (50, [-2 ** 31, 50]), (50, [20, 10]),
    (9000, [0, 8000, 10, 20, 9000]), (9000, [0, 100, 50, 9000, 9000]), (9000, [9000, 0, 9000]), (9000, [0, 9000, 9001]),
    (9000, [5000, 4999, 6000]), (9000, [0, 3, 2] + [2] * 4000 + [9000]), (9000, list(range(0, 8000)) + [7000, 9000]),
]


@pytest.mark.parametrize("T,cu", BAD, ids=lambda v: "%d_borders" % len(v) if isinstance(v, list) else str(v))
@pytest.mark.parametrize("gate", ["softmax", "sigmoid_norm"])
def test_all_sequences_count_as_empty(T, cu, gate):
    E, k, S = 24, 3, len(cu) - 1
    g = torch.Generator().manual_seed(T + S)
    z = torch.randn((T, E), generator=g).to(DEV)
    idx = torch.topk(z, k, 1).indices.int()
    desc = fs.make_balance(T, E, k, gate, S, 0.5)
    cu_d = torch.tensor(cu, dtype=torch.int32, device=DEV)
    new = lambda *s, dt=torch.float32: torch.full(s, 77, dtype=dt, device=DEV)
    ws = torch.full((fs.fs_balance_ws_bytes(desc),), 0xA5, dtype=torch.uint8, device=DEV)

    def step(borders):
        counts, tokens, probs, loss = new(S, E, dt=torch.int32), new(S, dt=torch.int32), new(S, E), new(1)
        dz = torch.full((T, E), 5.0, device=DEV)
        fs.fs_balance_loss(desc, z, idx, counts, tokens, probs, loss, ws, cu=borders)
        torch.cuda.synchronize()
        err = fs.fs_get_error()
        fs.fs_balance_loss_backward(desc, z, counts, tokens, None, dz, cu=borders)
        torch.cuda.synchronize()
        back = fs.fs_get_error()
        return err, back, counts, tokens, probs, loss, dz
    err, back, counts, tokens, probs, loss, dz = step(cu_d)
    assert err == (5, 2) and back in ((0, 0), (5, 2))
    assert not counts.any() and not tokens.any() and (probs == 0).all() and float(loss) == 0.0
    rows = (dz == 0).all(1) | (dz == 5).all(1)
    assert rows.all(), "rows with a gradient: %s" % (~rows).nonzero().flatten().tolist()[:8]
    named = torch.zeros(T, dtype=torch.bool)
    for q0, q1 in zip(cu, cu[1:]):
        named[max(0, q0):max(0, min(T, q1))] = True
    assert (dz[~named] == 5).all()                                     # rows that no sequence names are left
    again = step(cu_d)
    assert all(torch.equal(a, b) for a, b in zip((counts, tokens, probs, loss, dz), again[2:]))
    # and the same workspace serves the right borders afterwards
    good = torch.linspace(0, T, S + 1).int().to(DEV)
    err, back, counts, tokens, probs, loss, dz = step(good)
    assert err == (0, 0) and back == (0, 0)
    assert torch.equal(tokens, good[1:] - good[:-1]) and int(counts.sum()) == T * k and float(loss) > 0
    assert not (dz == 5).any()
