"""The balance loss's operands are held against the descriptor as it is when the call is made, without a GPU: a
descriptor whose fields change after make_balance is no way past the checks."""
import pytest
import torch

from mixture_experts_layer_expert_gb300 import build, fs

INVALID = 1


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    """Operands in host memory stand for the device's: every refusal comes before the library is called."""
    build.build()
    monkeypatch.setattr(fs, "_here", lambda stream: (-1, 0))

    class NoCalls:
        fs_balance_ws_bytes = staticmethod(fs.lib().fs_balance_ws_bytes)

        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(fs, "lib", lambda: NoCalls())


def operands(T, E, k, S):
    i32, f32 = torch.int32, torch.float32
    z = lambda *s, dt=f32: torch.zeros(s, dtype=dt)
    return dict(logits=z(T, E), topk_idx=z(T, k, dt=i32), counts=z(S, E, dt=i32), tokens=z(S, dt=i32), probs=z(S, E),
                loss=z(1), ws=z(1 << 20, dt=torch.uint8), cu=z(S + 1, dt=i32), mask=z(T, dt=torch.uint8), bias=z(E))


@pytest.mark.parametrize("field,to", [("T", 128), ("T", 32), ("E", 64), ("E", 8), ("k", 4), ("n_seqs", 5), ("n_seqs", 2)])
def test_a_changed_descriptor_refuses_operands_of_the_old_sizes(field, to):
    desc = fs.make_balance(64, 16, 2, "softmax", 3, 0.5)
    ops = operands(64, 16, 2, 3)
    setattr(desc, field, to)
    with pytest.raises(fs.FsError) as e:
        fs.fs_balance_loss(desc, **ops)
    assert e.value.status == INVALID
    if field == "k":                     # the gradient does not read the indices
        return
    back = {n: ops[n] for n in ("logits", "counts", "tokens", "bias", "cu", "mask")}
    with pytest.raises(fs.FsError) as e:
        fs.fs_balance_loss_backward(desc, d_loss=None, d_logits=torch.zeros(64, 16), **back)
    assert e.value.status == INVALID


@pytest.mark.parametrize("name", ["logits", "topk_idx", "counts", "tokens", "probs", "loss", "cu", "mask", "bias"])
def test_operands_of_other_sizes_are_refused(name):
    desc = fs.make_balance(64, 16, 2, "softmax", 3, 0.5)
    ops = operands(64, 16, 2, 3)
    ops[name] = torch.cat([ops[name], ops[name][:1]])
    with pytest.raises(fs.FsError) as e:
        fs.fs_balance_loss(desc, **ops)
    assert e.value.status == INVALID


def test_right_operands_reach_the_library():
    with pytest.raises(AssertionError, match="fs_balance_loss was called"):
        fs.fs_balance_loss(fs.make_balance(64, 16, 2, "softmax", 3, 0.5), **operands(64, 16, 2, 3))
