"""Sizes of the balance loss at the end of its range, without a GPU."""
import pytest

from mixture_experts_layer_expert_gb300 import build, fs


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("T", [1, 152 * 8, 2132483648, 2133348537, 2133499904, 2 ** 31 - 8193])
@pytest.mark.parametrize("n_seqs", [1, 2, 65535])
@pytest.mark.parametrize("E", [1, 8, 512])
def test_workspace_is_a_slot_per_block_and_sequence(T, n_seqs, E):
    """At most 152 blocks, and a slot of sums, counts and rows for each of them and each sequence; the sequences' shares of
    the loss, one per 32 experts; eight arrays' rounding to 256 bytes."""
    slots = min((T + 7) // 8, 152) + n_seqs
    least = (n_seqs + 1) * E * 8
    most = slots * (E * 8 + 4) + n_seqs * ((E + 31) // 32) * 4 + 152 * 4 + 8 * 256
    assert least <= fs.fs_balance_ws_bytes(fs.make_balance(T, E, 1, "softmax", n_seqs, 1.0)) <= most
