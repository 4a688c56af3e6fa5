"""GPU parity of absorbed attention where a block's pieces of one tile, its rings
of stages and its running maxima are at work: many short sequences, many tiles a
block, scores that grow along the sequence.  Against the 64-bit definitions with
the bounds of latent_ref.py."""
import pytest
import torch

from mixture_experts_layer_expert_gb300 import fs
from test_gpu_latent import Decode, SENTINEL, _no_dev_error

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _loaded():
    fs.lib()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,n_q", [(128, 1), (80, 1), (128, 2)])
def test_decode_pieces_of_one_tile(cache, H, n_q):
    """Every piece is one tile of at most 128 records: its first tile, where the two halves of a row's records exchange
    maxima, is also its last, where they exchange sums.  Scores of a few tens set the two apart."""
    lens = [1 + (37 * i) % 128 for i in range(400)]
    p = Decode(H, lens, n_q, 64, cache, q_std=8.0)
    p.run()
    _no_dev_error()
    p.check()
    first, lse = p.out.clone(), p.lse.clone()
    for _ in range(20):
        p.out.fill_(SENTINEL)
        p.lse.fill_(SENTINEL)
        p.run()
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    _no_dev_error()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,n_q", [(48, 4), (43, 3), (20, 16)])
def test_decode_last_row_block_half_empty(cache, H, n_q):
    """More than 128 query rows whose last 128-row block has at most 64: its second CTA has none."""
    p = Decode(H, [700, 0, 3, 129, 2500], n_q, 64, cache)
    p.run()
    _no_dev_error()
    p.check()
