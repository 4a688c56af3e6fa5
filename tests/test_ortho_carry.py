"""The documented accuracy of orthogonalised updates, for the roundings that the kernels make (no GPU)."""
import pytest
import torch

import ortho_carry as carry
import ortho_ref as ref


@pytest.mark.parametrize("m,n", [(32, 40), (128, 128), (200, 128), (96, 500), (64, 4500), (150, 333), (333, 260)])
@pytest.mark.parametrize("form", ["small", "tiled"])
@pytest.mark.parametrize("rank", ["full", "few", "one"])
def test_usual_steps_stay_within_the_documented_distance(m, n, form, rank):
    """0.3% of the exact result, the rounding to bf16 included, for gradients of any rank."""
    r = {"full": 2 * min(m, n), "few": max(2, min(m, n) // 16), "one": 1}[rank]
    g = ref.gradient(m, n, r, m + r)
    want = ref.exact(g)
    got = carry.rounded(g, form=form).to(torch.bfloat16).double()
    assert float((got - want).norm() / want.norm()) < 3e-3


def test_the_byte_is_worth_carrying():
    """Without it, X in a single fp16 number, a gradient of few tokens is more than 1% off."""
    g = ref.gradient(150, 500, 24, 7)
    want = ref.exact(g)
    x = ref.start(g, 1e-7)
    for a, b, c in ref.USUAL:
        x = carry.fp16(x, 13)
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    assert float((x - want).norm() / want.norm()) > 1e-2
    assert float((carry.rounded(g, form="tiled") - want).norm() / want.norm()) < 2e-3


def test_the_byte_reaches_nineteen_bits():
    """H and the byte together: off by at most a 508th of H's step, so 2^-19 of a value's power of two; what a byte can hold."""
    x = torch.cat([torch.linspace(-1, 1, 4001, dtype=torch.float64), torch.logspace(-8, 0, 500, 2.0, dtype=torch.float64)])
    h = carry.fp16(x, 13)
    off = (h + carry.rest_in_a_byte(x, h, 13) - x).abs()
    step = torch.exp2(torch.floor(torch.log2(h.abs().clamp_min(2.0 ** -27))) - 10)
    assert (off <= step / 508 * (1 + 1e-9)).all()


def test_powers_of_two():
    assert carry.powers(ref.USUAL) == [13, 13, 12]
    assert carry.powers([(0.5, 0.0, 0.0)]) == [14, 14, 14]
