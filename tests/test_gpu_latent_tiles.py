"""GPU parity of absorbed attention where a block's pieces of one tile, its rings
of stages and its running maxima are at work (many short sequences, many tiles a
block, scores that grow along the sequence), and expanded attention over long
keys.  Against the 64-bit definitions with the bounds of latent_ref.py."""
import math

import pytest
import torch

import latent_ref as ref
from mixture_experts_layer_expert_gb300 import fs
from test_gpu_latent import DEV, SCALE, SENTINEL, Decode, Prefill, _no_dev_error, gen, randn

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


class Rising(Decode):
    """Records whose score jumps by 7.5 (15) over the rest, at positions of a sequence's second and later tiles: the
    running maximum is raised by more than 2^8 in the middle of a block's work, while what came before still makes
    several percent of the row's sum, so that a sum or an output that is not rescaled (or twice) shows.  Every fourth
    head falls where the others rise."""

    def __init__(self, H, lens, n_q, page, cache, seed=0):
        super().__init__(H, lens, n_q, page, cache, seed)
        g = gen(seed + 77)
        u = torch.where(torch.rand(512, generator=g, device=DEV) < 0.5, -1.0, 1.0) / math.sqrt(512)
        sign = torch.where(torch.arange(H, device=DEV) % 4 == 3, -1.0, 1.0)
        self.ql.copy_(randn(g, self.ql.shape, 0.2, torch.float32) + 7.5 / (10 * SCALE) * sign[:, None] * u)
        self.qr.mul_(0.3)
        for b, n in enumerate(lens):
            i = torch.arange(n, device=DEV)
            c, kr = randn(g, (n, 512), 1.0, torch.float32), randn(g, (n, 64))
            c -= (c @ u)[:, None] * u                                    # scores rise by the jumps alone
            jump = (i % 211 == 130).float() + (i % 601 == 400).float()
            c = (c + 10 * jump[:, None] * u).to(torch.bfloat16)
            slots = self.table[b].long()[i // page] * page + i % page
            fs.fs_latent_cache_write(self.desc, c, kr, slots, self.cache)
            cb, kb = torch.empty_like(c), torch.empty_like(kr)
            fs.fs_latent_cache_read(self.desc, self.cache, slots, cb, kb)
            self.rows[b] = (cb, kb)

    def check_rises(self):
        """Three heads of four exceed the first 128 records' maximum by more than 2^8 at record 130."""
        c, kr = self.rows[0]
        s = torch.cat([self.ql[0], self.qr[0]], -1).double() @ torch.cat([c, kr], -1)[:131].double().T * SCALE
        over = (s[:, 130] - s[:, :128].amax(1)) / math.log(2.0) > 8.0
        assert over.float().mean() > 0.6


# query rows 16, 32, 64 (one CTA), 128, 256, 300, 512 (CTA pairs, one to four row blocks); pages that are a tile's half or
# whole, that end inside a tile, that are no multiple of four
VARIANTS = [(16, 1, 64), (16, 1, 48), (32, 1, 48), (16, 2, 7), (64, 1, 7), (16, 4, 64), (128, 1, 64), (128, 1, 7),
            (128, 2, 48), (100, 3, 64), (128, 4, 48)]


def _run_twice_and_check(p):
    p.check_rises()
    p.run()
    _no_dev_error()
    p.check()
    first, lse = p.out.clone(), p.lse.clone()
    p.ws.fill_(0xFF)
    p.out.fill_(SENTINEL)
    p.run()
    _no_dev_error()
    assert torch.equal(p.out, first) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,n_q,page", VARIANTS)
def test_decode_raised_maxima_in_many_sequences(cache, H, n_q, page):
    """Several pieces of several tiles a block: rings wrap, Q changes, maxima rise inside a piece."""
    _run_twice_and_check(Rising(H, [200 + (97 * i) % 201 for i in range(300)], n_q, page, cache))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,n_q,page", VARIANTS)
def test_decode_raised_maxima_in_a_long_sequence(cache, H, n_q, page):
    """A sequence over all blocks, several tiles each, with shorter ones behind it; partials of rows that have risen and
    rows that have not meet in the join."""
    _run_twice_and_check(Rising(H, [40000, 9, 4000], n_q, page, cache))


@pytest.mark.parametrize("H,lq,lk,causal", [
    (3, [300], [9000], True),                  # a chunk of a prompt behind a long cached prefix
    (2, [2300, 1, 130], [2300, 4100, 5000], True),
    (2, [700], [3000], False),
])
@pytest.mark.parametrize("q_std", [1.0, 12.0])
def test_prefill_long_keys(H, lq, lk, causal, q_std):
    """Dozens of key tiles an item; with scores of some tens maxima rise in the middle of them."""
    p = Prefill(H, lq, lk, causal, q_std=q_std)
    p.forward()
    p.backward()
    _no_dev_error()
    p.check_forward()
    p.check_backward()


def test_fp8_cache_over_the_whole_exponent_range():
    """A row's largest value from bf16's smallest subnormal to its largest number: what is read back is code * scale
    exactly; only 2^128 (from magnitudes above 31 2^123) has no bf16 and is infinity."""
    g = gen(8)
    e = torch.arange(-133, 128, device=DEV)
    c = (torch.rand((e.numel(), 512), generator=g, device=DEV).double() * 2 - 1) * ref.pow2(e)[:, None]
    c[:, 7] = ref.pow2(e)                                            # the row's exponent, whatever was drawn
    c[:, 8] = ref.pow2(e) * 2.0 ** -9
    c[-1, 9] = 2.0 ** 128 * (1 - 2.0 ** -8)                          # the largest bf16
    c = c.float().to(torch.bfloat16)
    assert c.isfinite().all()
    T = c.shape[0]
    desc = fs.make_latent_cache(T, 1, "fp8")
    buf = fs.latent_cache_empty(desc)
    slots, kr = torch.arange(T, device=DEV), randn(g, (T, 64))
    fs.fs_latent_cache_write(desc, c, kr, slots, buf)
    cb, kb = torch.empty_like(c), torch.empty_like(kr)
    fs.fs_latent_cache_read(desc, buf, slots, cb, kb)
    _no_dev_error()
    want, _ = ref.fp8_rows(c)
    want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * math.inf, want)
    assert want.isinf().sum() == 1 and torch.equal(cb.double(), want) and torch.equal(kb, kr)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,n_q", [(16, 2), (64, 1), (128, 1), (128, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_decode_nan_and_infinity_stay_in_their_sequence(cache, H, n_q, value):
    """NaN or infinity in the last record of two sequences and in a query row of a third: every other row keeps its
    result bit for bit (the blocks that hold them hold other sequences too)."""
    lens = [40 + (29 * i) % 150 for i in range(400)]
    p = Decode(H, lens, n_q, 16, cache)
    p.run()
    _no_dev_error()
    p.check()
    keep, lse = p.out.clone(), p.lse.clone()
    bad = [5, 333]
    for b in bad:
        last = lens[b] - 1
        rec = p.cache.view(-1, p.cache.shape[-1])[int(p.table[b, last // 16]) * 16 + last % 16]
        if cache == "bf16":
            rec[:512:3] = value
        else:
            rec[:512:3] = 0x7F                                       # E4M3 has NaN only
            if math.isinf(value):
                rec[640:644].view(torch.float32).fill_(value)        # the scale
    p.ql[77 * n_q, H // 2, 11] = value
    p.out.fill_(SENTINEL)
    p.lse.fill_(SENTINEL)
    p.run()
    _no_dev_error()
    same = torch.ones(p.out.shape[:2], dtype=torch.bool, device=DEV)
    for b in bad:
        same[b * n_q:(b + 1) * n_q] = False
    same[77 * n_q, H // 2] = False
    assert torch.equal(p.out[same], keep[same]) and torch.equal(p.lse[same], lse[same])
    newest = torch.stack([p.out[b * n_q + n_q - 1, :, :512] for b in bad])
    assert not newest.isfinite().all(-1).any()                       # the rows that see the record show it
    assert not p.out[77 * n_q, H // 2, :512].isfinite().all()
