"""GPU parity of the attention operators (rotary positions, paged latent cache,
absorbed and expanded latent attention with its gradient) against their 64-bit
definitions, with bounds counted from the roundings (latent_ref.py)."""
import math

import pytest
import torch

import latent_ref as ref
from mixture_experts_layer_expert_gb300 import fs

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALE = 1.0 / math.sqrt(192)
SCALED = dict(base=10000.0, factor=40.0, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0, mscale=1.25)
SENTINEL = 7.0


@pytest.fixture(autouse=True, scope="module")
def _loaded():
    fs.lib()


def _no_dev_error():
    torch.cuda.synchronize()
    st, code = fs.fs_get_error()
    assert st == 0, "device error word = %d" % code


def _dev_error(want):
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (5, want)
    assert fs.fs_get_error() == (0, 0)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


# ------------------------------------------------------------------- rotary

@pytest.mark.parametrize("T,H,d,layout,dtype,kw", [
    (1, 1, 16, "interleaved", "bf16", {}),
    (1, 128, 64, "half", "bf16", {}),
    (37, 3, 64, "interleaved", "f32", SCALED),
    (300, 16, 128, "half", "f32", SCALED),
    (65, 9, 256, "interleaved", "bf16", SCALED),
    (130, 17, 80, "half", "bf16", dict(base=500000.0)),
    (1025, 8, 32, "half", "f32", {}),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(T, H, d, layout, dtype, kw, inverse):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = gen(T + H + d)
    full = randn(g, (T, H, d + 32), dtype=dt)              # the rotated part sits inside the head
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    edge = [2 ** 31 - 1, -5, 0, 163839]
    pos[:min(T, 4)] = ints(edge[:min(T, 4)])
    out = torch.full((T, H, d + 16), SENTINEL, dtype=dt, device=DEV)
    x, y = full[..., 16:16 + d], out[..., 8:8 + d]
    keep = full.clone()
    fs.fs_rope(fs.make_rope(d, layout, **kw), pos, x, y, inverse=inverse)
    _no_dev_error()
    want, mag = ref.rope(x, pos, d, layout, inverse, **kw)
    # sine and cosine: argument and result roundings, the products and the sum
    tol = 12 * ref.ULP32 * mag + (ref.HALF * want.abs() if dt == torch.bfloat16 else 0.0) + 1e-30
    ref.within(y, want, tol, "rope")
    assert torch.equal(full, keep) and (out[..., :8] == SENTINEL).all() and (out[..., 8 + d:] == SENTINEL).all()
    fs.fs_rope(fs.make_rope(d, layout, **kw), pos, x, x, inverse=inverse)             # in place
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(full[..., :16], keep[..., :16])


def test_rope_inverse_is_the_gradient():
    """<g, R x> = <R^T g, x> and the difference quotient along a direction (R is linear)."""
    g = gen(5)
    T, H, d = 50, 4, 64
    pos = torch.randint(0, 200000, (T,), generator=g, device=DEV, dtype=torch.int32)
    rope = fs.make_rope(d, "interleaved", **SCALED)
    x, dy, v = (randn(g, (T, H, d), dtype=torch.float32) for _ in range(3))
    y, dx, y2 = (torch.empty_like(x) for _ in range(3))
    fs.fs_rope(rope, pos, x, y)
    fs.fs_rope(rope, pos, dy, dx, inverse=True)
    fs.fs_rope(rope, pos, x + v, y2)
    _no_dev_error()
    n, size = x.numel(), (dy.double().abs() * (y2.double().abs() + y.double().abs() + 4)).sum()
    tol = 16 * ref.ULP32 * size
    assert abs((dy.double() * y.double()).sum() - (dx.double() * x.double()).sum()) < tol
    assert abs((dy.double() * (y2.double() - y.double())).sum() - (dx.double() * v.double()).sum()) < 2 * tol


def test_rope_transposed_layout():
    """Heads outermost in memory ([H, T, d])."""
    g = gen(6)
    x = randn(g, (5, 33, 64)).transpose(0, 1)
    y = torch.empty((5, 33, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    fs.fs_rope(fs.make_rope(64), pos, x, y)
    _no_dev_error()
    want, mag = ref.rope(x, pos, 64, "interleaved")
    ref.within(y, want, ref.HALF * want.abs() + 12 * ref.ULP32 * mag, "rope")


# -------------------------------------------------------------------- cache

def _rows_with_edges(g, T):
    c = randn(g, (T, 512)) * ref.pow2(torch.randint(-20, 12, (T, 1), generator=g, device=DEV)).float()
    c = c.to(torch.bfloat16)
    if T > 3:
        c[1] = 0
        c[2] = c[2].clamp(-56.0, 56.0)
        c[2, 5] = 56.0                       # 448 / 8: the scale's boundary
    return c


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("T,page,n_pages,layout", [(1, 1, 1, None), (7, 48, 3, "interleaved"), (300, 64, 9, "half"),
                                                   (1000, 100, 11, "interleaved")])
def test_cache_write_read(cache, T, page, n_pages, layout):
    g = gen(T + page)
    desc = fs.make_latent_cache(n_pages, page, cache)
    buf = fs.latent_cache_empty(desc)
    buf.view(torch.uint8).fill_(0x55)
    before = buf.clone()
    wide = torch.zeros((T, 512 + 64 + 8), dtype=torch.bfloat16, device=DEV)      # the down-projection's output
    wide[:, :512], wide[:, 512:576] = _rows_with_edges(g, T), randn(g, (T, 64))
    c, kr = wide[:, :512], wide[:, 512:576]
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].contiguous()
    if T > 5:
        slots[3] = -1                                                           # a padding row
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    rope = None if layout is None else fs.make_rope(64, layout, **SCALED)
    fs.fs_latent_cache_write(desc, c, kr, slots, buf, rope=rope, pos=pos if rope is not None else None)
    c_back = torch.full((T, 520), SENTINEL, dtype=torch.bfloat16, device=DEV)
    kr_back = torch.full((T, 64), SENTINEL, dtype=torch.bfloat16, device=DEV)
    fs.fs_latent_cache_read(desc, buf, slots, c_back[:, :512], kr_back)
    _no_dev_error()
    live = slots >= 0
    want, scale = ref.fp8_rows(c) if cache == "fp8" else (c.double(), None)
    assert torch.equal(c_back[live, :512].double(), want[live])
    assert (c_back[~live] == SENTINEL).all() and (kr_back[~live] == SENTINEL).all() and (c_back[:, 512:] == SENTINEL).all()
    if rope is None:
        assert torch.equal(kr_back, kr)
    else:
        want, mag = ref.rope(kr[:, None], pos, 64, layout, **SCALED)
        ref.within(kr_back[live], want[live, 0], (ref.HALF * want.abs() + 12 * ref.ULP32 * mag)[live, 0], "k_rope")
    rec, old = buf.view(torch.uint8).view(n_pages * page, -1), before.view(torch.uint8).view(n_pages * page, -1)
    untouched = torch.ones(n_pages * page, dtype=torch.bool, device=DEV)
    untouched[slots[live]] = False
    assert torch.equal(rec[untouched], old[untouched])
    if cache == "fp8":
        assert torch.equal(rec[slots[live], 640:644].contiguous().view(torch.float32).double(), scale[live])
        assert (rec[slots[live], 644:] == 0).all()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_cache_slot_past_the_end(cache):
    g = gen(1)
    desc = fs.make_latent_cache(2, 4, cache)
    buf = fs.latent_cache_empty(desc)
    buf.view(torch.uint8).zero_()
    c, kr = randn(g, (3, 512)), randn(g, (3, 64))
    slots = ints([0, 8, 7], torch.int64)
    fs.fs_latent_cache_write(desc, c, kr, slots, buf)
    _dev_error(5)
    cb, kb = torch.full_like(c, SENTINEL), torch.full_like(kr, SENTINEL)
    fs.fs_latent_cache_read(desc, buf, slots, cb, kb)
    _dev_error(5)
    assert (cb[1] == SENTINEL).all() and torch.equal(kb[0], kr[0]) and torch.equal(kb[2], kr[2])


def test_cache_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: records behind that offset."""
    desc = fs.make_latent_cache(64 * 1024, 64, "bf16")                          # 4.8 GB
    buf = fs.latent_cache_empty(desc)
    n = 64 * 1024 * 64
    g = gen(2)
    slots = ints([n - 1, n // 2, 0, n - 64], torch.int64)
    c, kr = randn(g, (4, 512)), randn(g, (4, 64))
    fs.fs_latent_cache_write(desc, c, kr, slots, buf)
    cb, kb = torch.empty_like(c), torch.empty_like(kr)
    fs.fs_latent_cache_read(desc, buf, slots, cb, kb)
    _no_dev_error()
    assert torch.equal(cb, c) and torch.equal(kb, kr)
    assert torch.equal(buf.view(n, 576)[n - 1, :512], c[0])
    # absorbed attention over the last page: offsets past 32 bits in the reader too
    buf.view(n, 576)[n - 64:].copy_(randn(g, (64, 576)))
    ql, qr = randn(g, (1, 16, 512), 0.5), randn(g, (1, 16, 64))
    out = torch.empty_like(ql)
    lse = torch.empty((1, 16), dtype=torch.float32, device=DEV)
    ws = _decode_ws(16, 1, 1)
    fs.fs_latent_decode(desc, ql, qr, buf, ints([[64 * 1024 - 1]]), ints([50]), SCALE, out, lse, ws)
    _no_dev_error()
    rec = buf.view(n, 576)[n - 64:n - 14]
    want, wl, tol, tl = ref.attend(torch.cat([ql, qr], -1)[0], rec, rec[:, :512], SCALE,
                                   torch.ones((16, 50), dtype=torch.bool, device=DEV))
    ref.within(out[0], want, tol, "out")
    ref.within(lse[0], wl, tl, "lse")


# ----------------------------------------------------------------- absorbed

def _decode_ws(H, B, n_q):
    return torch.empty(fs.fs_latent_decode_ws_bytes(H, B, n_q), dtype=torch.uint8, device=DEV)


class Decode:
    """A decode problem: cache pages in shuffled order, NaN in every record no sequence owns."""

    def __init__(self, H, lens, n_q, page, cache, seed=0, q_std=0.5):
        g = gen(seed + H + n_q + page)
        self.H, self.lens, self.n_q, self.page, B = H, lens, n_q, page, len(lens)
        need = [(n + page - 1) // page for n in lens]
        total = sum(need) + 2
        self.desc = fs.make_latent_cache(total, page, cache)
        self.cache = fs.latent_cache_empty(self.desc)
        if cache == "bf16":
            self.cache.fill_(float("nan"))
        else:
            self.cache.fill_(0x7F)                                   # E4M3 NaN codes, NaN scale
        perm = (torch.randperm(total - 2, generator=g, device=DEV) + 1).to(torch.int32) if total > 2 else None
        self.table = torch.full((B, max(max(need), 1) + 1), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
        self.rows, at = [], 0
        for b, n in enumerate(lens):
            if need[b]:
                self.table[b, :need[b]] = perm[at:at + need[b]]
                at += need[b]
            c, kr = randn(g, (n, 512)), randn(g, (n, 64))
            if n:
                i = torch.arange(n, device=DEV)
                slots = self.table[b].long()[i // page] * page + i % page
                fs.fs_latent_cache_write(self.desc, c, kr, slots, self.cache)
                cb, kb = torch.empty_like(c), torch.empty_like(kr)
                fs.fs_latent_cache_read(self.desc, self.cache, slots, cb, kb)
                c, kr = cb, kb
            self.rows.append((c, kr))
        R = B * n_q
        wide = randn(g, (R, H, 576 + 8))
        self.ql, self.qr = wide[..., :512], wide[..., 512:576]
        self.ql *= q_std
        self.seq = ints(lens)
        self.out = torch.full((R, H, 520), SENTINEL, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((R, H), SENTINEL, device=DEV)
        self.ws = _decode_ws(H, B, n_q)

    def run(self, stream=None):
        fs.fs_latent_decode(self.desc, self.ql, self.qr, self.cache, self.table, self.seq, SCALE,
                            self.out[..., :512], self.lse, self.ws, stream)

    def check(self):
        for b, n in enumerate(self.lens):
            c, kr = self.rows[b]
            for j in range(self.n_q):
                r, end = b * self.n_q + j, max(0, n - (self.n_q - 1 - j))
                k = torch.cat([c, kr], -1)[:end]
                want, wl, tol, tl = ref.attend(torch.cat([self.ql[r], self.qr[r]], -1), k, c[:end], SCALE,
                                               torch.ones((self.H, end), dtype=torch.bool, device=DEV))
                ref.within(self.out[r, :, :512], want, tol, "out of row %d" % r)
                ref.within(self.lse[r], wl, tl, "lse of row %d" % r)
        assert (self.out[..., 512:] == SENTINEL).all()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("H,lens,n_q,page", [
    (1, [1], 1, 1),
    (16, [0, 1, 63, 64, 65, 127, 128, 129], 1, 64),
    (16, [5000], 1, 64),
    (5, [333, 2, 0, 700], 2, 48),
    (128, [1000, 31, 257], 1, 16),
    (128, [640, 3, 1], 4, 100),
    (64, [191, 1500], 1, 128),
    (24, [90, 3000, 1], 3, 7),
    (128, [50], 16, 64),
    (100, [2049, 77], 1, 64),
    (32, [152], 1, 48),                                     # far fewer tiles than SMs: empty ranges between pieces
    (48, [190, 1, 65], 1, 64),
])
def test_decode(cache, H, lens, n_q, page):
    p = Decode(H, lens, n_q, page, cache)
    p.run()
    _no_dev_error()
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_decode_many_sequences(cache):
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(0, 200, (400,), generator=g)]
    lens[7] = 3001
    p = Decode(16, lens, 1, 64, cache)
    p.run()
    _no_dev_error()
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_decode_thousands_of_sequences_of_one_token_or_none(cache):
    p = Decode(3, [i % 2 for i in range(5000)], 1, 2, cache)
    p.run()
    _no_dev_error()
    p.check()


@pytest.mark.parametrize("H", [2, 128])
def test_decode_long_sequence(H):
    """One sequence over all SMs; the short one behind it shares the last range."""
    p = Decode(H, [70001, 9], 1, 64, "bf16")
    p.run()
    _no_dev_error()
    p.check()


@pytest.mark.parametrize("H,cache", [(16, "fp8"), (80, "bf16")])
def test_decode_shared_and_repeated_pages(H, cache):
    """Sequences that share a prefix's pages, and one whose table names a page twice; lse not asked for."""
    p = Decode(H, [640, 300, 200], 1, 64, cache)
    p.table[1, :2] = p.table[0, :2]
    p.table[2, 1] = p.table[2, 0]
    cut = lambda t, u: tuple(torch.cat([x[:128], y[128:]]) for x, y in zip(t, u))
    p.rows[1] = cut(p.rows[0], p.rows[1])
    p.rows[2] = tuple(torch.cat([x[:64], x[:64], x[128:]]) for x in p.rows[2])
    p.run()
    _no_dev_error()
    p.check()
    first = p.out.clone()
    p.out.fill_(SENTINEL)
    fs.fs_latent_decode(p.desc, p.ql, p.qr, p.cache, p.table, p.seq, SCALE, p.out[..., :512], None, p.ws)
    _no_dev_error()
    assert torch.equal(p.out, first)


def test_decode_heads_outside_rows():
    """Queries and outputs laid out head by head."""
    p = Decode(48, [129, 700], 2, 64, "bf16")
    p.run()
    hm = lambda t, w: t[..., :w].transpose(0, 1).contiguous().transpose(0, 1)
    out = hm(torch.full_like(p.out, SENTINEL), 512)
    lse = torch.empty_like(p.lse)
    fs.fs_latent_decode(p.desc, hm(p.ql, 512), hm(p.qr, 64), p.cache, p.table, p.seq, SCALE, out, lse, p.ws)
    _no_dev_error()
    assert torch.equal(out, p.out[..., :512]) and torch.equal(lse, p.lse)


def test_calls_on_two_streams_at_once():
    """Decode and prefill, forward and backward, in turn on two streams with a workspace each."""
    jobs = [(Decode(128, [900, 2000, 5], 1, 64, "bf16", seed=s), Prefill(4, [300, 129], [300, 200], True)) for s in (0, 1)]

    def run(d, f):
        d.run()
        f.forward()
        f.backward()
        return [t.clone() for t in (d.out, d.lse, f.out, f.lse, f.dq, f.dkr, f.dkv)]
    want = [run(*j) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [None, None]
    for _ in range(3):
        for i, (s, j) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i] = run(*j)
    _no_dev_error()
    for w, t in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, t))


def test_decode_large_scores():
    """Scores of several hundred: the running maximum, not the exponent's range, carries them."""
    p = Decode(16, [700, 64], 1, 64, "bf16", q_std=20.0)
    p.run()
    _no_dev_error()
    p.check()


def test_decode_repeats_and_replays_bit_identically():
    p = Decode(128, [900, 2000, 5], 1, 64, "bf16")
    p.run()
    _no_dev_error()
    first, lse = p.out.clone(), p.lse.clone()
    p.ws.fill_(0xFF)                                                 # what an earlier call left there
    p.out.fill_(SENTINEL)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.run()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for _ in range(2):
        p.out.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    p.lens = [901, 1999, 5]                                          # lengths are read on the device at replay
    p.seq.copy_(ints(p.lens))
    p.rows[0] = tuple(torch.cat([t, t[:1]]) for t in p.rows[0])
    slot = p.table[0, 900 // 64].long() * 64 + 900 % 64
    p.cache.view(-1, 576)[slot] = torch.cat([p.rows[0][0][-1], p.rows[0][1][-1]])
    p.rows[1] = tuple(t[:1999] for t in p.rows[1])
    graph.replay()
    _no_dev_error()
    p.check()


def test_decode_bad_page_and_length():
    """A page outside the cache leaves its positions out, a length outside the table empties its sequence."""
    p = Decode(16, [200, 200, 130], 1, 64, "bf16")
    keep = [i for i in range(200) if not 64 <= i < 128]
    p.table[0, 1] = p.desc.n_pages
    p.table[2, 0] = -1
    p.seq[1] = 64 * p.table.shape[1] + 1
    p.run()
    _dev_error(5)
    p.rows[0] = tuple(t[keep] for t in p.rows[0])
    p.rows[2] = tuple(t[64:] for t in p.rows[2])
    p.lens = [len(keep), 0, 66]
    p.check()
    p.seq[1] = -1
    p.run()
    _dev_error(5)
    p.check()


# ----------------------------------------------------------------- expanded

class Prefill:
    """Packed sequences with NaN rows behind the last one."""

    def __init__(self, H, lq, lk, causal, seed=0, tail=5, q_std=1.0):
        g = gen(seed + H + sum(lq))
        self.H, self.lq, self.lk, self.causal = H, lq, lk, causal
        Tq, Tk = sum(lq) + tail, sum(lk) + tail
        self.q = randn(g, (Tq, H, 200), q_std)[..., :192]
        kv = randn(g, (Tk, H, 256))
        self.kr = randn(g, (Tk, 72))[:, :64]
        if tail:
            self.q[-tail:], kv[-tail:], self.kr[-tail:] = (float("nan"),) * 3
        self.kn, self.v = kv[..., :128], kv[..., 128:]
        cu = lambda n: ints([sum(n[:i]) for i in range(len(n) + 1)])
        self.cu_q, self.cu_k = cu(lq), cu(lk)
        full = lambda *s: torch.full(s, SENTINEL, dtype=torch.bfloat16, device=DEV)
        self.out = full(Tq, H, 128)
        self.lse = torch.full((H, Tq), SENTINEL, device=DEV)
        self.do = randn(g, (Tq, H, 128))
        self.dq, self.dkr, self.dkv = full(Tq, H, 192), full(Tk, 64), full(Tk, H, 256)
        self.ws = torch.empty(fs.fs_latent_prefill_backward_ws_bytes(H, Tq, Tk), dtype=torch.uint8, device=DEV)
        self.ws.fill_(0xFF)
        self.tail = tail

    def args(self):
        return (self.q, self.kn, self.kr, self.v, self.cu_q, self.cu_k, self.causal, SCALE)

    def forward(self):
        fs.fs_latent_prefill(*self.args(), self.out, self.lse)

    def backward(self):
        fs.fs_latent_prefill_backward(*self.args(), self.out, self.lse, self.do, self.dq, self.dkv[..., :128],
                                      self.dkr, self.dkv[..., 128:], self.ws)

    def seqs(self):
        a = b = 0
        for n, m in zip(self.lq, self.lk):
            yield slice(a, a + n), slice(b, b + m), ref.visible(n, m, self.causal, DEV)
            a, b = a + n, b + m

    def head(self, sq, sk, h):
        k = torch.cat([self.kn[sk, h], self.kr[sk]], -1)
        return self.q[sq, h], k, self.v[sk, h]

    def check_forward(self):
        for sq, sk, vis in self.seqs():
            for h in range(self.H):
                q, k, v = self.head(sq, sk, h)
                want, wl, tol, tl = ref.attend(q, k, v, SCALE, vis)
                ref.within(self.out[sq, h], want, tol, "out")
                ref.within(self.lse[h, sq], wl, tl, "lse")
        n = sum(self.lq)
        assert (self.out[n:] == SENTINEL).all() and (self.lse[:, n:] == SENTINEL).all()

    def check_backward(self):
        for sq, sk, vis in self.seqs():
            dkr = tkr = 0.0
            for h in range(self.H):
                q, k, v = self.head(sq, sk, h)
                want, tol = ref.attend_grad(q, k, v, SCALE, vis, self.out[sq, h], self.lse[h, sq], self.do[sq, h])
                ref.within(self.dq[sq, h], want[0], tol[0], "dq")
                ref.within(self.dkv[sk, h, :128], want[1][:, :128], tol[1][:, :128], "dk_nope")
                ref.within(self.dkv[sk, h, 128:], want[2], tol[2], "dv")
                # the sum over heads rounds once: fp32 head sums, then bf16
                t = tol[1][:, 128:] - ref.HALF * want[1][:, 128:].abs()
                dkr, tkr = dkr + want[1][:, 128:], tkr + t + 8 * self.H * ref.ULP32 * want[1][:, 128:].abs()
            ref.within(self.dkr[sk], dkr, tkr + ref.HALF * dkr.abs(), "dk_rope")
        n, m = sum(self.lq), sum(self.lk)
        assert (self.dq[n:] == SENTINEL).all() and (self.dkr[m:] == SENTINEL).all()
        assert (self.dkv[m:] == SENTINEL).all()


PREFILL = [
    (1, [1], [1], True),
    (2, [128], [128], True),
    (3, [127, 1, 129], [127, 1, 129], True),
    (2, [300], [300], False),
    (16, [257, 0, 64, 5], [257, 3, 64, 0], True),
    (4, [1, 100, 130], [513, 228, 140], True),              # behind a prefix
    (2, [200, 5], [70, 1], True),                           # more queries than keys: rows that see nothing
    (5, [33, 400], [290, 17], False),
    (2, [1100], [1100], True),
    (128, [70, 3], [70, 90], True),
]


@pytest.mark.parametrize("H,lq,lk,causal", PREFILL)
def test_prefill(H, lq, lk, causal):
    p = Prefill(H, lq, lk, causal)
    p.forward()
    _no_dev_error()
    p.check_forward()


@pytest.mark.parametrize("H,lq,lk,causal", PREFILL)
def test_prefill_backward(H, lq, lk, causal):
    p = Prefill(H, lq, lk, causal)
    p.forward()
    p.backward()
    _no_dev_error()
    p.check_backward()


def test_prefill_large_scores():
    p = Prefill(2, [200, 77], [200, 77], True, q_std=30.0)
    p.forward()
    p.backward()
    _no_dev_error()
    p.check_forward()
    p.check_backward()


def test_prefill_no_tail_and_neighbours():
    """A NaN in one sequence stays in it."""
    p = Prefill(2, [100, 60], [100, 60], True, tail=0)
    p.kn[120], p.v[130], p.kr[125], p.q[140], p.do[141] = (float("nan"),) * 5
    p.forward()
    p.backward()
    _no_dev_error()
    p.lq, p.lk = [100], [100]
    p.tail = 60
    p.out[100:], p.lse[:, 100:], p.dq[100:], p.dkr[100:], p.dkv[100:] = (SENTINEL,) * 5
    p.check_forward()
    p.check_backward()


def test_prefill_difference_quotient():
    """The gradient against central differences of sum(d_out . out), evaluated in 64 bits."""
    p = Prefill(2, [40], [40], True, tail=0)
    p.forward()
    p.backward()
    _no_dev_error()
    g = gen(9)

    def loss(q, kn, kr, v):
        vis, s = ref.visible(40, 40, True, DEV), 0.0
        for h in range(2):
            o, _, _, _ = ref.attend(q[:, h], torch.cat([kn[:, h], kr], -1), v[:, h], SCALE, vis)
            s = s + (o * p.do[:, h].double()).sum()
        return s

    base = [t.double() for t in (p.q, p.kn, p.kr, p.v)]
    for i, grad in enumerate((p.dq, p.dkv[..., :128], p.dkr, p.dkv[..., 128:])):
        d = torch.randn(base[i].shape, generator=g, device=DEV, dtype=torch.float64)
        eps = 1e-4
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + eps * d, base[i] - eps * d
        num = (loss(*up) - loss(*dn)) / (2 * eps)
        ana = (grad.double() * d).sum()
        # every gradient element within 3 half steps of bf16 of a sum of about 40 terms of its size
        tol = 3 * ref.HALF * (grad.double().abs() * d.abs()).sum() + 1e-4
        assert abs(num - ana) < tol, (i, float(num), float(ana), float(tol))


def test_prefill_repeats_and_replays_bit_identically():
    p = Prefill(4, [300, 129], [300, 200], True)
    p.forward()
    p.backward()
    _no_dev_error()
    keep = [t.clone() for t in (p.out, p.lse, p.dq, p.dkr, p.dkv)]
    p.ws.fill_(0xAA)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward()
        p.backward()
    for _ in range(2):
        for t in (p.out, p.lse, p.dq, p.dkr, p.dkv):
            t.fill_(SENTINEL)
        graph.replay()
        _no_dev_error()
        assert all(torch.equal(a, b) for a, b in zip(keep, (p.out, p.lse, p.dq, p.dkr, p.dkv)))


def test_prefill_many_sequences_and_heads_outside_rows():
    """Hundreds of short sequences, empty ones among them, with operands laid out head by head."""
    g = torch.Generator().manual_seed(5)
    lq = [int(x) for x in torch.randint(0, 9, (300,), generator=g)]
    lk = [int(n + x) if n else int(x) for n, x in zip(lq, torch.randint(0, 9, (300,), generator=g))]
    p = Prefill(3, lq, lk, True)
    p.forward()
    p.backward()
    _no_dev_error()
    p.check_forward()
    p.check_backward()
    hm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    q, kn, v, do, out = hm(p.q), hm(p.kn), hm(p.v), hm(p.do), hm(torch.full_like(p.out, SENTINEL))
    lse = torch.full_like(p.lse, SENTINEL)
    fs.fs_latent_prefill(q, kn, p.kr, v, p.cu_q, p.cu_k, True, SCALE, out, lse)
    assert torch.equal(out, p.out) and torch.equal(lse, p.lse)
    dq, dkn, dv = (hm(torch.full_like(t, SENTINEL)) for t in (q, kn, v))
    dkr = torch.full_like(p.dkr, SENTINEL)
    fs.fs_latent_prefill_backward(q, kn, p.kr, v, p.cu_q, p.cu_k, True, SCALE, out, lse, do, dq, dkn, dkr, dv, p.ws)
    _no_dev_error()
    assert torch.equal(dq, p.dq) and torch.equal(dkr, p.dkr)
    assert torch.equal(dkn, p.dkv[..., :128]) and torch.equal(dv, p.dkv[..., 128:])


def test_prefill_bad_offsets():
    """Offsets that run backwards or past the rows leave their sequence and set the error word."""
    for bad in ([0, 200, 100], [0, 100, 10 ** 6], [0, -7, 100]):
        p = Prefill(2, [100, 50], [100, 50], True)
        p.cu_q.copy_(ints(bad))
        p.forward()
        _dev_error(2)
        assert (p.out[150:] == SENTINEL).all()
        p = Prefill(2, [100, 50], [100, 50], True)
        p.forward()
        _no_dev_error()
        p.cu_k.copy_(ints(bad))
        p.backward()
        _dev_error(2)


# ------------------------------------------------- the operators as one layer

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_sub_layer_prefill_then_decode(cache):
    """A prompt through rotary, cache write and expanded attention, then two new tokens through the absorbed form
    over the cache: the absorbed result times W_UV equals the expanded form over all tokens."""
    g = gen(21)
    H, T, n_q, page = 16, 150, 2, 48
    L = T + n_q
    w_uk, w_uv = (torch.randn((H, 128, 512), generator=g, device=DEV) / math.sqrt(512) for _ in range(2))
    c, kr = randn(g, (L, 512)), randn(g, (L, 64))
    q = randn(g, (L, H, 192))
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    rope = fs.make_rope(64, "interleaved", **SCALED)
    desc = fs.make_latent_cache(5, page, cache)
    buf = fs.latent_cache_empty(desc)
    slots = (torch.arange(L, device=DEV) + page).contiguous()                  # pages 1 ..
    fs.fs_rope(rope, pos, q[..., 128:], q[..., 128:])
    fs.fs_latent_cache_write(desc, c[:T], kr[:T], slots[:T], buf, rope=rope, pos=pos[:T])         # the prompt
    fs.fs_latent_cache_write(desc, c[T:], kr[T:], slots[T:], buf, rope=rope, pos=pos[T:])         # the new tokens
    cb, kb = torch.empty_like(c), torch.empty_like(kr)
    fs.fs_latent_cache_read(desc, buf, slots, cb, kb)
    kn = torch.einsum("hnl,tl->thn", w_uk, cb.float()).to(torch.bfloat16)
    v = torch.einsum("hnl,tl->thn", w_uv, cb.float()).to(torch.bfloat16)
    out = torch.empty((L, H, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((H, L), device=DEV)
    cu = ints([0, L])
    fs.fs_latent_prefill(q, kn, kb, v, cu, cu, True, SCALE, out, lse)
    ql = torch.einsum("thn,hnl->thl", q[T:, :, :128].float(), w_uk).to(torch.bfloat16)
    o = torch.empty((n_q, H, 512), dtype=torch.bfloat16, device=DEV)
    ldec = torch.empty((n_q, H), device=DEV)
    fs.fs_latent_decode(desc, ql, q[T:, :, 128:], buf, ints([[1, 2, 3, 4]]), ints([L]), SCALE, o, ldec,
                        _decode_ws(H, 1, n_q))
    _no_dev_error()
    got = torch.einsum("hnl,thl->thn", w_uv.double(), o.double())
    # both sides round their own operands to bf16 (k_n, v, q_l, p, out): a handful of half steps of values of size one
    s_tol = 2 * ref.HALF * SCALE * (q[T:].double().norm(dim=-1) * math.sqrt(192)).amax()
    assert (ldec.double() - lse[:, T:].T.double()).abs().max() < s_tol
    assert (got - out[T:].double()).norm() < (4 * ref.HALF + 2 * s_tol) * out[T:].double().norm()
