"""The router's balance loss, counts and gradient against the 64-bit definition,
against differences of the loss, and inside the trainer's step.

Tolerances.  A score is an exponential (2 units of 2^-23 plus its argument's
rounding, |z| 2^-23 for logits below 32) over a sum of E of them, so within
(2 |z| + 8 + E / 32 + 10) 2^-23 < 2^-16 of itself; mean scores add T rounded
terms in a tree of at most T / 8 + 40 steps per lane, 2^-24 each; the gradient's
factor f - <f, s> is a difference whose error is that of <f, s>, at most 2^-16
max f.  All bounds are sums of those."""
import math

import pytest
import torch

from mixture_experts_layer_expert_gb300 import configs, fs, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -16
GATES = ["softmax", "softmax_renorm", "sigmoid", "sigmoid_norm"]


def no_error():
    torch.cuda.synchronize()
    assert fs.fs_get_error() == (0, 0)


def reference(z, idx, gate, coef, cu, mask, bias=None, d_loss=1.0):
    """counts, tokens, probs, loss, gradient in 64 bits, sequence by sequence."""
    T, E = z.shape
    k, S = idx.shape[1], len(cu) - 1
    z = z.double() + (0 if bias is None else bias.double())
    counts, tokens = torch.zeros((S, E), dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    probs, grad, loss = torch.zeros((S, E)).double(), torch.full((T, E), math.nan).double(), 0.0
    for q in range(S):
        rows = torch.arange(cu[q], cu[q + 1])
        grad[rows] = 0.0
        rows = rows[mask[rows] != 0]
        n = tokens[q] = len(rows)
        if n == 0:
            continue
        counts[q] = torch.bincount(idx[rows].flatten().long(), minlength=E).int()
        leaf = z[rows].requires_grad_()
        if gate.startswith("softmax"):
            s = torch.softmax(leaf, 1)
        else:
            ls = torch.nn.functional.logsigmoid(leaf)
            s = torch.softmax(ls, 1)                         # sigma / sum sigma, at any depth
        part = coef / S * (counts[q].double() * E / (k * n) * s.mean(0)).sum()
        part.backward()
        probs[q], grad[rows] = s.mean(0).detach(), leaf.grad * d_loss
        loss += float(part.detach())
    return counts, tokens, probs, loss, grad


def call(z, idx, gate, coef, cu=None, mask=None, bias=None, d_loss=None, fill=5.0):
    T, E = z.shape
    S = 1 if cu is None else len(cu) - 1
    desc = fs.make_balance(T, E, idx.shape[1], gate, S, coef)
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    new = lambda *s, dt=torch.float32: torch.full(s, 77, dtype=dt, device=DEV)
    counts, tokens = new(S, E, dt=torch.int32), new(S, dt=torch.int32)
    probs, loss, dz = new(S, E), new(1), torch.full((T, E), fill, device=DEV)
    ws = torch.full((fs.fs_balance_ws_bytes(desc),), 0xFF, dtype=torch.uint8, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)
    kw = dict(bias=dev(bias), cu=cu, mask=dev(mask))
    zd = z if z.is_cuda else z.to(DEV)
    fs.fs_balance_loss(desc, zd, idx.to(DEV), counts, tokens, probs, loss, ws, **kw)
    fs.fs_balance_loss_backward(desc, zd, counts, tokens, dev(d_loss), dz, **kw)
    no_error()
    return [t.cpu() for t in (counts, tokens, probs, loss, dz)]


def check(got, want, T, E, gate, coef, S, d_loss=1.0, fill=5.0):
    counts, tokens, probs, loss, dz = got
    wc, wt, wp, wl, wg = want
    assert torch.equal(counts, wc) and torch.equal(tokens, wt)
    steps = (T / 8 + 40) * 2.0 ** -24
    assert ((probs.double() - wp).abs() <= wp * (REL + steps)).all()
    assert abs(float(loss) - wl) <= abs(wl) * (REL + steps + (E + S) * 2.0 ** -24) + 1e-45
    left = wg.isnan()
    assert (dz[left] == fill).all()
    # |dz| error: scale s (REL |f - <f,s>| + REL max f (the difference's own)), scale = d_loss coef / (S n), f <= E / k, n >= 1
    off = (dz.double() - wg).abs()[~left]
    return off


def bound(z, idx, gate, coef, cu, mask, bias, d_loss):
    """Error allowed to each gradient entry: |scale| s max_f 4 REL (times 1 - sigma, at most 1)."""
    T, E = z.shape
    k, S = idx.shape[1], len(cu) - 1
    zz = z.double() + (0 if bias is None else bias.double())
    s = torch.softmax(zz if gate.startswith("softmax") else torch.nn.functional.logsigmoid(zz), 1)
    room = torch.zeros((T, E)).double()
    for q in range(S):
        rows = torch.arange(cu[q], cu[q + 1])
        rows = rows[mask[rows] != 0]
        if len(rows) == 0:
            continue
        f = torch.bincount(idx[rows].flatten().long(), minlength=E).double() * E / (k * len(rows))
        room[rows] = abs(d_loss * coef) / (S * len(rows)) * s[rows] * f.max() * 4 * REL
    return room + 1e-44


CASES = [
    # T, E, k, borders, masked share, bias, row padding
    (1, 1, 1, None, 0, False, 0), (1, 8, 2, None, 0, True, 0), (2, 3, 3, None, 0, False, 1), (17, 33, 5, None, 0.5, True, 3),
    (256, 8, 2, None, 0, False, 0), (1000, 64, 6, None, 0.1, False, 0), (777, 130, 8, None, 0, True, 2),
    (5000, 256, 8, None, 0, False, 0), (300, 512, 16, None, 0.3, True, 0), (129, 511, 16, None, 0, False, 5),
    (1000, 128, 8, [0, 0, 1, 400, 400, 990, 990], 0.2, True, 4), (64, 16, 4, [3, 10, 60], 0, False, 0),
    (500, 12, 3, list(range(0, 501)), 0, False, 0), (9000, 40, 4, [0, 16, 32, 48, 4000, 8999], 0.4, True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d" % c[:2])
@pytest.mark.parametrize("gate", GATES)
def test_against_definition(case, gate):
    T, E, k, cu, share, with_bias, pad = case
    g = torch.Generator().manual_seed(T + E)
    full = torch.randn((T, E + pad), generator=g) * 2 + 0.5 * torch.randn((1, E + pad), generator=g)
    z = full[:, :E]
    bias = torch.randn(E, generator=g) if with_bias else None
    idx = torch.topk(z if bias is None else z + bias, k, 1).indices.int()
    mask = (torch.rand(T, generator=g) >= share).to(torch.uint8) if share else None
    d_loss = torch.tensor([-1.75])
    got = call(full.to(DEV)[:, :E], idx, gate, 0.03, cu, mask, bias, d_loss)
    borders, on = cu or [0, T], torch.ones(T) if mask is None else mask
    want = reference(z, idx, gate, 0.03, borders, on, bias, -1.75)
    off = check(got, want, T, E, gate, 0.03, len(borders) - 1)
    room = bound(z, idx, gate, 0.03, borders, on, bias, -1.75)
    assert (off <= room[~want[4].isnan()]).all(), "%.3e over its bound" % float((off - room[~want[4].isnan()]).max())


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_far_logits(gate):
    """Rows far from zero, experts at -infinity, rows of -infinity: finite, and as in 64 bits."""
    T, E, k = 40, 24, 2
    g = torch.Generator().manual_seed(1)
    z = torch.randn((T, E), generator=g)
    z[:8] += 80.0
    z[8:16] -= 90.0
    z[16:20, 5:9] = -math.inf
    idx = torch.topk(z, k, 1).indices.int()
    z2 = z.clone()
    z2[20:22] = -math.inf
    counts, tokens, probs, loss, dz = call(z2, idx, gate, 1.0)
    assert probs.isfinite().all() and dz.isfinite().all() and (dz[20:22] == 0).all()
    ls = z2.double() if gate == "softmax" else torch.nn.functional.logsigmoid(z2.double())
    s = torch.softmax(ls, 1).nan_to_num(0.0)
    # z near 90: the argument's rounding alone is 90 * 2^-23 relative, and twice that with the row's maximum
    assert ((probs[0].double() - s.mean(0)).abs() <= s.mean(0) * 4 * REL).all()
    f = counts[0].double() * E / (k * T)
    d = s / T * (f - (f * s).sum(1, keepdim=True)) * (1 if gate == "softmax" else torch.sigmoid(-z2.double()))
    assert ((dz.double() - d).abs() <= s / T * f.max() * 8 * REL + 1e-44).all()


def test_nan_stays_in_its_row_and_sequence():
    T, E, k = 64, 16, 2
    g = torch.Generator().manual_seed(2)
    z = torch.randn((T, E), generator=g)
    idx = torch.topk(z, k, 1).indices.int()
    clean = call(z, idx, "softmax", 1.0, [0, 32, 64])
    z[40, 3] = math.nan
    z[41, 2] = math.inf
    got = call(z, idx, "softmax", 1.0, [0, 32, 64])
    assert torch.equal(got[2][0], clean[2][0]) and got[2][1].isnan().all() and got[3].isnan().all()
    rows = torch.tensor([i for i in range(T) if i not in (40, 41)])
    assert torch.equal(got[4][rows], clean[4][rows]) and got[4][40].isnan().all()
    mask = torch.ones(T, dtype=torch.uint8)
    mask[40] = mask[41] = 0
    got = call(z, idx, "softmax", 1.0, [0, 32, 64], mask)
    assert all(t.isfinite().all() for t in got[2:]) and (got[4][40:42] == 0).all()


def test_bad_indices_and_borders_are_reported():
    T, E, k = 50, 8, 2
    z = torch.randn((T, E), generator=torch.Generator().manual_seed(4)).to(DEV)
    idx = torch.topk(z, k, 1).indices.int()
    want = torch.bincount(idx.flatten().long().cpu(), minlength=E)
    for bad in (-1, E, 2 ** 31 - 1):
        i2 = idx.clone()
        was = int(i2[7, 1])
        i2[7, 1] = bad
        desc = fs.make_balance(T, E, k, "softmax", 1, 1.0)
        new = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
        counts, ws = new(1, E, dt=torch.int32), new(fs.fs_balance_ws_bytes(desc), dt=torch.uint8)
        fs.fs_balance_loss(desc, z, i2, counts, new(1, dt=torch.int32), new(1, E), new(1), ws)
        torch.cuda.synchronize()
        assert fs.fs_get_error() == (5, 1)
        w = want.clone()
        w[was] -= 1
        assert torch.equal(counts[0].cpu().long(), w)
    desc = fs.make_balance(T, E, k, "softmax", 2, 1.0)
    ws = new(fs.fs_balance_ws_bytes(desc), dt=torch.uint8)
    for bad in ([0, 60, 60], [-3, 20, 50], [0, 30, 20], [0, 10, 2 ** 31 - 1]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        counts, tokens = new(2, E, dt=torch.int32), new(2, dt=torch.int32)
        fs.fs_balance_loss(desc, z, idx, counts, tokens, new(2, E), new(1), ws, cu=cu)
        torch.cuda.synchronize()
        assert fs.fs_get_error() == (5, 2)
        dz = torch.full((T, E), 3.0, device=DEV)
        fs.fs_balance_loss_backward(desc, z, counts, tokens, None, dz, cu=cu)
        torch.cuda.synchronize()
        fs.fs_get_error()


@pytest.mark.parametrize("gate", GATES)
def test_gradient_against_differences(gate):
    """Central differences of the 64-bit loss with the counts held: the gradient is the loss's."""
    T, E, k = 9, 6, 2
    g = torch.Generator().manual_seed(6)
    z = torch.randn((T, E), generator=g)
    idx = torch.topk(z, k, 1).indices.int()
    dz = call(z, idx, gate, 2.0)[4].double()
    on, step = torch.ones(T), 1e-4
    for t, e in [(0, 0), (3, 5), (8, 2), (4, 4)]:
        up, down = z.double().clone(), z.double().clone()
        up[t, e] += step
        down[t, e] -= step
        d = (reference(up, idx, gate, 2.0, [0, T], on)[3] - reference(down, idx, gate, 2.0, [0, T], on)[3]) / (2 * step)
        # third derivatives of the scores are below 1: step^2 / 6, and 1e-16 / step of rounding
        assert abs(float(dz[t, e]) - d) <= 2.0 * E / k / T * (step ** 2 + 4 * REL) + 1e-11


def test_repeats_replays_and_streams():
    T, E, k = 3000, 96, 4
    g = torch.Generator().manual_seed(8)
    z = torch.randn((T, E), generator=g)
    idx = torch.topk(z, k, 1).indices.int()
    a = call(z, idx, "sigmoid_norm", 0.5, [0, 700, 2900])
    b = call(z, idx, "sigmoid_norm", 0.5, [0, 700, 2900])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    desc = fs.make_balance(T, E, k, "sigmoid_norm", 2, 0.5)
    cu = torch.tensor([0, 700, 2900], dtype=torch.int32, device=DEV)
    new = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
    counts, tokens, probs, loss = new(2, E, dt=torch.int32), new(2, dt=torch.int32), new(2, E), new(1)
    dz, ws, zd, di = torch.full((T, E), 5.0, device=DEV), new(fs.fs_balance_ws_bytes(desc), dt=torch.uint8), z.to(DEV), idx.to(DEV)

    def both(stream=None):
        fs.fs_balance_loss(desc, zd, di, counts, tokens, probs, loss, ws, cu=cu, stream=stream)
        fs.fs_balance_loss_backward(desc, zd, counts, tokens, None, dz, cu=cu, stream=stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for go in (graph.replay, graph.replay, lambda: both(side)):
        for t in (counts, tokens, probs, loss):
            t.zero_()
        torch.cuda.synchronize()
        go()
        no_error()
        assert all(torch.equal(x, y.cpu()) for x, y in zip(a, (counts, tokens, probs, loss, dz)))


@pytest.mark.parametrize("gate", GATES)
def test_in_the_training_step(gate):
    """The trainer's router gradient with the balance term against the one without it plus the term's own:
    dW_R gains dz^T u, dx gains dz W_R (last block: nothing else reads its logits)."""
    cfg = configs.LayerConfig("bal", T=300, d=256, E=12, k=2, c=128, n_shared=1, c_shared=128, L=2, gate=gate, dtype="bf16")
    prob = synth.make_problem(cfg, device=DEV)
    tr = fs.FarSkipTrainer(cfg, prob["blocks"])
    tr.forward(prob["x"])
    d_o = torch.randn((cfg.T, cfg.d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    zero = torch.zeros_like(d_o)
    plain = {k: v.clone() for k, v in tr.backward(d_o)[1][-1].items()}
    loss, counts = tr.balance_loss(0.7)
    no_error()
    assert loss.shape == (2, 1) and torch.equal(counts.sum((1, 2)).cpu(), torch.full((2,), cfg.T * cfg.k))
    tr.backward(zero, d_balance=torch.tensor([0.0], device=DEV))
    no_error()
    assert all(not g.any() for gr in tr.grads for g in gr.values())      # nothing but the balance term's zero
    tr.backward(zero, d_balance=torch.tensor([200.0], device=DEV))
    no_error()
    alone, dx = tr.grads, tr.dx.clone()
    # the last block by itself: u and z are its saved input and logits
    z, idx = tr._routing(1)
    def saved(ptr, shape, dt):
        at = ptr.value - tr.saved.data_ptr()
        n = math.prod(shape) * 4
        return tr.saved[at:at + n].view(dt).view(shape)
    zt, it = saved(z, (cfg.T, cfg.E), torch.float32).cpu(), saved(idx, (cfg.T, cfg.k), torch.int32).cpu()
    half = tr.saved.numel() // 2
    u = tr.saved[half:half + cfg.T * cfg.d * 2].view(torch.bfloat16).view(cfg.T, cfg.d).cpu().double()
    on = torch.ones(cfg.T)
    want = reference(zt, it, gate, 0.7, [0, cfg.T], on, None, 200.0)
    assert abs(float(loss[1]) - want[3]) <= abs(want[3]) * 2 * REL
    dw = want[4].T @ u
    # dz enters the product as bf16 (half a step, 2^-8), sums fp32
    room = want[4].abs().T @ u.abs() * (2.0 ** -8 + cfg.T * 2.0 ** -23)
    assert ((alone[-1]["dW_R"].cpu().double() - dw).abs() <= room + 1e-30).all()
    # partial wiring: the second block reads o_1* = x + S_1, so its term reaches x and the first shared experts, not the routed
    assert dx.any() and alone[0]["dW1s"].any() and not alone[0]["dW1"].any()
    tr.backward(d_o)                                                         # and without it nothing has changed
    no_error()
    assert all(torch.equal(plain[k], v) for k, v in tr.grads[-1].items())


def test_backward_needs_its_loss():
    cfg = configs.LayerConfig("bal", T=64, d=128, E=4, k=1, c=128, n_shared=0, c_shared=0, L=1, gate="softmax", dtype="bf16")
    prob = synth.make_problem(cfg, device=DEV)
    tr = fs.FarSkipTrainer(cfg, prob["blocks"])
    tr.forward(prob["x"])
    with pytest.raises(fs.FsError):
        tr.backward(torch.zeros((64, 128), device=DEV), d_balance=torch.ones(1, device=DEV))


def test_borders_change_between_steps():
    """Steps of one trainer with other borders, on the current and on another stream, against a fresh trainer's step: what
    rows that are now outside every sequence had in an earlier step does not come back."""
    cfg = configs.LayerConfig("bal", T=300, d=256, E=12, k=2, c=128, n_shared=0, c_shared=0, L=2, gate="softmax_renorm",
                              dtype="bf16")
    prob = synth.make_problem(cfg, device=DEV)
    d_o = torch.randn((cfg.T, cfg.d), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    one = torch.tensor([100.0], device=DEV)

    def step(tr, cu, stream=None):
        tr.forward(prob["x"], stream=stream)
        tr.balance_loss(0.5, cu=cu, stream=stream)
        dx, grads = tr.backward(d_o, d_balance=one, stream=stream)
        torch.cuda.synchronize()
        no_error()
        return [dx.clone()] + [g[n].clone() for g in grads for n in sorted(g)]

    borders = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 150, 300], [0, 40, 90], [100, 100, 101], [0, 90])]
    side = torch.cuda.Stream()
    tr = fs.FarSkipTrainer(cfg, prob["blocks"])
    torch.cuda.synchronize()
    for i, cu in enumerate(borders):
        got = step(tr, cu, side if i % 2 else None)
        want = step(fs.FarSkipTrainer(cfg, prob["blocks"]), cu)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_a_refused_loss_is_no_loss():
    cfg = configs.LayerConfig("bal", T=64, d=256, E=8, k=2, c=128, n_shared=0, c_shared=0, L=1, gate="sigmoid_norm",
                              dtype="bf16")
    prob = synth.make_problem(cfg, device=DEV)
    tr = fs.FarSkipTrainer(cfg, prob["blocks"])
    tr.forward(prob["x"])
    tr.balance_loss(1.0)
    for bad in (dict(cu=torch.tensor([0, 64], device=DEV)), dict(mask=torch.ones(63, dtype=torch.uint8, device=DEV))):
        with pytest.raises(fs.FsError):
            tr.balance_loss(1.0, **bad)
        with pytest.raises(fs.FsError):
            tr.backward(torch.zeros((cfg.T, cfg.d), device=DEV), d_balance=torch.ones(1, device=DEV))


@pytest.mark.parametrize("gate", GATES)
def test_every_expert_chosen(gate):
    """k = E: every f is one whatever the scores, so that the loss is coef and its gradient exactly zero."""
    g = torch.Generator().manual_seed(8)
    for T, E in ((1, 1), (33, 2), (1201, 16)):
        z, idx = torch.randn((T, E), generator=g) * 3, torch.argsort(torch.randn((T, E), generator=g), 1).int()
        counts, tokens, probs, loss, dz = call(z, idx, gate, 0.9)
        assert (counts == T).all() and not dz.any()
        assert abs(float(loss) - 0.9) <= 0.9 * (REL + (T / 8 + 40 + E) * 2.0 ** -24)


@pytest.mark.parametrize("gate", GATES)
def test_even_counts_leave_no_gradient(gate):
    T, E, k = 640, 8, 2
    idx = ((torch.arange(T)[:, None] * k + torch.arange(k)) % E).int()
    got = call(torch.randn((T, E), generator=torch.Generator().manual_seed(2)), idx, gate, 1.0)
    assert (got[0] == T * k // E).all() and not got[4].any()
