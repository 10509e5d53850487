"""The output head's cross entropy and its gradient against their definitions
in 64 bits.

Bounds, with e = 2^-24 (fp32) and b = 2^-8 (bf16) unit roundoffs.  A product
over K terms on the tensor cores adds 16 at a time into fp32, so it is off by
at most (K / 16 + 16) 4 e times the sum of the terms' magnitudes.  Logits are
off by dz, that bound over dim.  Then
  loss: 2 dz (the target's logit and the log of the sum) and 64 e of its size;
  dh:   a term of sum p W is off by b (p in bf16) and 4 dz, the sum over the
        vocabulary by the bound above, the target's term by 4 dz, the result by b;
  dW:   the same with 2 b (p, and h with its factor, in bf16) over the tokens."""
import math

import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu

E, B = 2.0 ** -24, 2.0 ** -8


def _acc(k):
    return (k / 16 + 16) * 4 * E


def _inputs(n, v, d, seed, ignored=0.2, scale=2.0, ids=torch.int64):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((n, d), generator=g).bfloat16()
    w = (torch.randn((v, d), generator=g) * (scale / math.sqrt(d))).bfloat16()
    t = (torch.rand(n, generator=g, dtype=torch.float64) ** 3 * v).long().clamp_(0, v - 1)
    bad = torch.tensor([-100, -1, v, v + 9])[torch.randint(0, 4, (n,), generator=g)]
    t = torch.where(torch.rand(n, generator=g) < ignored, bad, t)
    return h, w, t.to(ids)


def _reference(h, w, t, g=None, ignore=-100):
    """Exact loss, dh, dW and their bounds (without the results' rounding)."""
    n, v, d = h.shape[0], w.shape[0], h.shape[1]
    hd, wd, t = h.double().cuda(), w.double().cuda(), t.long().cuda()
    ok = (t >= 0) & (t < v) & (t != ignore)
    i = ok.nonzero()[:, 0]
    loss, dh, dw = (torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((n,), (n, d), (v, d)))
    bl, bh, bw = torch.zeros_like(loss), torch.zeros_like(dh), torch.zeros_like(dw)
    if len(i) == 0:
        return (loss, dh, dw), (bl, bh, bw)
    g = torch.full((n,), 1.0 / len(i), dtype=torch.float64) if g is None else g.double()
    hi, ti, gi = hd[i], t[i], g.cuda()[i][:, None]
    z = hi @ wd.T
    dz = (_acc(d) * (hi.abs() @ wd.abs().T)).amax(1)
    loss[i] = torch.logsumexp(z, 1) - z.gather(1, ti[:, None])[:, 0]
    bl[i] = 2 * dz + 64 * E * (1 + loss[i].abs())
    p = torch.softmax(z, 1)
    hot = torch.zeros_like(p).scatter_(1, ti[:, None], 1.0)
    dl, rest = (p - hot) * gi, p * (1 - hot) * gi.abs()
    edge = ((1 - p) * hot * (64 * E + 8 * dz[:, None]) + hot * p * (4 * dz[:, None] + 64 * E)) * gi.abs()
    dh[i] = dl @ wd
    bh[i] = (rest * (1.1 * B + 4 * dz[:, None] + _acc(v) + 64 * E) + edge) @ wd.abs()
    dw += dl.T @ hi
    bw += (rest * (2.2 * B + 4 * dz[:, None] + _acc(n) + 64 * E) + edge * (1 + n * E)).T @ hi.abs()
    return (loss, dh, dw), (bl, bh, bw)


def _check(got, want, bound, names=("loss", "dh", "dW")):
    for x, y, b, name in zip(got, want, bound, names):
        u = B if x.dtype == torch.bfloat16 else 2 * E
        off = (x.double() - y).abs()
        lim = b + u * (y.abs() + b) + 1e-37
        assert torch.all(off <= lim), f"{name}: {float((off - lim).max()):.3g} over, {float((off / lim).max()):.3g} times"


SHAPES = [(1, 1, 8), (1, 2, 8), (2, 7, 16), (24, 1000, 64), (63, 255, 72), (64, 256, 64), (65, 257, 136),
          (127, 1003, 264), (128, 512, 128), (129, 5003, 192), (255, 300, 1000), (257, 513, 328), (300, 2050, 512),
          (700, 777, 64), (1030, 1300, 264), (40, 20011, 776), (512, 20, 72), (513, 20, 72), (5000, 600, 72)]


@pytest.mark.parametrize("n,v,d", SHAPES)
@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_loss_and_gradient(n, v, d, ignored):
    h, w, t = _inputs(n, v, d, n + v, ignored, ids=torch.int32 if n % 2 else torch.int64)
    want, bound = _reference(h, w, t)
    ws = torch.full((ns.head_workspace_size(n, v, d),), 255, dtype=torch.uint8, device="cuda")
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), workspace=ws)
    assert ns.read_error(ws) == 0
    assert [x.dtype for x in got] == [torch.float32, torch.bfloat16, torch.bfloat16]
    _check(got, want, bound)
    _check((ns.muon_head_loss(h.cuda(), w.cuda(), t.cuda()),), want[:1], bound[:1])


@pytest.mark.parametrize("pieces", [1, 2, 3, 5, 99])
@pytest.mark.parametrize("n,v,d", [(33, 1300, 64), (300, 2050, 264), (270, 5000, 776)])
def test_pieces_of_the_vocabulary(pieces, n, v, d):
    h, w, t = _inputs(n, v, d, 3)
    want, bound = _reference(h, w, t)
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), pieces=pieces)
    _check(got, want, bound)
    one = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), pieces=1)
    assert torch.equal(got[0], one[0]) and torch.equal(got[2], one[2])
    assert ns.head_workspace_size(n, v, d, True, 4) < ns.head_workspace_size(n, v, d, True, 1)


@pytest.mark.parametrize("pieces", [1, 3])
def test_given_loss_gradients_and_fp32_accumulation(pieces):
    n, v, d = 290, 1500, 136
    h, w, t = _inputs(n, v, d, 4)
    g = torch.randn(n, generator=torch.Generator().manual_seed(5))
    g[::7] = 0.0
    want, bound = _reference(h, w, t, g)
    dtable = torch.full((v, d), float("nan"), device="cuda")
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), dloss=g.cuda(), dtable=dtable, pieces=pieces)
    assert got[2] is dtable
    _check(got, want, bound)
    start = torch.randn((v, d), generator=torch.Generator().manual_seed(6)).cuda()
    more = start.clone()
    ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), dloss=g.cuda(), dtable=more, accumulate=True, pieces=pieces)
    assert torch.equal(more, start + dtable)


def _extreme(n, v, d, gap):
    """Targets whose logit lies `gap` below the largest (0: at random)."""
    h, w, t = _inputs(n, v, d, 7, 0.1, scale=1.0)
    top = torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(8))
    w[:, -1], h[:, -1] = 0, 1
    w[top[: n // 2] % v, -1] = gap
    return h, w, t


@pytest.mark.parametrize("gap", [30.0, 43.0, 60.0, 100.0, 300.0, -300.0])
@pytest.mark.parametrize("pieces", [1, 2])
def test_targets_far_from_the_largest_logit(gap, pieces):
    # Beyond a loss of 44 a row's tiles are computed again with its largest logit.
    n, v, d = 600, 900, 72
    h, w, t = _extreme(n, v, d, gap)
    want, bound = _reference(h, w, t)
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), pieces=pieces)
    _check(got, want, bound)
    _check((ns.muon_head_loss(h.cuda(), w.cuda(), t.cuda()),), want[:1], bound[:1])


def test_only_some_tiles_are_computed_again():
    n, v, d = 1100, 700, 64
    h, w, t = _inputs(n, v, d, 9, 0.0)
    w[5] = 0
    w[5, 0] = 100
    h[:, 0] = 0
    h[t == 60, 0] = 1.5  # sorted by target: these rows share a tile or two
    assert 0 < int((t == 60).sum()) < 200
    want, bound = _reference(h, w, t)
    assert float(want[0].max()) > 100
    _check(ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda()), want, bound)


def test_confident_tokens_keep_their_gradient():
    # p of the target within 1e-4 of one: its term is -g (1 - p), not the
    # difference of two rounded numbers.
    n, v, d = 64, 512, 64
    h, w, t = _inputs(n, v, d, 10, 0.0, scale=0.1)
    t = torch.arange(n) * 3
    w[:] = 0
    w[t] = torch.eye(d).bfloat16()[:n] * 16
    h = torch.eye(d).bfloat16()[:n]
    want, bound = _reference(h, w, t)
    assert 0 < float(want[0].max()) < 1e-3
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda())
    _check(got, want, bound)
    assert torch.all((got[1].double() - want[1]).abs() <= 0.02 * want[1].abs() + 1e-9)


@pytest.mark.parametrize("pieces", [1, 2])
def test_masked_tokens_touch_nothing(pieces):
    n, v, d = 300, 700, 136
    h, w, t = _inputs(n, v, d, 11, 0.5)
    bad = (t < 0) | (t >= v)
    args = dict(dloss=torch.rand(n).cuda(), pieces=pieces)
    ref = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), **args)
    dirty = h.clone()
    dirty[bad] = float("nan")
    dirty[bad.nonzero()[::2, 0]] = float("-inf")
    args["dloss"] = torch.where(bad.cuda(), float("nan"), args["dloss"])
    got = ns.muon_head_loss_grad(dirty.cuda(), w.cuda(), t.cuda(), **args)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert not ref[0][bad.cuda()].any() and not ref[1][bad.cuda()].any()
    assert torch.equal(ns.muon_head_loss(dirty.cuda(), w.cuda(), t.cuda()), ns.muon_head_loss(h.cuda(), w.cuda(), t.cuda()))


def test_no_token_has_a_loss():
    h, w, _ = _inputs(70, 600, 64, 12)
    t = torch.full((70,), 3)
    for dtype in (torch.bfloat16, torch.float32):
        dtable = torch.full((600, 64), float("nan"), dtype=dtype, device="cuda")
        got = ns.muon_head_loss_grad((h * float("nan")).cuda(), w.cuda(), t.cuda(), ignore_index=3, dtable=dtable)
        assert not any(x.any() or torch.isnan(x).any() for x in got)
    got = ns.muon_head_loss_grad(h[:0].cuda(), w.cuda(), t[:0].cuda())
    assert got[0].shape == (0,) and got[1].shape == (0, 64) and not got[2].any()
    got = ns.muon_head_loss_grad(h.cuda(), w[:0].cuda(), t.cuda())
    assert not got[0].any() and not got[1].any() and got[2].shape == (0, 64)
    assert not ns.muon_head_loss(h.cuda(), w[:0].cuda(), t.cuda()).any()


def test_ignore_index_inside_the_vocabulary():
    h, w, t = _inputs(90, 50, 64, 13, 0.0)
    want, bound = _reference(h, w, t, ignore=0)
    assert 0 < int((t == 0).sum())
    _check(ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), ignore_index=0), want, bound)


def test_bad_rows_give_what_the_definition_gives():
    # A NaN or infinite logit makes its own token's loss and dh NaN (and dW, a
    # sum over tokens); other tokens' losses and dh are untouched.
    n, v, d = 80, 300, 64
    h, w, t = _inputs(n, v, d, 14, 0.0)
    ref = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda())
    h[9, 4], h[33, 7] = float("nan"), float("inf")
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda())
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[9] = bad[33] = True
    assert torch.equal(torch.isnan(got[0]), bad) and torch.isnan(got[1][bad]).all()
    assert torch.equal(got[0][~bad], ref[0][~bad]) and torch.equal(got[1][~bad], ref[1][~bad])


def test_gradient_against_differences():
    # d/dt of sum(dloss * loss(h + t a, W + t c)) from central differences of
    # the definition in 64 bits.
    n, v, d, step = 50, 333, 72, 1e-4
    h, w, t = _inputs(n, v, d, 15)
    g = torch.randn(n, generator=torch.Generator().manual_seed(16)).double()
    a = torch.randn((n, d), generator=torch.Generator().manual_seed(17)).double()
    c = torch.randn((v, d), generator=torch.Generator().manual_seed(18)).double() / math.sqrt(d)
    ok = (t >= 0) & (t < v)

    def f(s):
        z = (h.double() + s * a) @ (w.double() + s * c).T
        return float((g * (torch.logsumexp(z, 1) - z.gather(1, torch.where(ok, t, 0)[:, None])[:, 0]))[ok].sum())

    slope = (f(step) - f(-step)) / (2 * step)
    dtable = torch.empty((v, d), device="cuda")
    _, dh, dw = ns.muon_head_loss_grad(h.cuda(), w.cuda(), t.cuda(), dloss=g.float().cuda(), dtable=dtable)
    _, (_, bh, bw) = _reference(h, w, t, g)
    got = float((dh.cpu().double() * a).sum() + (dw.cpu().double() * c).sum())
    lim = float(((bh.cpu() + B * dh.cpu().double().abs()) * a.abs()).sum() + (bw.cpu() * c.abs()).sum())
    assert abs(got - slope) <= lim + 1e3 * step * step


def test_deterministic_streams_and_graph_replay():
    n, v, d = 500, 3000, 264
    h, w, t = (x.cuda() for x in _inputs(n, v, d, 19))
    ref = ns.muon_head_loss_grad(h, w, t)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ns.muon_head_loss_grad(h, w, t), ref))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ns.muon_head_loss_grad(h, w, t)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ws = torch.empty(ns.head_workspace_size(n, v, d), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ns.muon_head_loss_grad(h, w, t, workspace=ws)
    h.copy_(h.flip(0))
    t.copy_(t.flip(0))
    ws.fill_(255)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0].flip(0))
    _check(got[1:], *(x[1:] for x in _reference(h.cpu(), w.cpu(), t.cpu())), names=("dh", "dW"))


def test_a_wait_that_runs_out_reports_and_returns():
    # A budget far below a healthy call's waits: the kernels give up, say so in
    # the error word, and the next call is right.
    n, v, d = 300, 4000, 512
    h, w, t = (x.cuda() for x in _inputs(n, v, d, 20))
    ref = ns.muon_head_loss_grad(h, w, t)
    ws = torch.empty(ns.head_workspace_size(n, v, d), dtype=torch.uint8, device="cuda")
    ns.set_wait_budget(1)
    try:
        ns.muon_head_loss_grad(h, w, t, workspace=ws)
        torch.cuda.synchronize()
        assert ns.read_error(ws) == ns._lib.DEVERR_WAIT_TIMEOUT
    finally:
        ns.set_wait_budget(0)
    got = ns.muon_head_loss_grad(h, w, t, workspace=ws)
    assert ns.read_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def _confident(n, v, d, level, seed):
    """Dense rows whose target holds about 1 - `level` of the probability; the
    logits are shifted together, so that the targets' are 25 to 45 and no
    power of two.  Every target is a row of its own."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((v, d), generator=g)
    common = torch.randn(d, generator=g)
    t = torch.randperm(v, generator=g)[:n]
    want = math.log(v / level)
    h = w[t] * (want / w[t].square().sum(1, keepdim=True)) + common * (17.3 / common.square().sum())
    return h.bfloat16(), (w + common).bfloat16(), t


@pytest.mark.parametrize("level", [1e-3, 1e-5, 1e-7])
@pytest.mark.parametrize("n,v,d", [(40, 1500, 768), (300, 1003, 2048), (70, 5003, 4096), (4200, 5003, 256)])
@pytest.mark.parametrize("pieces", [1, 2])
def test_confident_tokens_of_dense_rows(n, v, d, level, pieces):
    # With 1 - p small, the loss is 1 - p to first order and the target's term
    # -g (1 - p): both as exact, relative to themselves, as the gaps between the
    # logits are.  A gap is off by 2 dz, an exponential of it by 8 e and the
    # rounding of its argument (e times the gap, below 100), their sum by 64 e:
    # `off` of 1 - p, in all.
    h, w, t = _confident(n, v, d, level, n + d)
    hd, wd, tc = h.double().cuda(), w.double().cuda(), t.cuda()
    z = hd @ wd.T
    dz = (_acc(d) * (hd.abs() @ wd.abs().T)).amax(1, keepdim=True)
    off = 1.1 * (2 * dz + 256 * E)
    zt = z.gather(1, tc[:, None])
    hot = torch.zeros_like(z).scatter_(1, tc[:, None], 1.0)
    rest = (torch.exp(z - zt) * (1 - hot)).sum(1, keepdim=True)  # (1 - p) / p, without cancellation
    loss = torch.log1p(rest)
    assert level / 10 < float(rest.median()) < level * 10 and float(off.max()) < 0.01
    p = torch.exp(z - zt) * (1 - hot) / (1 + rest)
    want = [loss[:, 0], (p @ wd - rest / (1 + rest) * wd[tc]) / n, (p - hot * rest / (1 + rest)).T @ hd / n]
    top = rest / (1 + rest) * off / n  # of the targets' terms
    terms = p / n * (1.1 * B + 4 * dz + _acc(v) + 64 * E)
    bound = [(loss * off)[:, 0], terms @ wd.abs() + top * wd[tc].abs(),
             (p / n * (2.2 * B + 4 * dz + _acc(n) + 64 * E) + hot * top * (1 + n * E)).T @ hd.abs()]
    dtable = torch.empty((v, d), device="cuda")
    got = ns.muon_head_loss_grad(h.cuda(), w.cuda(), tc, dtable=dtable, pieces=pieces)
    only = ns.muon_head_loss(h.cuda(), w.cuda(), tc)
    assert not (got[0] < 0).any() and not (only < 0).any()
    _check((only,), want[:1], bound[:1])
    _check(got, want, bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [300, 4500])
def test_a_call_that_gave_up_returns_no_numbers(n, dtype):
    # Without a workspace of the caller's the error word is out of reach: a call
    # whose waits ran out answers NaN throughout, and the next one is right.
    v, d = 4000, 512
    h, w, t = (x.cuda() for x in _inputs(n, v, d, 21))
    start = torch.ones((v, d), dtype=dtype, device="cuda")
    args = dict(accumulate=True) if dtype == torch.float32 else {}
    ref = [x.clone() for x in ns.muon_head_loss_grad(h, w, t, dtable=start.clone(), **args)]
    alone = ns.muon_head_loss(h, w, t)
    ns.set_wait_budget(1)
    try:
        got = ns.muon_head_loss_grad(h, w, t, dtable=start.clone(), **args)
        only = ns.muon_head_loss(h, w, t)
        torch.cuda.synchronize()
    finally:
        ns.set_wait_budget(0)
    for x in (*got, only):
        assert torch.isnan(x).all()
    got = ns.muon_head_loss_grad(h, w, t, dtable=start.clone(), **args)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert torch.equal(ns.muon_head_loss(h, w, t), alone)
