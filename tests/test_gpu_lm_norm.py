"""Layer norm and its gradient against their definitions in 64 bits.

Bounds, with e = 2^-24: a row's sums are taken over at most 32 terms a thread
(16 backward) and a tree over the threads, so a sum is off by at most S e times the
sum of magnitudes with S = 64 for rows of up to 32768 (16384 backward) elements
and S = 64 + dim / 1024 beyond."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(1, 1), (1, 8), (3, 5), (2, 31), (9, 768), (1, 1001), (33, 1024), (130, 2050), (7, 4096), (5, 4099), (301, 264),
          (4, 8192), (3, 8200), (2, 16384), (2, 16390), (2, 32768), (2, 32776), (3, 40001), (384, 300), (385, 300), (48, 4096), (49, 4096)]


def _values(shape, seed, dtype, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def _terms(dim):
    return 64 + dim / 1024


def _stats64(x, eps):
    x = x.double()
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    return mean, var, (var + eps).rsqrt()


def _forward_bound(x, w, b, eps):
    """Exact (y, mean, rstd) and the bounds of each, before y's rounding."""
    S, xd = _terms(x.shape[-1]), x.double()
    mean, var, rstd = _stats64(x, eps)
    dm = S * E * xd.abs().mean(-1)
    # The variance about a mean that is off by dm is off by dm^2; each square by 4 e.
    dv = (S + 6) * E * var + dm ** 2
    dr = rstd * (0.5 * dv / (var + eps) + 6 * E)
    wd = w.double()
    c = xd - mean[..., None]
    y = c * rstd[..., None] * wd + (0 if b is None else b.double())
    dy = wd.abs() * (rstd[..., None] * dm[..., None] + c.abs() * (dr[..., None] + 4 * E * rstd[..., None]))
    # dr may be as large as rstd where the variance vanishes against the mean's error.
    dy = dy + wd.abs() * dm[..., None] * dr[..., None] + 2 * E * y.abs()
    return (y, dy), (mean, dm + E * mean.abs()), (rstd, dr)


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_forward(rows, dim, types):
    x = _values((rows, dim), 1, T[types[0]], 1.5, 0.5)
    w, b = _values((dim,), 2, T[types[1]], 0.3, 1.0), _values((dim,), 3, T[types[1]])
    for bias in (b, None):
        got = ns.muon_layer_norm(x.cuda(), w.cuda(), None if bias is None else bias.cuda(), eps=1e-5)
        want = _forward_bound(x, w, bias, 1e-5)
        for g, (ref, bound), u in zip(got, want, (U[x.dtype], 0, 0)):
            assert torch.all((g.cpu().double() - ref).abs() <= bound + u * (ref.abs() + bound) + 1e-37)


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_gradient_against_the_formula(rows, dim, types):
    x, dy = _values((rows, dim), 4, T[types[0]], 1.5, 0.5), _values((rows, dim), 5, T[types[0]])
    w = _values((dim,), 6, T[types[1]], 0.3, 1.0)
    mean, _, rstd = _stats64(x, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    dx, dw, db = ns.muon_layer_norm_grad(dy.cuda(), x.cuda(), w.cuda(), mean.cuda(), rstd.cuda())
    S = _terms(dim)
    r, g = rstd.double()[:, None], dy.double()
    xh = (x.double() - mean.double()[:, None]) * r
    dxh = 2 * E * xh.abs() + E * r * (x.double().abs() + mean.double().abs()[:, None])  # the subtraction and the product
    a = g * w.double()
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    d1 = (S + 2) * E * a.abs().mean(1, keepdim=True)
    d2 = (S + 3) * E * (a * xh).abs().mean(1, keepdim=True) + (a.abs() * dxh).mean(1, keepdim=True)
    ref = r * (a - m1 - xh * m2)
    bound = r * (d1 + xh.abs() * d2 + dxh * m2.abs() + 6 * E * (a.abs() + m1.abs() + (xh * m2).abs()))
    bound = bound * 1.01  # products of two of these errors
    assert torch.all((dx.cpu().double() - ref).abs() <= bound + U[x.dtype] * (ref.abs() + bound) + 1e-37)
    n = rows + 64
    for got, t, extra in ((dw, g * xh, (g.abs() * dxh).sum(0)), (db, g, 0)):
        assert got.dtype == torch.float32
        assert torch.all((got.cpu().double() - t.sum(0)).abs() <= n * E * t.abs().sum(0) + extra * 1.01 + 1e-37)
    dx2, dw2, none = ns.muon_layer_norm_grad(dy.cuda(), x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), bias=False)
    assert none is None and torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dim", [5, 264, 4100])
def test_gradient_against_differences(dim):
    # d/dt of <layer_norm(x + t u; w + t v, b + t v), dy> from central differences in 64 bits.
    rows, h = 6, 1e-4
    x, dy = _values((rows, dim), 7, torch.float32).double(), _values((rows, dim), 8, torch.float32).double()
    w, b = _values((dim,), 9, torch.float32, 0.3, 1.0).double(), _values((dim,), 10, torch.float32).double()
    u, v = _values((rows, dim), 11, torch.float32).double(), _values((dim,), 12, torch.float32).double()

    def f(t):
        xx = x + t * u
        m, _, r = _stats64(xx, 1e-3)
        return float((((xx - m[:, None]) * r[:, None] * (w + t * v) + b + t * v) * dy).sum())

    slope = (f(h) - f(-h)) / (2 * h)
    y, mean, rstd = ns.muon_layer_norm(x.float().cuda(), w.float().cuda(), b.float().cuda(), eps=1e-3)
    dx, dw, db = ns.muon_layer_norm_grad(dy.float().cuda(), x.float().cuda(), w.float().cuda(), mean, rstd)
    parts = [(dx.cpu().double() * u), (dw.cpu().double() * v), (db.cpu().double() * v)]
    got = sum(float(p.sum()) for p in parts)
    # Differences: h^2 times a third derivative of order one a row; the kernels: 256 e of what is added up.
    size = sum(float(p.abs().sum()) for p in parts)
    assert abs(got - slope) <= 256 * E * size + 100 * h * h * size


def test_constant_rows_and_large_means():
    # No variance: y is the bias and rstd is 1 / sqrt(eps).  A mean of 1e4
    # standard deviations: the variance is taken about it, so it stays right.
    w, b = torch.ones(512, device="cuda"), _values((512,), 13, torch.float32).cuda()
    x = torch.full((3, 512), 2.5, device="cuda")
    y, mean, rstd = ns.muon_layer_norm(x, w, b, eps=1e-4)
    assert torch.equal(y, b.expand(3, 512)) and torch.equal(mean, torch.full((3,), 2.5, device="cuda"))
    assert torch.all((rstd - 100.0).abs() <= 1e-4)
    x = _values((4, 512), 14, torch.float32, 1.0, 1e4)
    got = ns.muon_layer_norm(x.cuda(), w, b)
    for g, (ref, bound) in zip(got, _forward_bound(x, w.cpu(), b.cpu(), 1e-5)):
        assert torch.all((g.cpu().double() - ref).abs() <= bound + 2 * E * ref.abs())


def test_a_bad_row_stays_in_its_row():
    x = _values((40, 264), 15, torch.float32).cuda()
    dy, w = _values((40, 264), 16, torch.float32).cuda(), torch.ones(264, device="cuda")
    y, mean, rstd = ns.muon_layer_norm(x, w)
    dx = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)[0]
    x2 = x.clone()
    x2[7, 3], x2[11, 5] = float("nan"), float("inf")
    y2, mean2, rstd2 = ns.muon_layer_norm(x2, w)
    dx2 = ns.muon_layer_norm_grad(dy, x2, w, mean2, rstd2)[0]
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[7] = keep[11] = False
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.isnan(y2[7]).all() and torch.isnan(dx2[7]).all() and torch.isnan(y2[11, 5])


def test_in_place_and_any_alignment_and_shapes():
    for dim in (264, 4096, 40000):
        x, dy = _values((6, dim), 17, torch.bfloat16).cuda(), _values((6, dim), 18, torch.bfloat16).cuda()
        w, b = _values((dim,), 19, torch.float32).cuda(), _values((dim,), 20, torch.float32).cuda()
        y, mean, rstd = ns.muon_layer_norm(x, w, b)
        dx, dw, db = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)
        xi = x.clone()
        assert torch.equal(ns.muon_layer_norm(xi, w, b, out=xi)[0], y) and torch.equal(xi, y)
        for name in ("dy", "x"):
            xi, gi = x.clone(), dy.clone()
            got = ns.muon_layer_norm_grad(gi, xi, w, mean, rstd, dx=gi if name == "dy" else xi)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
        y3, m3, _ = ns.muon_layer_norm(x.view(2, 3, dim), w, b)
        assert torch.equal(y3.view(6, dim), y) and m3.shape == (2, 3)
        y1, m1, r1 = ns.muon_layer_norm(x[0], w, b)
        assert torch.equal(y1, y[0]) and m1.shape == ()
        room = torch.zeros(6 * dim + 8, dtype=torch.bfloat16, device="cuda")
        moved = room[1:1 + 6 * dim].view(6, dim)
        moved.copy_(x)
        ym, mm, rm = ns.muon_layer_norm(moved, w, b)
        # Another width of access sums in another order.
        assert torch.all((mm - mean).abs() <= 128 * E * x.float().abs().mean(1))
        assert torch.all((ym.float() - y.float()).abs() <= 2.0 ** -7 * y.float().abs() + 1e-4)


def test_no_rows():
    x, w = torch.empty((0, 24), device="cuda"), torch.ones(24, device="cuda")
    y, mean, rstd = ns.muon_layer_norm(x, w)
    assert y.shape == (0, 24) and mean.shape == (0,)
    dx, dw, db = ns.muon_layer_norm_grad(x, x, w, mean, rstd)
    assert dx.shape == (0, 24) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows,dim", [(100003, 33), (70001, 72), (40011, 264), (20011, 1001), (6001, 2050), (4001, 4099),
                                      (2003, 8199), (1901, 16384), (5003, 6020)])
@pytest.mark.parametrize("types", [("bf16", "fp32"), ("fp32", "bf16")])
def test_many_rows(rows, dim, types):
    # Rows in turns of a grid that stays; odd lengths start on any byte pair.
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn((rows, dim), generator=g, device="cuda").mul_(1.5).add_(s).to(T[types[0]]) for s in (0.5, 0.0))
    w, b = (torch.randn(dim, generator=g, device="cuda").to(T[types[1]]) for _ in range(2))
    y, mean, rstd = ns.muon_layer_norm(x, w, b)
    dx, dw, db = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)
    S, sums, size = _terms(dim), [0, 0], [0, 0]
    for i in range(0, rows, 4096):
        q = slice(i, i + 4096)
        want = _forward_bound(x[q], w, b, 1e-5)
        for got, (ref, bound), u in zip((y[q], mean[q], rstd[q]), want, (U[x.dtype], 0, 0)):
            assert torch.all((got.double() - ref).abs() <= bound + u * (ref.abs() + bound) + 1e-37)
        r, gr = rstd[q].double()[:, None], dy[q].double()
        xh = (x[q].double() - mean[q].double()[:, None]) * r
        a = gr * w.double()
        m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
        ref = r * (a - m1 - xh * m2)
        e1, e2 = (S + 8) * E * a.abs().mean(1, keepdim=True), (S + 16) * E * (a * xh).abs().mean(1, keepdim=True)
        bound = r * (e1 + xh.abs() * e2 + 16 * E * (a.abs() + m1.abs() + (xh * m2).abs()))
        assert torch.all((dx[q].double() - ref).abs() <= bound + U[x.dtype] * (ref.abs() + bound) + 1e-37)
        for k, t in enumerate((gr * xh, gr)):
            sums[k], size[k] = sums[k] + t.sum(0), size[k] + t.abs().sum(0)
    for got, ref, s in zip((dw, db), sums, size):
        assert torch.all((got.double() - ref).abs() <= (rows / 64 + 128) * E * s)


def test_many_rows_and_determinism():
    x, dy = _values((70001, 72), 21, torch.bfloat16).cuda(), _values((70001, 72), 22, torch.bfloat16).cuda()
    w = torch.ones(72, device="cuda")
    y, mean, rstd = ns.muon_layer_norm(x, w)
    dx, dw, db = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, t in ((dw, dy.double() * xh), (db, dy.double())):
        assert torch.all((got.double() - t.sum(0)).abs() <= 1024 * E * t.abs().sum(0))
    for _ in range(3):
        again = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))


def test_other_stream_and_graph_replay():
    x, dy = _values((50, 520), 23, torch.bfloat16).cuda(), _values((50, 520), 24, torch.bfloat16).cuda()
    w = _values((520,), 25, torch.float32).cuda()
    y, mean, rstd = ns.muon_layer_norm(x, w)
    ref = ns.muon_layer_norm_grad(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, m2, r2 = ns.muon_layer_norm(x, w)
        got = ns.muon_layer_norm_grad(dy, x, w, m2, r2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y2, y) and all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3, m3, r3 = ns.muon_layer_norm(x, w)
        got3 = ns.muon_layer_norm_grad(dy, x, w, m3, r3)
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, y.flip(0)) and torch.equal(got3[0], ref[0].flip(0))
