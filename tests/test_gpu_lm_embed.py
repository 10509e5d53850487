"""Token embedding and its gradient against their definitions in 64 bits.

Bounds, with e = 2^-24 (fp32 unit roundoff) and u the result type's: the
lookup rounds the fp32 product and the result; a gradient row of k tokens is a
sum of k fp32 terms in some order, off by at most k e times the sum of their
magnitudes, then scaled and rounded."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}  # one rounding and the fp32 product's
TINY = 1e-37


def _ids(n, vocab, seed, dtype=torch.int64, bad=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(n, generator=g, dtype=torch.float64) ** 3 * vocab).long().clamp_(0, max(vocab - 1, 0))
    out = torch.tensor([-1, -100, vocab, vocab + 5])[torch.randint(0, 4, (n,), generator=g)]
    return torch.where(torch.rand(n, generator=g) < bad, out, ids).to(dtype)


def _values(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _rows(ids, vocab):
    return [(t, int(v)) for t, v in enumerate(ids.tolist()) if 0 <= v < vocab]


def _grad64(dy, ids, vocab, scale):
    """(exact gradient, sum of magnitudes, tokens per row) in 64 bits."""
    ok = (ids >= 0) & (ids < vocab)
    at, d = ids[ok].long(), dy[ok].double()
    z = torch.zeros((vocab, dy.shape[1]), dtype=torch.float64)
    return (z.index_add(0, at, d) * scale, z.index_add(0, at, d.abs()) * abs(scale),
            torch.zeros(vocab, dtype=torch.float64).index_add(0, at, torch.ones(len(at), dtype=torch.float64)))


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 1, 1), (1, 50, 8), (3, 7, 5), (17, 100, 24), (130, 33, 1000),
                                               (1025, 1000, 260), (77, 999, 2056), (5, 40, 8194)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("ids_type", [torch.int32, torch.int64])
def test_lookup(tokens, vocab, dim, types, ids_type):
    ti, to = ({"bf16": torch.bfloat16, "fp32": torch.float32}[t] for t in types)
    table = _values((vocab, dim), 1, ti)
    ids = _ids(tokens, vocab, 2, ids_type)
    scale = float(torch.tensor(1.7))
    got = ns.muon_embed(table.cuda(), ids.cuda(), scale=scale, dtype=to)
    assert got.dtype == to and got.shape == (tokens, dim)
    ok = (ids >= 0) & (ids < vocab)
    ref = table.double()[torch.where(ok, ids, 0).long()] * scale * ok[:, None]
    assert torch.all((got.cpu().double() - ref).abs() <= (U[to] + 2 * E) * ref.abs() + TINY)


def test_lookup_of_no_tokens_and_from_an_empty_table():
    table = torch.ones((4, 8), device="cuda")
    assert ns.muon_embed(table, torch.zeros((0,), dtype=torch.int64, device="cuda")).shape == (0, 8)
    out = ns.muon_embed(table[:0], torch.zeros((3,), dtype=torch.int64, device="cuda"))
    assert torch.equal(out, torch.zeros_like(out))


def test_lookup_keeps_the_ids_shape_and_any_alignment():
    table = _values((60, 24), 3, torch.bfloat16).cuda()
    ids = _ids(30, 60, 4, bad=0).cuda()
    ref = ns.muon_embed(table, ids)
    assert torch.equal(ns.muon_embed(table, ids.view(5, 3, 2)), ref.view(5, 3, 2, 24))
    for shift in (1, 2, 4):  # a table and an output that start inside a 16-byte line
        room = torch.zeros(60 * 24 + 8, dtype=torch.bfloat16, device="cuda")
        moved = room[shift:shift + 60 * 24].view(60, 24)
        moved.copy_(table)
        assert torch.equal(ns.muon_embed(moved, ids), ref)
        out = torch.zeros(30 * 24 + 8, dtype=torch.bfloat16, device="cuda")
        ns.muon_embed(table, ids, out=out[shift:shift + 30 * 24].view(30, 24))
        assert torch.equal(out[shift:shift + 30 * 24].view(30, 24), ref)
        assert not out[:shift].any() and not out[shift + 30 * 24:].any()


GRAD = [(1, 1, 1), (1, 5, 8), (2, 3, 3), (31, 7, 20), (32, 7, 64), (33, 2, 257), (64, 1, 264), (65, 1000, 40),
        (257, 33, 1000), (256, 100, 72), (512, 100, 72), (1025, 100, 72), (500, 2, 9), (1000, 70000, 24), (2047, 130, 16), (2049, 130, 16), (5000, 17, 72), (20000, 3, 8),
        (40001, 300000, 9), (16384, 513, 520)]


@pytest.mark.parametrize("tokens,vocab,dim", GRAD)
@pytest.mark.parametrize("types", [("bf16", "fp32"), ("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(tokens, vocab, dim, types, accumulate):
    ti, to = ({"bf16": torch.bfloat16, "fp32": torch.float32}[t] for t in types)
    dy = _values((tokens, dim), 5, ti)
    ids = _ids(tokens, vocab, 6, torch.int32 if tokens % 2 else torch.int64)
    scale = float(torch.tensor(-0.3))
    start = _values((vocab, dim), 7, to) if accumulate else None
    exact, size, count = _grad64(dy, ids, vocab, scale)
    got = (start.clone().cuda() if accumulate
           else torch.full((vocab, dim), float("nan"), dtype=to, device="cuda"))
    r = ns.muon_embed_grad(dy.cuda(), ids.cuda(), vocab, scale=scale, dtable=got, accumulate=accumulate)
    assert r is got
    bound = (count[:, None] + 2) * E * size
    if accumulate:
        exact = exact + start.double()
        bound = bound + E * exact.abs()
    off = (got.cpu().double() - exact).abs()
    assert torch.all(off <= bound + U[to] * (exact.abs() + bound) + TINY)
    if accumulate:  # rows without tokens are left alone, bit for bit
        assert torch.equal(got.cpu()[count == 0], start[count == 0])


@pytest.mark.parametrize("tokens,vocab,dim", [(257, 50257, 256), (1023, 20011, 601), (4096, 700, 20000), (4097, 30000, 401),
                                              (300, 900000, 40)])
@pytest.mark.parametrize("to", [torch.float32, torch.bfloat16])
def test_gradient_into_large_tables(tokens, vocab, dim, to):
    # Tables whose zeroing takes longer than ranking the tokens, on both sides
    # of the sizes that divide it; every row is written, whatever it held.
    dy, ids = _values((tokens, dim), 31, torch.bfloat16).cuda(), _ids(tokens, vocab, 32).cuda()
    got = torch.full((vocab, dim), float("nan"), dtype=to, device="cuda")
    ns.muon_embed_grad(dy, ids, vocab, dtable=got)
    ok = (ids >= 0) & (ids < vocab)
    rows, at = torch.unique(ids[ok], return_inverse=True)
    z = torch.zeros((len(rows), dim), dtype=torch.float64, device="cuda")
    exact, size = z.index_add(0, at, dy[ok].double()), z.index_add(0, at, dy[ok].double().abs())
    bound = (torch.bincount(at)[:, None] + 2) * E * size
    assert torch.all((got[rows].double() - exact).abs() <= bound + U[to] * (exact.abs() + bound) + TINY)
    got[rows] = 0
    assert not got.any()


@pytest.mark.parametrize("tokens", [33, 3000, 70000])
def test_gradient_of_one_token_repeated(tokens):
    # One row takes every token: a sum over pieces, sorted by one CTA or several.
    dy = _values((tokens, 40), 8, torch.float32)
    ids = torch.full((tokens,), 2, dtype=torch.int64)
    exact, size, count = _grad64(dy, ids, 5, 1.0)
    got = ns.muon_embed_grad(dy.cuda(), ids.cuda(), 5).cpu().double()
    assert torch.all((got - exact).abs() <= (count[:, None] + 2) * E * size + TINY)


def test_gradient_is_the_adjoint_of_the_lookup():
    # <embed(D), dY> = <D, embed_grad(dY)>, both sides summed in 64 bits.
    tokens, vocab, dim = 700, 90, 136
    D, dy = _values((vocab, dim), 9, torch.float32).cuda(), _values((tokens, dim), 10, torch.float32).cuda()
    ids = _ids(tokens, vocab, 11).cuda()
    a = (ns.muon_embed(D, ids, scale=0.5).double() * dy.double())
    b = (D.double() * ns.muon_embed_grad(dy, ids, vocab, scale=0.5).double())
    assert abs(float(a.sum() - b.sum())) <= 4 * tokens * E * float(a.abs().sum())


def test_gradient_is_deterministic_and_takes_any_alignment():
    tokens, vocab, dim = 9000, 400, 48
    dy, ids = _values((tokens, dim), 12, torch.bfloat16).cuda(), _ids(tokens, vocab, 13).cuda()
    ref = ns.muon_embed_grad(dy, ids, vocab)
    for _ in range(3):
        assert torch.equal(ns.muon_embed_grad(dy, ids, vocab), ref)
    room = torch.zeros(tokens * dim + 8, dtype=torch.bfloat16, device="cuda")
    moved = room[3:3 + tokens * dim].view(tokens, dim)
    moved.copy_(dy)
    assert torch.equal(ns.muon_embed_grad(moved, ids, vocab), ref)


def test_masked_tokens_touch_nothing():
    # NaN and infinity in the rows of masked tokens stay out of the gradient,
    # and a NaN row of one token stays in that token's row.
    tokens, vocab, dim = 500, 40, 24
    dy, ids = _values((tokens, dim), 14, torch.float32), _ids(tokens, vocab, 15, bad=0.3)
    bad = (ids < 0) | (ids >= vocab)
    ref = ns.muon_embed_grad(dy.cuda(), ids.cuda(), vocab)
    dirty = dy.clone()
    dirty[bad] = float("nan")
    dirty[bad.nonzero()[::2, 0]] = float("inf")
    assert torch.equal(ns.muon_embed_grad(dirty.cuda(), ids.cuda(), vocab), ref)
    one = int((~bad).nonzero()[7, 0])
    dirty[one] = float("nan")
    got = ns.muon_embed_grad(dirty.cuda(), ids.cuda(), vocab)
    hit = torch.zeros(vocab, dtype=torch.bool)
    hit[ids[one]] = True
    assert torch.equal(torch.isnan(got).all(1).cpu(), hit) and torch.equal(got[~hit.cuda()], ref[~hit.cuda()])


def test_gradient_without_any_token():
    ids = torch.full((50,), -1, dtype=torch.int32, device="cuda")
    dy = torch.full((50, 16), float("nan"), device="cuda")
    assert torch.equal(ns.muon_embed_grad(dy, ids, 9), torch.zeros((9, 16), device="cuda"))
    assert torch.equal(ns.muon_embed_grad(dy[:0], ids[:0], 9), torch.zeros((9, 16), device="cuda"))
    keep = torch.ones((9, 16), device="cuda")
    ns.muon_embed_grad(dy, ids, 9, dtable=keep, accumulate=True)
    ns.muon_embed_grad(dy[:0], ids[:0], 9, dtable=keep, accumulate=True)
    assert torch.equal(keep, torch.ones_like(keep))


def test_rows_beyond_32_bit_offsets():
    # A table of more than 2^32 bytes and 2^31 elements: the last rows.
    vocab, dim = 270000, 8200
    table = torch.zeros((vocab, dim), dtype=torch.bfloat16, device="cuda")
    table[-2:] = _values((2, dim), 16, torch.bfloat16).cuda()
    ids = torch.tensor([vocab - 1, 0, vocab - 2], device="cuda")
    assert torch.equal(ns.muon_embed(table, ids), table[ids])
    dy = _values((3, dim), 17, torch.bfloat16).cuda()
    ns.muon_embed_grad(dy, ids, vocab, dtable=table)
    assert torch.equal(table[ids], dy)
    assert int(torch.count_nonzero(table.view(torch.int16))) == int(torch.count_nonzero(dy.view(torch.int16)))


def test_other_streams_and_graph_replay():
    tokens, vocab, dim = 3000, 200, 64
    dy, ids = _values((tokens, dim), 18, torch.bfloat16).cuda(), _ids(tokens, vocab, 19).cuda()
    ref = ns.muon_embed_grad(dy, ids, vocab)
    table = ref.clone()
    look = ns.muon_embed(table, ids)
    ws = torch.empty(ns.embed_grad_workspace_size(tokens, vocab, dim), dtype=torch.uint8, device="cuda")
    got, out = torch.empty_like(ref), torch.empty_like(look)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ns.muon_embed_grad(dy, ids, vocab, dtable=got, workspace=ws)
        ns.muon_embed(got, ids, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref) and torch.equal(out, look)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ns.muon_embed_grad(dy, ids, vocab, dtable=got, workspace=ws)
        ns.muon_embed(got, ids, out=out)
    dy2 = dy * 2  # exact, so the sums double exactly
    dy.copy_(dy2)
    got.zero_()
    ws.fill_(255)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ref * 2) and torch.equal(out, look * 2)
