"""What the binding refuses on a GPU: other types, shapes, devices, strided
tensors and short workspaces, before anything is launched."""
import pytest
import torch

import newton_schulz_07_gb300 as ns

pytestmark = pytest.mark.gpu


def _c(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_embedding():
    table, ids = _c(10, 8), _c(4, dtype=torch.int64)
    dy = _c(4, 8)
    many, mdy = _c(1600, dtype=torch.int64), _c(1600, 8)
    for error, f in (
            (TypeError, lambda: ns.muon_embed(table.half(), ids)), (TypeError, lambda: ns.muon_embed(table, ids.short())),
            (TypeError, lambda: ns.muon_embed(table, ids.cpu())), (ValueError, lambda: ns.muon_embed(table[0], ids)),
            (ValueError, lambda: ns.muon_embed(_c(8, 10).t(), ids)), (ValueError, lambda: ns.muon_embed(table, _c(8, dtype=torch.int64)[::2])),
            (ValueError, lambda: ns.muon_embed(table, ids, out=_c(4, 9))),
            (ValueError, lambda: ns.muon_embed(table, ids, out=_c(4, 8), dtype=torch.bfloat16)),
            (ns.MuonNSError, lambda: ns.muon_embed(table, ids, scale=float("nan"))),
            (ns.MuonNSError, lambda: ns.muon_embed(table, ids, out=table[:4])),
            (ValueError, lambda: ns.muon_embed_grad(dy, ids[:3], 10)), (ValueError, lambda: ns.muon_embed_grad(dy[0], ids, 10)),
            (ValueError, lambda: ns.muon_embed_grad(dy, ids, 10, accumulate=True)),
            (ValueError, lambda: ns.muon_embed_grad(dy, ids, 10, dtable=_c(9, 8))),
            (ValueError, lambda: ns.muon_embed_grad(dy, ids, 10, workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
            (ns.MuonNSError, lambda: ns.muon_embed_grad(mdy, many, 10, workspace=_c(8)))):
        with pytest.raises(error):
            f()


def test_layer_norm():
    x, w, m = _c(4, 8), _c(8), _c(4)
    big, bm = _c(30000, 8), _c(30000)
    for error, f in (
            (TypeError, lambda: ns.muon_layer_norm(x.half(), w)), (ValueError, lambda: ns.muon_layer_norm(x, w[:7])),
            (TypeError, lambda: ns.muon_layer_norm(x, w, w.bfloat16())), (ValueError, lambda: ns.muon_layer_norm(x.t(), _c(4))),
            (TypeError, lambda: ns.muon_layer_norm(x, w, out=x.bfloat16())), (ns.MuonNSError, lambda: ns.muon_layer_norm(_c(4, 0), _c(0))),
            (ns.MuonNSError, lambda: ns.muon_layer_norm(x, w, eps=-1.0)), (ValueError, lambda: ns.muon_layer_norm(_c(), w)),
            (TypeError, lambda: ns.muon_layer_norm_grad(x.bfloat16(), x, w, m, m)),
            (ValueError, lambda: ns.muon_layer_norm_grad(x[:3], x, w, m, m)), (ValueError, lambda: ns.muon_layer_norm_grad(x, x, w, m[:3], m)),
            (TypeError, lambda: ns.muon_layer_norm_grad(x, x, w, m.bfloat16(), m)),
            (ns.MuonNSError, lambda: ns.muon_layer_norm_grad(big, big, w, bm, bm, workspace=_c(1)))):
        with pytest.raises(error):
            f()


def test_head():
    b = torch.bfloat16
    h, w, t = _c(4, 16, dtype=b), _c(10, 16, dtype=b), _c(4, dtype=torch.int64)
    f, g = ns.muon_head_loss, ns.muon_head_loss_grad
    for error, call in (
            (TypeError, lambda: f(h.float(), w, t)), (TypeError, lambda: f(h, w.float(), t)), (TypeError, lambda: f(h, w, t.float())),
            (ValueError, lambda: f(h, w[:, :8].contiguous(), t)), (ValueError, lambda: f(h, w[0], t)), (ValueError, lambda: f(h, w, t[:3])),
            (ValueError, lambda: f(h, _c(16, 10, dtype=b).t(), t)), (ns.MuonNSError, lambda: f(_c(4, 12, dtype=b), _c(10, 12, dtype=b), t)),
            (ns.MuonNSError, lambda: f(h, w, t, workspace=_c(64))), (TypeError, lambda: g(h, w, t, dloss=_c(4, dtype=b))),
            (ValueError, lambda: g(h, w, t, dloss=_c(3))), (ValueError, lambda: g(h, w, t, accumulate=True)),
            (ValueError, lambda: g(h, w, t, dtable=_c(9, 16))), (TypeError, lambda: g(h, w, t, dtable=_c(10, 16, dtype=torch.float16))),
            (ns.MuonNSError, lambda: g(h, w, t, dtable=_c(10, 16, dtype=b), accumulate=True)),
            (ns.MuonNSError, lambda: g(h, w, t, dtable=w)), (ns.MuonNSError, lambda: g(h, w, t, pieces=-1)),
            (ValueError, lambda: g(h, w, t, workspace=torch.zeros(1 << 20, dtype=torch.uint8)))):
        with pytest.raises(error):
            call()


def test_axes_past_an_int():
    # 64 columns of 2^32 + 64, were a C int to keep the low bits: refused, not
    # computed on the first columns.
    n = (1 << 32) + 64
    x = torch.empty((1, n), dtype=torch.bfloat16, device="cuda")
    ids, m = _c(1, dtype=torch.int64), _c(1)
    for f in (lambda: ns.muon_embed(x, ids), lambda: ns.muon_embed_grad(x, ids, 1, dtable=torch.empty_like(x)), lambda: ns.muon_layer_norm(x, x[0]),
              lambda: ns.muon_layer_norm_grad(x, x, x[0], m, m), lambda: ns.muon_head_loss(x, x, ids),
              lambda: ns.muon_head_loss_grad(x, x, ids)):
        with pytest.raises(ns.MuonNSError):
            f()
    h = _c(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ns.MuonNSError):
        ns.muon_head_loss_grad(h, h, _c(2, dtype=torch.int64), pieces=1 << 32)
