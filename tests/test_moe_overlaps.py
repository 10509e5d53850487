"""Outputs that lie over other arrays of the same call are refused before a device is
touched."""
import pytest

from newton_schulz_07_gb300 import _lib
from test_moe_abi import _caller

BAD, ALIGN = _lib.ERR_INVALID_ARG, _lib.ERR_ALIGNMENT
A, B, C, D, E, F, G, H = (i << 32 for i in range(1, 9))

_norm = _caller("muon_rms_norm", x=A, xt=0, res=B, w=C, wt=1, rows=50, d=24, eps=1e-6, s=D, y=E, rstd=F)
_norm8 = _caller("muon_rms_norm8", x=A, xt=0, res=B, w=C, wt=1, rows=50, d=24, eps=1e-6, s=D, y=E, sc=G, rstd=F)
_norm_grad = _caller("muon_rms_norm_grad", dy=A, s=B, xt=0, w=C, wt=1, rstd=D, dsum=E, rows=40000, d=24, ds=F, dw=G, ws=H, wsb=1 << 20)


@pytest.mark.parametrize("call", [_norm, _norm8])
@pytest.mark.parametrize("kw", [dict(s=C), dict(y=C), dict(y=C - 16), dict(rstd=C), dict(rstd=A), dict(rstd=B + 4), dict(rstd=D), dict(rstd=E)])
def test_norm(call, kw):
    assert call(**kw) == BAD


def test_norm8():
    for kw in (dict(sc=A), dict(sc=B), dict(sc=C + 4), dict(sc=D), dict(sc=E + 8), dict(sc=F), dict(y=D), dict(rstd=G + 196)):
        assert _norm8(**kw) == BAD, kw
    assert _norm8(sc=F + 200) not in (BAD, ALIGN)  # right behind the last of 50


@pytest.mark.parametrize("kw", [
    dict(ds=C), dict(ds=D), dict(ds=G), dict(ds=H), dict(dw=A), dict(dw=B), dict(dw=C), dict(dw=D + 4), dict(dw=E + 8), dict(dw=F),
    dict(dw=H), dict(ws=A), dict(ws=B), dict(ws=C), dict(ws=D + 256), dict(ws=E), dict(ws=F), dict(ws=G)])
def test_norm_grad(kw):
    assert _norm_grad(**kw) == BAD


def test_arrays_that_are_not_looked_at():
    # Without a residual s is not written; few rows need no workspace.
    for call, kw in ((_norm, dict(res=None, s=E)), (_norm, dict(res=None, s=C)), (_norm_grad, dict(rows=3, ws=A)), (_norm, dict(rstd=None))):
        assert call(**kw) not in (BAD, ALIGN), kw


_quantize = _caller("muon_quantize8", x=A, xt=0, batch=2, rows=300, d=264, square=0, q=B, sc=C)


def test_quantize():
    for kw in (dict(sc=A), dict(sc=A + 2 * 2 * 300 * 264 - 4), dict(sc=B), dict(sc=B - 4 * 2 * 300 * 3 + 4)):
        assert _quantize(**kw) == BAD, kw
    for kw in (dict(sc=A + 2 * 2 * 300 * 264), dict(sc=B - 4 * 2 * 300 * 3), dict(sc=B - 4 * 2 * 3 * 3, square=1)):
        assert _quantize(**kw) not in (BAD, ALIGN), kw
    assert _quantize(sc=B - 4 * 2 * 3 * 3 + 4, square=1) == BAD


_experts = _caller("muon_experts", x=A, W=B, off=C, rows=50, e=3, o=16, d=24, y=D, err=E)
_experts_grad = _caller("muon_experts_grad", dy=A, x=B, W=C, off=D, rows=50, e=3, o=16, d=24, dx=E, dW=F, wt=1, acc=0, err=G)
_experts8 = _caller("muon_experts8", x=A, xs=B, W=C, Ws=D, off=E, rows=50, e=3, o=16, d=32, y=F, err=G)


def test_experts():
    for kw in (dict(y=C), dict(y=C - 2 * 50 * 16 + 16), dict(y=E), dict(err=A + 4), dict(err=B), dict(err=C + 12), dict(err=D + 2 * 50 * 16 - 4)):
        assert _experts(**kw) == BAD, kw
    for kw in (dict(err=C + 16), dict(err=D + 2 * 50 * 16), dict(err=None), dict(y=C + 16)):
        assert _experts(**kw) not in (BAD, ALIGN), kw


def test_experts_grad():
    for kw in (dict(dx=D), dict(dW=D), dict(dx=G), dict(dW=G), dict(err=A), dict(err=B + 8), dict(err=C), dict(err=D + 12), dict(err=E), dict(err=F)):
        assert _experts_grad(**kw) == BAD, kw
    for kw in (dict(dx=None, err=E), dict(dW=None, err=F), dict(err=D + 16)):
        assert _experts_grad(**kw) not in (BAD, ALIGN), kw


def test_experts8():
    for kw in (dict(y=E), dict(y=G), dict(err=A), dict(err=B + 196), dict(err=C), dict(err=D + 8), dict(err=E), dict(err=F)):
        assert _experts8(**kw) == BAD, kw
    for kw in (dict(err=B + 200), dict(err=D + 12)):
        assert _experts8(**kw) not in (BAD, ALIGN), kw


_combine_grad = _caller("muon_combine_grad", dout=A, y=B, yt=0, s=C, g=D, n=50, k=2, rows=900, d=24, dy=E, dg=F)


def test_combine_grad():
    for kw in (dict(dg=A), dict(dg=A + 2 * 50 * 24 - 4), dict(dg=B + 8), dict(dg=B + 2 * 900 * 24 - 4)):
        assert _combine_grad(**kw) == BAD, kw
        assert _combine_grad(**kw, dy=None) == BAD, kw
    for kw in (dict(dg=A + 2 * 50 * 24), dict(dg=B + 2 * 900 * 24)):
        assert _combine_grad(**kw) not in (BAD, ALIGN), kw
